"""The query-side operators on the GPU against fp64 references: rotate (norm
and RoPE), append (into the paged cache) and attend (paged attention with a
shared prefix), their padding, masks, strides, errors, streams and graphs."""
import math

import pytest
import torch

from query_cases import BF, Paged, attend_reference, inv_freq, rotate_tolerance, rotated

pytestmark = pytest.mark.gpu

LLAMA3 = (8.0, 1.0, 4.0, 8192)


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_injection_gather_b200 as p
    return p


def make(pkg, D, H, interleaved=False, theta=1e4, llama3=None, layers=2):
    style = pkg.IS_ROPE_INTERLEAVED if interleaved else pkg.IS_ROPE_ROTATE_HALF
    l3 = dict(factor=llama3[0], low_freq_factor=llama3[1], high_freq_factor=llama3[2],
              original_max_position=llama3[3]) if llama3 else None
    return pkg.FactStore(layers, H, D, pkg.RopeConfig(theta=theta, style=style, llama3=l3), capacity_tokens=256,
                         max_facts=8, max_batch_requests=16, max_batch_fact_ids=16, max_batch_blocks=64)


def within(got, ref, tol):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(),
                           float((got.double() - ref).abs()[bad].max()), float(ref[bad][0]), float(tol[bad][0]))


# ---------------------------------------------------------------- rotate

@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,Hq,H", [(1, 4, 1), (7, 14, 2), (130, 5, 3)])
def test_rotate(pkg, D, interleaved, norm, T, Hq, H):
    g = torch.Generator(device="cuda").manual_seed(D + T)
    qkv = torch.randn(T, Hq + 2 * H, D, device="cuda", generator=g).to(BF)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + H]
    pos = torch.randint(0, 140000, (T,), device="cuda", dtype=torch.int32, generator=g)
    pos[0] = 2 ** 31 - 1 if T > 1 else 0
    qw = (1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(BF) if norm else None
    kw = (1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(BF) if norm else None
    llama3 = LLAMA3 if D == 128 else None
    with make(pkg, D, H, interleaved, 5e5, llama3) as s:
        qo, ko = s.rotate(q, pos, k=k, q_weight=qw, k_weight=kw, eps=1e-5)
        f = inv_freq(D, 5e5, llama3)
        for got, x, w in ((qo, q, qw), (ko, k, kw)):
            ref, mag = rotated(x, w, 1e-5, pos, f, interleaved)
            # both sides' angles are an fp64 product: off by 2^-52 of itself
            far = 2.0 ** -51 * pos.double()[:, None, None] * mag
            within(got, ref, rotate_tolerance(ref, mag) + far)
        only, none = s.rotate(q, pos, q_weight=qw, eps=1e-5)
        assert none is None and torch.equal(only, qo)
        assert s.last_query_error() == (0, 0)


def test_rotate_norm_on_one_of_the_two(pkg):
    """Query and key rows of one warp, one normed and the other not."""
    T, Hq, H, D = 5, 3, 2, 64
    x = torch.randn(T, Hq + H, D, device="cuda").to(BF)
    q, k = x[:, :Hq].contiguous(), x[:, Hq:].contiguous()
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 11
    w = torch.rand(D, device="cuda").to(BF)
    with make(pkg, D, H) as s:
        f = inv_freq(D, 1e4)
        for qw, kw in ((w, None), (None, w)):
            qo, ko = s.rotate(q, pos, k=k, q_weight=qw, k_weight=kw)
            for got, src, wt in ((qo, q, qw), (ko, k, kw)):
                ref, mag = rotated(src, wt, 1e-6, pos, f, False)
                within(got, ref, rotate_tolerance(ref, mag))


def test_rotate_in_place_and_padding(pkg):
    T, Hq, H, D = 9, 6, 2, 128
    x = torch.randn(T, Hq + H, D, device="cuda").to(BF)
    pos = torch.tensor([3, -1, 0, 900, -5, 77, 1, 2, -2147483648], device="cuda", dtype=torch.int32)
    with make(pkg, D, H) as s:
        want_q = torch.full((T, Hq, D), 9.0, device="cuda", dtype=BF)
        want_k = torch.full((T, H, D), 9.0, device="cuda", dtype=BF)
        s.rotate(x[:, :Hq], pos, k=x[:, Hq:], q_out=want_q, k_out=want_k)
        assert (want_q[pos < 0] == 9).all() and (want_k[pos < 0] == 9).all()
        y = x.clone()
        s.rotate(y[:, :Hq], pos, k=y[:, Hq:], q_out=y[:, :Hq], k_out=y[:, Hq:])
        assert torch.equal(y[pos >= 0, :Hq], want_q[pos >= 0]) and torch.equal(y[pos >= 0, Hq:], want_k[pos >= 0])
        assert torch.equal(y[pos < 0], x[pos < 0])
        # non-finite inputs stay in their pair
        z = torch.randn(1, 1, D, device="cuda").to(BF)
        z[0, 0, 5] = math.nan
        z[0, 0, 9] = math.inf
        o, _ = s.rotate(z, torch.tensor([7], device="cuda", dtype=torch.int32))
        odd = torch.zeros(D, dtype=torch.bool, device="cuda")
        odd[[5, 9, 5 + D // 2, 9 + D // 2]] = True
        assert torch.equal(~torch.isfinite(o[0, 0]), odd)
        e, _ = s.rotate(x[:0, :Hq], pos[:0])
        assert e.shape == (0, Hq, D)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("D,H,Hq,block,head_major,interleaved", [
    (128, 8, 32, 16, False, False), (128, 4, 28, 32, True, False), (64, 2, 14, 24, True, True), (32, 1, 1, 1, False, False),
    (256, 2, 4, 128, False, True), (64, 3, 9, 5, False, False)])
@pytest.mark.parametrize("T", [1, 45])
@pytest.mark.parametrize("norm", [False, True])
def test_append(pkg, D, H, Hq, block, head_major, interleaved, T, norm):
    nb, layers, layer = -(-T * 2 // block) + 2, 3, 1
    shape = (layers, nb, H, block, D) if head_major else (layers, nb, block, H, D)
    kc, vc = (torch.randn(shape, device="cuda").to(BF) for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    qkv = torch.randn(T, Hq + 2 * H, D, device="cuda").to(BF)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    pos = torch.randint(0, 100000, (T,), device="cuda", dtype=torch.int32)
    slots = torch.randperm(nb * block, device="cuda")[:T].contiguous()
    if T > 1:
        slots[3], pos[7], pos[9] = -1, -1, -3
        slots[9] = 10 ** 15  # of a padding token: not looked at
    w = (1 + 0.3 * torch.randn(D, device="cuda")).to(BF) if norm else None
    with make(pkg, D, H, interleaved, layers=layers) as s:
        cache = pkg.cache_desc(kc, vc, head_major=head_major)
        qo = torch.full((T, Hq, D), 5.0, device="cuda", dtype=BF)
        s.append(k, v, pos, slots, cache, layer, k_weight=w, q=q, q_weight=w, q_out=qo)
        assert s.last_query_error() == (0, 0)
        f = inv_freq(D, 1e4)
        live = pos >= 0
        ref, mag = rotated(q, w, 1e-6, pos, f, interleaved)
        within(qo[live], ref[live], rotate_tolerance(ref, mag)[live])
        assert (qo[~live] == 5).all()
        kept = (slots >= 0) & live
        ref, mag = rotated(k, w, 1e-6, pos, f, interleaved)
        b, o = slots[kept] // block, slots[kept] % block
        view = (lambda c: c[layer].transpose(1, 2) if head_major else c[layer])
        within(view(kc)[b, o], ref[kept], rotate_tolerance(ref, mag)[kept])
        assert torch.equal(view(vc)[b, o], v[kept])
        # nothing else changed
        view(k0)[b, o] = view(kc)[b, o]
        view(v0)[b, o] = view(vc)[b, o]
        assert torch.equal(kc, k0) and torch.equal(vc, v0)
        # without queries: the same cache
        k2, v2 = kc.clone(), vc.clone()
        view(k2)[b, o] = 0
        view(v2)[b, o] = 0
        assert s.append(k, v, pos, slots, pkg.cache_desc(k2, v2, head_major=head_major), layer, k_weight=w) is None
        assert torch.equal(k2, kc) and torch.equal(v2, vc)


def test_append_agrees_with_inject(pkg):
    """A fact's keys appended token by token are the keys that inject writes:
    both are the bf16 rounding of an fp32 rotation by the same angles, whose
    roundings differ only next to a midpoint."""
    L, H, D, n, B = 2, 4, 128, 200, 16
    k = torch.randn(L, H, n, D).to(BF)
    v = torch.randn(L, H, n, D).to(BF)
    with make(pkg, D, H, theta=5e5, llama3=LLAMA3) as s:
        s.put_fact(k, v)
        nb = 20
        shape = (L, nb, B, H, D)
        kc, vc, ka, va = (torch.zeros(shape, dtype=BF, device="cuda") for _ in range(4))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        table = torch.randperm(nb)[:nb].to(torch.int32).cuda().view(1, nb)
        slots = torch.empty(n, dtype=torch.int64, device="cuda")
        s.inject(i32([0, 1]), i32([0]), i32([37]), table, pkg.cache_desc(kc, vc), slots)
        assert s.last_error()[0] == 0
        pos = torch.arange(37, 37 + n, dtype=torch.int32, device="cuda")
        for layer in range(L):
            s.append(k[layer].transpose(0, 1).contiguous().cuda(), v[layer].transpose(0, 1).contiguous().cuda(), pos,
                     slots, pkg.cache_desc(ka, va), layer)
        assert s.last_query_error() == (0, 0)
        assert torch.equal(va, vc)
        same = (ka == kc).float().mean()
        assert same > 0.999
        assert (ka.double() - kc.double()).abs().max() <= 2.0 ** -7 * kc.double().abs().max()


def test_append_bad_slot_is_recorded_and_skipped(pkg):
    D, H, B, nb, T = 64, 2, 16, 4, 6
    kc, vc = (torch.zeros(1, nb, B, H, D, dtype=BF, device="cuda") for _ in range(2))
    k, v = (torch.randn(T, H, D, device="cuda").to(BF) for _ in range(2))
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    with make(pkg, D, H, layers=1) as s:
        for bad in (nb * B, -2, 2 ** 40):
            slots = torch.tensor([0, 5, bad, 9, 33, 63], device="cuda")
            kc.zero_(), vc.zero_()
            s.append(k, v, pos, slots, pkg.cache_desc(kc, vc))
            rc, detail = s.last_query_error()
            assert (rc, detail) == (pkg.IS_ERR_BAD_BLOCK, 2)
            assert s.last_query_error() == (0, 0)
            got = vc.view(nb * B, H, D)
            keep = [0, 1, 3, 4, 5]
            assert torch.equal(got[slots[keep]], v[keep])
            rest = torch.ones(nb * B, dtype=torch.bool, device="cuda")
            rest[slots[keep]] = False
            assert (got[rest] == 0).all()


# ---------------------------------------------------------------- attend

def check_attend(pkg, c, causal=True, scale=None, lse=True, **kw):
    with make(pkg, c.D, c.H) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache, head_major=c.head_major)
        T, Hq = c.q.shape[:2]
        out = torch.full((T, Hq, c.D), 3.0, dtype=BF, device="cuda")
        l = torch.full((T, Hq), 7.0, device="cuda") if lse else None
        c.call(s, cache, causal, out=out, lse=l, scale=scale, **kw)
        assert s.last_query_error() == (0, 0)
    n = c.q_off[-1]
    ref, rl, tol = c.reference(causal, scale)
    within(out[:n], ref[:n], tol[:n])
    assert (out[n:] == 3).all()
    if lse:
        assert (l[n:] == 7).all()
        none = torch.isinf(rl[:n])
        assert torch.equal(l[:n] == -math.inf, none)
        # the sum keeps the unrounded probabilities: scores' error plus logs'
        d = (l[:n].double() - rl[:n])[~none].abs()
        assert (d <= 2.0 ** -14 + 2.0 ** -18 * rl[:n][~none].abs()).all()
    return out


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G", [1, 4, 7])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("shared", [0, 37])
def test_attend_decode(pkg, D, G, head_major, shared):
    mem = [0, 1, 15, 16, 17, 127, 128, 129, 300, 555]
    check_attend(pkg, Paged(D * G, D, 2, G, 16, [1] * len(mem), mem, shared, head_major, extra_rows=2))


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shared", [0, 100])
@pytest.mark.parametrize("block", [16, 24])
def test_attend_ragged_queries(pkg, D, causal, shared, block):
    n = [3, 0, 17, 1, 64, 33, 0, 5]
    mem = [10, 20, 0, 300, 1, 129, 0, 63]
    check_attend(pkg, Paged(D + shared, D, 2, 4, block, n, mem, shared, extra_rows=3), causal)


@pytest.mark.parametrize("block", [1, 5, 16, 128])
@pytest.mark.parametrize("shared", [1, 127, 128, 513])
@pytest.mark.parametrize("n", [1, 70])
def test_attend_shared_edges(pkg, block, shared, n):
    """Prefixes that end inside a block, a tile, or on their borders."""
    check_attend(pkg, Paged(shared + block, 128, 1, 4, block, [n] * 3, [0, 1, 200], shared))


def test_attend_limits_below_the_prefix_and_empty_rows(pkg):
    """Requests that see less than the shared prefix, nothing at all, or whose
    first queries stand before every key; more cache than the causal limit."""
    kv = [0, 5, 40, 64, 90, 130, 1]
    n = [2, 3, 2, 1, 4, 3, 1]
    start = [0, 0, 38, 63, 10, 200, 0]
    for causal in (True, False):
        check_attend(pkg, Paged(5, 128, 2, 4, 16, n, [0] * 7, shared=64, kv=kv, start=start), causal)
        check_attend(pkg, Paged(6, 64, 2, 2, 16, n, [0] * 7, shared=0, kv=kv, start=start), causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,mem,H,G", [([1], [5000], 2, 4), ([1, 1], [3999, 20001], 1, 8), ([2], [9000], 1, 7),
                                       ([300], [1000], 1, 4), ([129, 1], [0, 2000], 2, 1)])
def test_attend_long(pkg, D, n, mem, H, G):
    check_attend(pkg, Paged(7, D, H, G, 16, n, mem, 0, qscale=2.0))


@pytest.mark.parametrize("requests,n", [(40, 1), (9, 31)])
def test_attend_long_shared_prefix(pkg, requests, n):
    mem = [(37 * r) % 211 for r in range(requests)]
    check_attend(pkg, Paged(8, 128, 2, 4, 16, [n] * requests, mem, shared=2050, qscale=2.0))


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("n,G", [(5, 4), (8, 4), (9, 7), (16, 4), (1, 40), (17, 4)])
def test_attend_a_few_tokens(pkg, D, n, G):
    """Units of 17 to 64 rows (and just past), with prefixes and splits."""
    check_attend(pkg, Paged(20 + n, D, 1, G, 16, [n, max(1, n - 3)], [5, 700], 90))
    check_attend(pkg, Paged(21 + n, D, 2, G, 32, [n], [1900], 0, head_major=True))


@pytest.mark.parametrize("D,block", [(256, 128), (32, 64), (64, 8), (128, 40)])
def test_attend_block_sizes(pkg, D, block):
    check_attend(pkg, Paged(30 + D, D, 3, 2, block, [1, 20, 3], [1, 300, 129], 0))


@pytest.mark.parametrize("D,G", [(128, 4), (64, 7), (128, 1)])
@pytest.mark.parametrize("shared,block", [(2048, 16), (1999, 16), (1030, 24), (1501, 1)])
def test_attend_prefix_in_a_grid_of_its_own(pkg, D, G, shared, block):
    """A prefix long enough, over enough requests, to be attended to once for
    all of them: requests that see less than the prefix, exactly it, one key
    more, nothing; one to a few queries; rows behind the last request."""
    R, H = 48, 4
    n = [1 + (r % 3 if G < 7 else 0) for r in range(R)]
    kv = [shared + n[r] + (37 * r) % 150 for r in range(R)]
    kv[3], kv[5], kv[7], kv[9], kv[11] = 0, 1, shared, shared + 1, shared // 2
    start = [max(0, k - m) for k, m in zip(kv, n)]
    start[9] = shared + 40
    # what decides, with the call's numbers
    assert shared * R * H * D * 4 >= 64 << 20 or D == 64
    for causal in (True, False):
        c = Paged(shared + G, D, H, G, block, n, [0] * R, shared=shared, kv=kv, start=start, extra_rows=3, qscale=1.5)
        check_attend(pkg, c, causal)


def test_prefix_grid_masked_values_and_bad_blocks(pkg):
    R, H, G, D, shared = 40, 4, 4, 128, 2000
    kv = [shared + 50 + r for r in range(R)]
    kv[2] = 700  # its queries see positions up to 699 of the prefix
    c = Paged(77, D, H, G, 16, [1] * R, [0] * R, shared=shared, kv=kv)
    with make(pkg, D, H) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        clean = c.call(s, cache)
        again = c.call(s, cache)
        assert torch.equal(clean, again)  # the same bits every time
        ref, _, tol = c.reference()
        within(clean, ref, tol)
        b, o = int(c.shared_blocks[750 // 16]), 750 % 16  # in a tile of request 2's, past its limit
        c.v[b, o, 1, 9] = math.nan
        c.k[b, o, 2, 3] = math.inf
        c.sync_cache()
        got = c.call(s, cache)
        within(got[2:3], ref[2:3], tol[2:3])
        assert not torch.isfinite(got[3, G:2 * G, 9]).any()
        c.v[b, o, 1, 9] = 0.5
        c.k[b, o, 2, 3] = 0.25
        c.sync_cache()
        good = c.call(s, cache)
        # a block of the prefix outside the cache: left out for all
        old = c.shared_blocks
        c.shared_blocks = old.clone()
        c.shared_blocks[10] = -3
        out = c.call(s, cache)
        assert s.last_query_error() == (pkg.IS_ERR_BAD_BLOCK, -1)
        keep = torch.tensor([j for j in range(kv[0]) if not 160 <= j < 176])
        table = torch.where(keep < shared, old[(keep // 16).clamp(max=len(old) - 1)], c.tables[0, keep // 16])
        K, V = c.k[table.long(), keep % 16].double(), c.v[table.long(), keep % 16].double()
        p = torch.softmax(torch.einsum("hgd,nhd->hgn", c.q[0].double().view(H, G, D), K) / math.sqrt(D), -1)
        want = torch.einsum("hgn,nhd->hgd", p, V).reshape(H * G, D)
        # summed key by key in fp32: the result's rounding alone is larger
        assert ((out[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12).all()
        # one of a request's own blocks: that request alone
        c.shared_blocks = old
        t = c.tables
        c.tables = t.clone()
        c.tables[5, 2010 // 16] = 10 ** 9
        out = c.call(s, cache)
        assert s.last_query_error() == (pkg.IS_ERR_BAD_BLOCK, 5)
        rest = [r for r in range(R) if r != 5]
        assert torch.equal(out[rest], good[rest]) and torch.isfinite(out[5]).all()


def test_prefix_grid_in_place_in_a_graph_and_on_two_streams(pkg):
    R, H, G, D, shared = 64, 2, 4, 128, 3000
    c = Paged(78, D, H, G, 16, [1] * R, [(11 * r) % 300 for r in range(R)], shared=shared)
    assert shared * R * H * D * 4 >= 64 << 20
    with make(pkg, D, H) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        ref, _, tol = c.reference()
        want = c.call(s, cache)
        within(want, ref, tol)
        q = c.q.clone()
        keep, c.q = c.q, q
        assert torch.equal(c.call(s, cache, out=q), want)
        c.q = keep
        meta = (c.i32(c.q_off), c.i32(c.start), c.i32(c.kv), c.tables.cuda(), cache, c.layer)
        kw = dict(max_q_len=1, shared_blocks=c.shared_blocks.cuda(), shared_len=shared)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        graphs, outs = [], []
        for st in streams:
            o = torch.zeros_like(want)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                s.attend(c.q, *meta, out=o, **kw)
            graphs.append(g), outs.append(o)
        for _ in range(5):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        eager = [s.attend(c.q, *meta, stream=st.cuda_stream, **kw) for st in streams for _ in range(3)]
        torch.cuda.synchronize()
        assert s.last_query_error() == (0, 0)
        for o in outs + eager:
            assert torch.equal(o, want)
        del graphs


@pytest.mark.parametrize("n", [1, 24, 80])
def test_offsets_past_32_bits(pkg, n):
    """Blocks 2^27 elements apart: element offsets past 2^32."""
    H, G, D, B, nb = 1, 4, 128, 16, 40
    stride = 1 << 27
    big = [torch.empty(stride * (nb - 1) + B * H * D, dtype=BF, device="cuda") for _ in range(2)]
    kc, vc = (x.as_strided((1, nb, B, H, D), (0, stride, H * D, D, 1)) for x in big)
    c = Paged(79, D, H, G, B, [n], [nb * B - n - 60], layers=1, layer=0, spare=0 if n > 1 else 3)
    blocks = c.k.shape[0]
    assert blocks <= nb
    kc[0, :blocks], vc[0, :blocks] = c.k, c.v
    c.k_cache, c.v_cache = kc, vc
    assert int(c.tables.max()) * stride > 2 ** 32
    check_attend(pkg, c)
    with make(pkg, D, H, layers=1) as s:
        k, v = (torch.randn(2, H, D, device="cuda").to(BF) for _ in range(2))
        slots = torch.tensor([(nb - 1) * B + 3, 36 * B], device="cuda")
        s.append(k, v, c.i32([0, 0]), slots, pkg.cache_desc(kc, vc))
        assert s.last_query_error() == (0, 0)
        assert torch.equal(vc[0, nb - 1, 3], v[0]) and torch.equal(kc[0, 36, 0], k[1])


def test_attend_uneven_splits(pkg):
    """A cluster's splits where some have no keys, next to a long request."""
    check_attend(pkg, Paged(80, 128, 2, 4, 16, [1, 1, 1], [0, 3000, 200]))
    check_attend(pkg, Paged(81, 256, 1, 4, 16, [1, 2], [1, 1500], kv=[0, 1501]))


def test_workspace_is_checked(pkg):
    from kv_cache_injection_gather_b200 import binding as B
    R, H, G, D, shared = 64, 2, 4, 128, 3000
    c = Paged(82, D, H, G, 16, [1] * R, [5] * R, shared=shared)
    with make(pkg, D, H) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        out = torch.zeros(R, H * G, D, dtype=BF, device="cuda")
        sb, tables = c.shared_blocks.cuda(), c.tables.cuda()
        ints = [c.i32(x) for x in (c.q_off, c.start, c.kv)]
        rows = lambda t: B.is_rows_t(t.data_ptr(), t.stride(0), t.stride(1), t.shape[1])  # noqa: E731
        args = B.is_attend_t(R, R, 1, tables.shape[1], *[t.data_ptr() for t in ints], tables.data_ptr(), sb.data_ptr(),
                             shared, 1, 0.0, c.layer, rows(c.q), rows(out), None)
        need = B.is_query_attend_workspace(s.query, args, cache)
        assert need >= R * H * G * (D * 4 + 8)
        work = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
        for ptr, size, rc in ((None, need, pkg.IS_ERR_INVALID_ARG), (work.data_ptr() + 16, need, pkg.IS_ERR_INVALID_ARG),
                              (work.data_ptr(), need - 1, pkg.IS_ERR_CAPACITY)):
            with pytest.raises(pkg.InjectError) as e:
                B.is_query_attend(s.query, args, cache, ptr, size, torch.cuda.current_stream().cuda_stream)
            assert e.value.status == rc
        B.is_query_attend(s.query, args, cache, work.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert torch.equal(out, c.call(s, cache))


def test_attend_many_requests(pkg):
    """More requests than one pass of the tile search covers, some empty."""
    n = [(7 * r) % 9 if r % 5 else 0 for r in range(700)]
    mem = [(13 * r) % 40 for r in range(700)]
    check_attend(pkg, Paged(9, 64, 1, 4, 16, n, mem, 0))


@pytest.mark.parametrize("n", [4, 130])
def test_masked_values_have_no_influence(pkg, n):
    """NaN and infinities in keys and values that a row does not see: slots
    past kv_len (all NaN already) and later positions of the same request.
    The rows that do not see them stay within the bounds of their own
    reference (they may be summed in another order)."""
    for bad in (math.nan, math.inf, -math.inf):
        c = Paged(10, 128, 2, 4, 16, [n], [100])
        check_attend(pkg, c)
        ref, _, tol = c.reference()
        last = c.kv[0] - 2  # seen by the last two queries alone
        b, o = int(c.tables[0, last // 16]), last % 16
        c.v[b, o, :, 3] = bad
        c.k[b, o, 1, 7] = bad
        c.sync_cache()
        with make(pkg, 128, 2) as s:
            got = c.call(s, pkg.cache_desc(c.k_cache, c.v_cache))
            assert s.last_query_error()[0] == 0
        within(got[: n - 2], ref[: n - 2], tol[: n - 2])
        assert not torch.isfinite(got[n - 2:, :, 3]).any()


def test_attend_large_scores_and_scale(pkg):
    """Scores in the thousands (a softmax with one winner), given scales."""
    c = Paged(11, 64, 2, 4, 16, [1, 5, 40], [200, 64, 10], qscale=30.0)
    check_attend(pkg, c, scale=1.5)
    check_attend(pkg, c, scale=1e-3)


def test_attend_default_bound_strides_and_in_place(pkg):
    c = Paged(12, 128, 2, 4, 16, [1, 6, 3], [50, 3, 170], shared=33)
    with make(pkg, 128, 2) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        want = c.call(s, cache)
        ref, _, tol = c.reference()
        loose = c.call(s, cache, max_q_len=None)  # bound: all tokens
        within(loose, ref, tol)
        q = c.q.clone()
        c.q = q
        assert torch.equal(c.call(s, cache, out=q), want)


@pytest.mark.parametrize("n", [1, 60])
def test_attend_bad_metadata_is_recorded_and_skipped(pkg, n):
    c = Paged(13, 64, 2, 4, 16, [n] * 4, [40, 50, 60, 70], shared=20)
    with make(pkg, 64, 2) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        clean = c.call(s, cache)

        def run(rc, detail, skipped, **change):
            old = {k: getattr(c, k) for k in change}
            for k, v in change.items():
                setattr(c, k, v)
            out = torch.full_like(clean, 4.0)
            kw = dict(out=out)
            kw["max_q_len"] = n
            c.call(s, cache, **kw)
            for k, v in old.items():
                setattr(c, k, v)
            assert s.last_query_error() == (rc, detail)
            for r in range(4):
                rows = slice(c.q_off[r], c.q_off[r + 1])
                if r in skipped:
                    assert (out[rows] == 4).all()
                elif r not in (detail,):
                    assert torch.equal(out[rows], clean[rows]), r
            return out

        at = lambda lst, i, v: lst[:i] + [v] + lst[i + 1:]  # noqa: E731
        run(pkg.IS_ERR_INVALID_ARG, 2, {2}, kv=at(c.kv, 2, -1))
        run(pkg.IS_ERR_INVALID_ARG, 1, {1}, start=at(c.start, 1, -4))
        run(pkg.IS_ERR_POSITION, 3, {3}, kv=at(c.kv, 3, c.width * 16 + 1))
        # a block outside the cache: its keys are left out
        for bad in (-1, c.k_cache.shape[1], 2 ** 31 - 1):
            t = c.tables.clone()
            t[1, 2] = bad  # positions 32 .. 47
            out = run(pkg.IS_ERR_BAD_BLOCK, 1, set(), tables=t)
            assert torch.isfinite(out).all()
        keep = [j for j in range(c.kv[1]) if not 32 <= j < 48]
        t0, t1 = c.q_off[1], c.q_off[2]
        blk = [int(c.shared_blocks[j // 16]) if j < c.shared else int(c.tables[1, j // 16]) for j in keep]
        K = c.k[blk, [j % 16 for j in keep]].double()
        V = c.v[blk, [j % 16 for j in keep]].double()
        for t in range(t0, t1):
            lim = c.start[1] + t - t0 + 1
            seen = torch.tensor([j < lim for j in keep], device="cuda")
            x = c.q[t].double().view(2, 4, 64)
            p = torch.softmax(torch.einsum("hgd,nhd->hgn", x, K[seen]) / 8, -1)
            want = torch.einsum("hgn,nhd->hgd", p, V[seen]).reshape(8, 64)
            # 2^-8 (|out| + sum p |v|), the latter below the largest |v|
            assert ((out[t].double() - want).abs() <= 2.0 ** -7 * V.abs().max()).all()
        bad = c.shared_blocks.clone()
        bad[0] = c.k_cache.shape[1]
        old, c.shared_blocks = c.shared_blocks, bad
        c.call(s, cache)
        c.shared_blocks = old
        assert s.last_query_error() == (pkg.IS_ERR_BAD_BLOCK, -1)
        assert torch.equal(c.call(s, cache), clean)


def test_attend_bad_offsets(pkg):
    c = Paged(14, 64, 1, 4, 16, [2, 2, 2], [9, 9, 9])
    with make(pkg, 64, 1) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        clean = c.call(s, cache)
        good = list(c.q_off)
        for off, detail in (([0, 2, 1, 6], 1), ([0, 2, 4, 7], 2), ([-1, 2, 4, 6], 0)):
            c.q_off = off
            out = torch.full_like(clean, 4.0)
            c.call(s, cache, out=out, max_q_len=2)
            c.q_off = good
            rc, d = s.last_query_error()
            assert (rc, d) == (pkg.IS_ERR_INVALID_ARG, detail)
        c.call(s, cache, max_q_len=1)  # a request has more than it says
        assert s.last_query_error() == (pkg.IS_ERR_INVALID_ARG, 0)


def test_attend_host_refusals(pkg):
    c = Paged(15, 64, 2, 2, 16, [1, 1], [9, 30])
    with make(pkg, 64, 2) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        E = pkg.InjectError
        for kw in (dict(max_q_len=0), dict(scale=math.inf)):
            with pytest.raises(E):
                c.call(s, cache, **kw)
        for kw in (dict(scale=0.0), dict(scale=-1.0), dict(shared_len=17, shared_blocks=c.i32([0])),
                   dict(out=torch.empty(2, 3, 64, dtype=BF, device="cuda")), dict(lse=torch.empty(2, 4).cuda().half()),
                   dict(out=torch.empty(2, 4, 64, device="cuda")), dict(out=torch.empty(2, 4, 64, dtype=BF))):
            with pytest.raises(ValueError):
                c.call(s, cache, **kw)
        c.layer = 2
        with pytest.raises(E):
            c.call(s, cache)
        c.layer = 1
        x = torch.empty(2, 3, 64, dtype=BF, device="cuda")
        c.q = x  # 3 query heads over 2 KV heads
        with pytest.raises(E):
            c.call(s, cache)
        odd = torch.empty(2, 4, 68, dtype=BF, device="cuda")[:, :, 1:65]  # neither aligned nor strides of 8
        c.q = odd
        with pytest.raises(E):
            c.call(s, cache)
        with pytest.raises(E):
            s.rotate(odd, c.i32([0, 1]))
        with pytest.raises(E):
            s.rotate(x, c.i32([0, 1]), eps=-1.0)
        with pytest.raises(ValueError):
            s.rotate(x, c.i32([0, 1]), k_weight=x[0, 0])
        with pytest.raises(ValueError):
            s.rotate(x, c.i32([0]))
        with pytest.raises(ValueError):
            s.rotate(x, torch.zeros(2, dtype=torch.int64, device="cuda"))
        with pytest.raises(E):
            s.append(x[:, :2], x[:, :2], c.i32([0, 1]), torch.zeros(2, dtype=torch.int64, device="cuda"), cache, 5)


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("n,mem,H,G,shared", [([1], [40001], 1, 4, 0), ([1, 3, 0, 1], [26000, 10, 7, 0], 1, 5, 37),
                                              ([2, 1], [17000, 33000], 2, 7, 0)])
def test_attend_keys_in_parts(pkg, D, n, mem, H, G, shared):
    """Few units of many keys: parts of the keys that a second grid joins, of
    which short requests leave most empty."""
    c = Paged(94, D, H, G, 16, n, mem, shared=shared, extra_rows=2)
    check_attend(pkg, c)
    c = Paged(95, D, H, G, 24, n, mem, shared=shared, head_major=True)
    check_attend(pkg, c, causal=False, scale=0.2)


def test_keys_in_parts_in_a_graph_with_bad_and_masked_blocks(pkg):
    H, G, D, B = 1, 4, 128, 16
    c = Paged(96, D, H, G, B, [2, 1], [30000, 20011])
    with make(pkg, D, H) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        clean = c.call(s, cache)
        assert s.last_query_error() == (0, 0)
        # the last key, which only the request's last query sees
        for x in (c.k_cache, c.v_cache):
            x[c.layer, int(c.tables[0, (c.kv[0] - 1) // B]), (c.kv[0] - 1) % B] = math.inf
        ref, _, tol = c.reference()
        within(c.call(s, cache)[:1], ref[:1], tol[:1])
        c.sync_cache()
        # a bad block's keys are left out
        t = c.tables
        c.tables = t.clone()
        c.tables[1, 900] = c.k_cache.shape[1]
        bad = c.call(s, cache)
        assert s.last_query_error() == (pkg.IS_ERR_BAD_BLOCK, 1)
        assert torch.equal(bad[:2], clean[:2]) and torch.isfinite(bad).all() and not torch.equal(bad, clean)
        c.tables = t
        # in place, captured and replayed
        q0 = c.q.clone()
        ints = [c.i32(x) for x in (c.q_off, c.start, c.kv)]
        tables = c.tables.cuda()
        run = lambda: s.attend(c.q, *ints, tables, cache, c.layer, max_q_len=2, out=c.q)  # noqa: E731
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(3):
            c.q.copy_(q0)
            graph.replay()
            assert torch.equal(c.q, clean)
        assert s.last_query_error() == (0, 0)


@pytest.mark.parametrize("n,R,shared", [(1, 3, 0), (70, 3, 0), (1, 64, 3000)])
def test_attend_scores_all_minus_infinity(pkg, n, R, shared):
    """Rows whose every score is -inf get zeros, as rows that see no key."""
    c = Paged(91, 128, 2, 4, 16, [n] * R, [300] * R, shared=shared)
    for x in (c.k, c.k_cache):
        x[~torch.isnan(x)] = 0
        x[..., 5] = -3e38
    c.q.zero_()
    c.q[:, ::2, 5] = 3e38  # even heads: 3e38 * -3e38; odd ones: 0, so the values' mean
    with make(pkg, 128, 2) as s:
        lse = torch.zeros(c.q.shape[:2], device="cuda")
        out = c.call(s, pkg.cache_desc(c.k_cache, c.v_cache), False, lse=lse)
        assert s.last_query_error() == (0, 0)
    assert (out[:, ::2] == 0).all() and (lse[:, ::2] == -math.inf).all()
    c.q.zero_()
    ref, rl, tol = c.reference(False)
    within(out[:, 1::2], ref[:, 1::2], tol[:, 1::2])
    assert torch.allclose(lse[:, 1::2].double(), rl[:, 1::2], atol=2.0 ** -14)


@pytest.mark.parametrize("n", [1, 60])
def test_attend_refuses_lengths_that_tiles_cannot_count(pkg, n):
    c = Paged(92, 64, 2, 4, 128, [n, n], [40, 50])
    with make(pkg, 64, 2) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        clean = c.call(s, cache)
        blocks = 2 ** 31 // 128
        tables = torch.zeros(2, blocks, dtype=torch.int32)
        tables[:, :c.width] = c.tables
        c.tables, c.kv = tables, [2 ** 31 - 128, c.kv[1]]
        out = torch.full_like(clean, 4.0)
        c.call(s, cache, out=out)
        assert s.last_query_error() == (pkg.IS_ERR_POSITION, 0)
        assert (out[:n] == 4).all() and torch.equal(out[n:], clean[n:])
        with pytest.raises(pkg.InjectError) as e:
            c.call(s, cache, shared_len=2 ** 31 - 128, shared_blocks=tables[0].cuda())
        assert e.value.status == pkg.IS_ERR_CAPACITY


def test_written_rows_of_stride_zero_are_refused(pkg):
    c = Paged(93, 64, 2, 2, 16, [1, 1], [9, 30])
    with make(pkg, 64, 2) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        pos, slots = c.i32([0, 1]), torch.tensor([-1, -1], device="cuda")
        one = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
        for bad in (one[:1].expand(2, 4, 64), one[:, :1].expand(2, 4, 64)):
            for call in (lambda: c.call(s, cache, out=bad), lambda: s.rotate(one, pos, q_out=bad),
                         lambda: s.rotate(one, pos, k=one, k_out=bad),
                         lambda: s.append(one[:, :2], one[:, :2], pos, slots, cache, q=one, q_out=bad)):
                with pytest.raises(pkg.InjectError) as e:
                    call()
                assert e.value.status == pkg.IS_ERR_INVALID_ARG
            # as inputs they repeat
            a, b = s.rotate(bad, pos)[0], s.rotate(bad.contiguous(), pos)[0]
            assert torch.equal(a, b)


# ---------------------------------------------------------------- together

def test_a_serving_step_and_its_graph(pkg):
    """inject -> append (queries rotated) -> attend, as an engine runs it for
    query tokens after a shared prefix; then the same step captured into a
    graph and replayed with other inputs, next to a second graph of the same
    handle on another stream."""
    L, H, G, D, B, P, R = 2, 2, 4, 128, 16, 40, 3
    Hq, nb = H * G, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(BF)  # noqa: E731
    facts = [rnd(L, H, n, D) for n in (20, 33, 7)]
    values = [rnd(L, H, n, D) for n in (20, 33, 7)]
    lens = [20 + 33, 7, 33 + 20 + 7]
    ids, ro = [0, 1, 2, 1, 0, 2], [0, 2, 3, 6]
    n = [4, 1, 9]
    f = inv_freq(D, 1e4)
    with make(pkg, D, H, layers=L) as s:
        for a, b in zip(facts, values):
            s.put_fact(a, b)
        kc, vc = (torch.full((L, nb, B, H, D), math.nan, dtype=BF, device="cuda") for _ in range(2))
        cache = pkg.cache_desc(kc, vc)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        perm = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        shared = perm[:3]  # positions 0 .. 39: two whole blocks and half a third
        tables = perm[3:3 + R * 8].view(R, 8).contiguous().cuda()
        prefix_k, prefix_v = rnd(P, H, D), rnd(P, H, D)
        pj = torch.arange(P)
        pslots = (shared[pj // B].long() * B + pj % B).cuda()
        for layer in range(L):
            s.append(prefix_k, prefix_v, i32(list(range(P))), pslots, cache, layer)
        s.inject(i32(ro), i32(ids), i32([P] * R), tables, cache)
        assert s.last_error()[0] == 0
        start = [P + x for x in lens]
        kv = [a + b for a, b in zip(start, n)]
        q_off = [0, 4, 5, 14]
        T = q_off[-1]
        pos = [start[r] + i for r in range(R) for i in range(n[r])]
        slots = torch.tensor([int(tables[r, (start[r] + i) // B]) * B + (start[r] + i) % B
                              for r in range(R) for i in range(n[r])], device="cuda")
        meta = (i32(q_off), i32(start), i32(kv), tables)
        positions, sh = i32(pos), shared.contiguous().cuda()

        def step(q, k, v, layer, out):
            qr = s.append(k, v, positions, slots, cache, layer, q=q)
            return s.attend(qr, *meta, cache, layer, max_q_len=9, shared_blocks=sh, shared_len=P, out=out)

        def want(q, k, v, layer):
            """From the definitions: prefix, facts and query tokens rotated
            to their positions, rounded to bf16 as the cache holds them."""
            out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
            tol = torch.zeros_like(out)
            for r in range(R):
                ks = [prefix_k] + [facts[i][layer].transpose(0, 1) for i in ids[ro[r]:ro[r + 1]]]
                vs = [prefix_v] + [values[i][layer].transpose(0, 1) for i in ids[ro[r]:ro[r + 1]]]
                rows = slice(q_off[r], q_off[r + 1])
                K, V = torch.cat(ks + [k[rows]]), torch.cat(vs + [v[rows]])
                m = len(K)
                assert m == kv[r]
                K = rotated(K, None, 0, torch.arange(m, device="cuda"), f, False)[0].to(BF)
                Q = rotated(q[rows], None, 0, torch.arange(start[r], m, device="cuda"), f, False)[0].to(BF)
                o, _, t = attend_reference(Q, [0, n[r]], [start[r]], [m], torch.arange(m).view(1, m), K[:, None],
                                           V[:, None], 1, None, 0, True, D ** -0.5)
                # q and k are rounded on both sides, now and then to different
                # neighbours (an fp32 rotation next to a midpoint, about one
                # element in 2^14): a step of 2^-7 in one of a row's D terms
                # moves its scores by 2^-7 |q_d k_d| scale < 2^-7 * 16 * 0.09
                # = 2^-6.5, so the result by at most 2^-5.5 A, and A <= 2^8 t
                out[rows], tol[rows] = o, t * (1 + 2.0 ** 2.5)
            return out, tol

        out = torch.empty(T, Hq, D, dtype=BF, device="cuda")
        q, k, v = rnd(T, Hq, D), rnd(T, H, D), rnd(T, H, D)
        for layer in range(L):
            step(q, k, v, layer, out)
            assert s.last_query_error() == (0, 0)
            ref, tol = want(q, k, v, layer)
            within(out, ref, tol)
        # two graphs, one per layer, replayed at the same time on two streams
        graphs, outs = [], []
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for layer in range(L):
            o = torch.zeros_like(out)
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=streams[layer]):
                step(q, k, v, layer, o)
            graphs.append(gr)
            outs.append(o)
        q.copy_(rnd(T, Hq, D)), k.copy_(rnd(T, H, D)), v.copy_(rnd(T, H, D))
        torch.cuda.synchronize()
        for _ in range(3):
            for layer in range(L):
                with torch.cuda.stream(streams[layer]):
                    graphs[layer].replay()
        torch.cuda.synchronize()
        assert s.last_query_error() == (0, 0)
        for layer in range(L):
            ref, tol = want(q, k, v, layer)
            within(outs[layer], ref, tol)
            fresh = step(q, k, v, layer, torch.empty_like(out))
            assert torch.equal(fresh, outs[layer])  # same inputs, same bits
        del graphs


def test_another_stream(pkg):
    """The stream argument: work and its outputs on a stream that is not the
    current one."""
    c = Paged(16, 128, 2, 4, 16, [1] * 5, [300, 20, 700, 1, 90], shared=600)
    with make(pkg, 128, 2) as s:
        cache = pkg.cache_desc(c.k_cache, c.v_cache)
        want = c.call(s, cache)
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        got = [c.call(s, cache, stream=st.cuda_stream) for _ in range(4)]
        st.synchronize()
        assert all(torch.equal(want, x) for x in got)
        assert s.last_query_error(st.cuda_stream) == (0, 0)
