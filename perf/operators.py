"""The query-side operators of a serving step, as cases to time and check.

After the retrieved facts are injected into a request's paged KV cache, the
model runs over the query tokens only.  Per layer that takes three operators:

  rotate   per-head RMS norm (optional) and the RoPE rotation of queries and
           keys, in one pass over both
  append   keys (normed, rotated) and values of new tokens written to their
           slots of the paged cache, the queries rotated on the way
  attend   attention of the query tokens over the paged cache, where the first
           shared_len positions of every request lie in the same blocks

With ``own`` false ``run`` computes them in elementary torch operations (fp32,
angles in fp64, one rounding at the end); with ``own`` true it calls this
package.  ``exact`` computes them in fp64.  Lengths follow from the case alone,
values and block tables from the seed.
"""
import math

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token of one request: latency
        dict(name="rotate 1 token", op="rotate", tokens=1, pad=0, q_heads=32, kv_heads=8, dim=128, interleaved=False,
             norm=True, llama3=True, far=4096),
        # a padded batch of query tokens, head_dim 64, adjacent pairs
        dict(name="rotate 333 tokens, pairs", op="rotate", tokens=333, pad=11, q_heads=14, kv_heads=2, dim=64,
             interleaved=True, norm=True, llama3=False, far=131072),
        # a long prompt at Llama-3.1-8B heads
        dict(name="rotate 16384 tokens", op="rotate", tokens=16384, pad=0, q_heads=32, kv_heads=8, dim=128,
             interleaved=False, norm=True, llama3=True, far=16384),
        # 100 concurrent requests decode one token each
        dict(name="append 100 tokens", op="append", tokens=100, pad=0, q_heads=32, kv_heads=8, dim=128,
             interleaved=False, norm=False, llama3=True, far=8192, block=16, head_major=False, with_q=True),
        # query tokens at Qwen2.5-7B heads, odd count, head-major cache, key norm
        dict(name="append 5001 tokens, head-major", op="append", tokens=5001, pad=13, q_heads=28, kv_heads=4, dim=128,
             interleaved=False, norm=True, llama3=False, far=65536, block=32, head_major=True, with_q=True),
        # a long prompt's keys and values
        dict(name="append 16384 tokens", op="append", tokens=16384, pad=0, q_heads=32, kv_heads=8, dim=128,
             interleaved=False, norm=False, llama3=True, far=32768, block=16, head_major=False, with_q=True),
        # one request decodes after its injected memory (about 50 facts)
        dict(name="attend decode, 1 request", op="attend", requests=1, q_min=1, q_max=1, kv_min=2113, kv_max=2113,
             shared=0, q_heads=32, kv_heads=8, dim=128, block=16, head_major=False, causal=True),
        # 100 concurrent requests decode: shared system prompt, own memories
        dict(name="attend decode, 100 requests, shared 4096", op="attend", requests=100, q_min=1, q_max=1, kv_min=800,
             kv_max=3200, shared=4096, q_heads=32, kv_heads=8, dim=128, block=16, head_major=False, causal=True),
        # a few requests with very long contexts decode
        dict(name="attend decode, 3 long requests", op="attend", requests=3, q_min=1, q_max=1, kv_min=60001,
             kv_max=131071, shared=0, q_heads=28, kv_heads=4, dim=128, block=16, head_major=False, causal=True),
        # a few speculated tokens each, head_dim 64, a prefix that ends inside a block of 24
        dict(name="attend 2-5 tokens, dim 64", op="attend", requests=16, q_min=2, q_max=5, kv_min=33, kv_max=1500,
             shared=1001, q_heads=14, kv_heads=2, dim=64, block=24, head_major=True, causal=True),
        # the query-only prefill of 100 requests after injection
        dict(name="attend 100 queries, shared 2048", op="attend", requests=100, q_min=16, q_max=64, kv_min=1200,
             kv_max=2900, shared=2048, q_heads=32, kv_heads=8, dim=128, block=16, head_major=False, causal=True),
        # ordinary prompts without a cached prefix
        dict(name="attend prompts of 4096", op="attend", requests=2, q_min=4000, q_max=4096, kv_min=0, kv_max=0,
             shared=0, q_heads=32, kv_heads=8, dim=128, block=16, head_major=False, causal=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend"])
    kv_heads, group = rng.choice([(8, 4), (4, 7), (2, 7), (2, 4), (1, 8), (4, 1)])
    dim = rng.choice([64, 128, 128])
    c = dict(op=op, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    if op != "attend":
        tokens = _log(rng, 1, 16384)
        c.update(tokens=tokens, pad=rng.randrange(0, 9) if tokens > 16 else 0, interleaved=rng.random() < 0.3,
                 norm=rng.random() < 0.5, llama3=rng.random() < 0.5, far=_log(rng, max(64, tokens), 131072))
        if op == "append":
            c.update(block=rng.choice([8, 16, 16, 24, 32, 64]), head_major=rng.random() < 0.4,
                     with_q=rng.random() < 0.7)
        return c
    requests = _log(rng, 1, 128)
    if rng.random() < 0.5:
        q_min = q_max = 1
    else:
        q_max = _log(rng, 2, max(2, min(4096, 6400 // requests)))
        q_min = rng.randint(1, q_max)
    # the plain form holds requests x q_max x q_heads x positions scores in
    # fp32, and the keys of every request: keep both below the largest cases
    room = min(130_000, int(5.0e8 / (requests * q_max * c["q_heads"])) - q_max,
               int(2.0e8 / (requests * kv_heads * dim)) - q_max)
    total = _log(rng, 2, max(2, room))
    shared = rng.choice([0, 1]) * rng.randint(0, total * 3 // 4)
    kv_max = max(1, total - shared)
    c.update(requests=requests, q_min=q_min, q_max=q_max, kv_min=rng.randint(0, kv_max), kv_max=kv_max, shared=shared,
             block=rng.choice([8, 16, 16, 24, 32, 64]), head_major=rng.random() < 0.4, causal=rng.random() < 0.85)
    return c


# ---------------------------------------------------------------- lengths

def _spread(lo, hi, n, shift):
    """n whole numbers over [lo, hi], evenly spread and shuffled."""
    return [lo + int((hi - lo + 1) * (((i + 1) * 0.6180339887498949 + shift) % 1.0)) for i in range(n)]


def _lengths(case):
    """Per request: query tokens, and cached tokens (shared ones, own ones,
    the query's)."""
    n = _spread(case["q_min"], case["q_max"], case["requests"], 0.0)
    mem = _spread(case["kv_min"], case["kv_max"], case["requests"], 0.37)
    return n, [case["shared"] + m + q for m, q in zip(mem, n)]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    return g


def _normal(g, *shape, scale=1.0):
    x = torch.empty(shape, dtype=BF16, device="cuda").normal_(generator=g)
    return x if scale == 1.0 else x.mul_(scale)


def _rope(case):
    return dict(theta=5e5 if case.get("llama3") else 1e6,
                llama3=dict(factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0,
                            original_max_position=8192) if case.get("llama3") else None)


def _handle(case, layers):
    """The store that a user's program holds: RoPE configuration, KV heads."""
    import kv_cache_injection_gather_b200 as pkg
    r = _rope(case)
    style = pkg.IS_ROPE_INTERLEAVED if case.get("interleaved") else pkg.IS_ROPE_ROTATE_HALF
    return pkg.FactStore(layers, case["kv_heads"], case["dim"],
                         pkg.RopeConfig(theta=r["theta"], style=style, llama3=r["llama3"]), capacity_tokens=64,
                         max_facts=1, max_batch_requests=256, max_batch_fact_ids=256, max_batch_blocks=4096)


def _cache(g, case, blocks, layers=2):
    H, D, B = case["kv_heads"], case["dim"], case["block"]
    shape = (layers, blocks, H, B, D) if case["head_major"] else (layers, blocks, B, H, D)
    return _normal(g, *shape), _normal(g, *shape)


def prepare(case, seed):
    g = _gen(seed)
    D, Hq, H = case["dim"], case["q_heads"], case["kv_heads"]
    s = dict(case)
    if case["op"] in ("rotate", "append"):
        T = case["tokens"] + case["pad"]
        s["live"] = case["tokens"]
        # one projection's output: the heads are slices of its rows
        qkv = _normal(g, T, (Hq + 2 * H) * D)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + H) * D].view(T, H, D)
        s["v"] = qkv[:, (Hq + H) * D:].view(T, H, D)
        s["q_weight"] = (1 + _normal(g, D, scale=0.2)) if case["norm"] else None
        s["k_weight"] = (1 + _normal(g, D, scale=0.2)) if case["norm"] else None
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["positions"][case["tokens"]:] = -1
        s["q_out"] = torch.zeros((T, Hq, D), dtype=BF16, device="cuda")
        s["k_out"] = torch.zeros((T, H, D), dtype=BF16, device="cuda")
        half = torch.arange(D // 2, dtype=torch.float64)
        f = _rope(case)["theta"] ** (-2.0 * half / D)
        if case["llama3"]:  # wavelengths past 8192 / 1 slowed 8 times, below 8192 / 4 kept, blended between
            turns = 8192 * f / (2 * math.pi)
            w = ((turns - 1) / 3).clamp(0, 1)
            f = f * (w + (1 - w) / 8)
        s["freq"] = f.cuda()
        if case["op"] == "append":
            B = case["block"]
            blocks = -(-case["tokens"] * 5 // (4 * B)) + 2
            s["k_cache"], s["v_cache"] = _cache(g, case, blocks)
            s["slots"] = torch.full((T,), -1, dtype=torch.int64, device="cuda")
            s["slots"][:case["tokens"]] = torch.randperm(blocks * B, generator=g, device="cuda")[:case["tokens"]]
    else:
        B, R, shared = case["block"], case["requests"], case["shared"]
        n, kv = _lengths(case)
        T, width = sum(n), -(-max(kv) // B)
        shared_blocks, first = -(-shared // B), shared // B
        blocks = shared_blocks + sum(-(-k // B) - first for k in kv) + 3
        ids = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        s["k_cache"], s["v_cache"] = _cache(g, case, blocks)
        s["q"] = _normal(g, T, Hq, D, scale=2.0)
        s["shared_blocks"] = ids[:shared_blocks].contiguous() if shared else None
        col = torch.arange(width, device="cuda")
        used = torch.tensor([-(-k // B) - first for k in kv], device="cuda")
        base = shared_blocks + torch.cumsum(used, 0) - used
        at = base[:, None] + col[None, :] - first
        live = (col[None, :] >= first) & (col[None, :] - first < used[:, None])
        s["block_tables"] = torch.where(live, ids[at.clamp(0, blocks - 1)], 0).to(torch.int32).contiguous()
        i32 = dict(dtype=torch.int32, device="cuda")
        s["q_offsets"] = torch.tensor([sum(n[:i]) for i in range(R + 1)], **i32)
        s["start_pos"] = torch.tensor([k - m for k, m in zip(kv, n)], **i32)
        s["kv_lens"] = torch.tensor(kv, **i32)
        s["q_width"], s["kv_width"] = max(n), max(kv)
        s["out"] = torch.zeros((T, Hq, D), dtype=BF16, device="cuda")
    if own:
        s["store"] = _handle(case, 2)
        if "k_cache" in s:
            import kv_cache_injection_gather_b200 as pkg
            s["cache"] = pkg.cache_desc(s["k_cache"], s["v_cache"], head_major=case["head_major"])
    return s


LAYER = 1  # the layer of the cache that the cases use


# ---------------------------------------------------------------- plain forms

def _norm_rotate(x, weight, positions, freq, interleaved):
    """[T][heads][D] bf16 -> normed (where there is a weight), rotated, bf16."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = positions.double()[:, None] * freq[None, :]
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x.chunk(2, -1)
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return y.to(BF16)


def _plain_rotate(s):
    n, pos = s["live"], s["positions"][:s["live"]]
    s["q_out"][:n] = _norm_rotate(s["q"][:n], s["q_weight"], pos, s["freq"], s["interleaved"])
    s["k_out"][:n] = _norm_rotate(s["k"][:n], s["k_weight"], pos, s["freq"], s["interleaved"])
    return s["q_out"], s["k_out"]


def _plain_append(s):
    n, pos = s["live"], s["positions"][:s["live"]]
    slots = s["slots"][:n]
    b, o = slots // s["block"], slots % s["block"]
    k = _norm_rotate(s["k"][:n], s["k_weight"], pos, s["freq"], s["interleaved"])
    if s["head_major"]:
        s["k_cache"][LAYER][b, :, o] = k
        s["v_cache"][LAYER][b, :, o] = s["v"][:n]
    else:
        s["k_cache"][LAYER][b, o] = k
        s["v_cache"][LAYER][b, o] = s["v"][:n]
    out = dict(k_cache=s["k_cache"][LAYER], v_cache=s["v_cache"][LAYER])
    if s["with_q"]:
        s["q_out"][:n] = _norm_rotate(s["q"][:n], s["q_weight"], pos, s["freq"], s["interleaved"])
        out["q"] = s["q_out"]
    return out


def _plain_attend(s):
    R, N, W, B, shared = s["requests"], s["q_width"], s["kv_width"], s["block"], s["shared"]
    Hq, H, D = s["q_heads"], s["kv_heads"], s["dim"]
    G, T = Hq // H, s["q"].shape[0]
    p = torch.arange(W, device="cuda")
    block = s["block_tables"][:, p // B].long()  # [R][W]
    if shared:
        head = s["shared_blocks"][(p // B).clamp(max=s["shared_blocks"].numel() - 1)].long()
        block = torch.where(p < shared, head, block)
    here = p[None, :] < s["kv_lens"][:, None]
    block = torch.where(here, block, 0)
    o = (p % B).expand(R, W)
    if s["head_major"]:
        k, v = s["k_cache"][LAYER][block, :, o], s["v_cache"][LAYER][block, :, o]
    else:
        k, v = s["k_cache"][LAYER][block, o], s["v_cache"][LAYER][block, o]
    k, v = k.float().permute(0, 2, 3, 1), v.float().permute(0, 2, 1, 3)  # [R][H][D][W], [R][H][W][D]
    i = torch.arange(N, device="cuda")
    row = (s["q_offsets"][:-1, None] + i).clamp(max=T - 1).long()
    q = s["q"][row].float().view(R, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, N * G, D)
    x = (q @ k).mul_(1.0 / math.sqrt(D)).view(R, H, N, G, W)
    seen = here[:, None, :]
    if s["causal"]:
        seen = seen & (p <= (s["start_pos"][:, None] + i)[:, :, None])
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True).view(R, H, N * G, 1)
    y = (x.view(R, H, N * G, W) @ v) / total.clamp(min=1e-30)
    y = y.view(R, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(R, N, Hq, D)
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    r = torch.searchsorted(s["q_offsets"][1:].contiguous(), t, right=True)
    return y[r, (t - s["q_offsets"][r]).long()].to(BF16)


# ---------------------------------------------------------------- one pass

def run(s):
    if not own:
        return {"rotate": _plain_rotate, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)
    store = s["store"]
    if s["op"] == "rotate":
        return store.rotate(s["q"], s["positions"], k=s["k"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                            q_out=s["q_out"], k_out=s["k_out"])
    if s["op"] == "append":
        q = store.append(s["k"], s["v"], s["positions"], s["slots"], s["cache"], LAYER, k_weight=s["k_weight"],
                         q=s["q"] if s["with_q"] else None, q_weight=s["q_weight"] if s["with_q"] else None,
                         q_out=s["q_out"] if s["with_q"] else None)
        out = dict(k_cache=s["k_cache"][LAYER], v_cache=s["v_cache"][LAYER])
        if s["with_q"]:
            out["q"] = q
        return out
    return store.attend(s["q"], s["q_offsets"], s["start_pos"], s["kv_lens"], s["block_tables"], s["cache"], LAYER,
                        max_q_len=s["q_width"], shared_blocks=s["shared_blocks"], shared_len=s["shared"],
                        causal=s["causal"], out=s["out"])


# ---------------------------------------------------------------- what a pass needs

def work(case):
    D, Hq, H = case["dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "rotate":
        rows = case["tokens"] * (Hq + H)
        return dict(bytes=rows * D * 4 + case["tokens"] * 4, flops=rows * D * (7 if case["norm"] else 3))
    if case["op"] == "append":
        heads = H + (Hq if case["with_q"] else 0)
        return dict(bytes=case["tokens"] * ((heads + H) * D * 4 + 12),
                    flops=case["tokens"] * heads * D * (7 if case["norm"] else 3))
    n, kv = _lengths(case)
    pairs = sum(m * k - (m * (m - 1) // 2 if case["causal"] else 0) for m, k in zip(n, kv))
    tokens = case["shared"] + sum(k - case["shared"] for k in kv)
    return dict(bytes=tokens * H * D * 4 + sum(n) * Hq * D * 4, flops=4.0 * pairs * Hq * D)


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_rows(x, weight, positions, case):
    D = case["dim"]
    z = x.double()
    if weight is not None:
        z = weight.double() * z / (z.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt()
    rope = _rope(case)
    freq = []
    for i in range(D // 2):
        f = math.exp(-2.0 * i / D * math.log(rope["theta"]))
        if rope["llama3"]:
            a, wave = rope["llama3"], 2 * math.pi / f
            long, short = a["original_max_position"] / a["low_freq_factor"], a["original_max_position"] / a["high_freq_factor"]
            if wave > long:
                f /= a["factor"]
            elif wave >= short:
                t = (a["original_max_position"] / wave - a["low_freq_factor"]) / (a["high_freq_factor"] - a["low_freq_factor"])
                f = t * f + (1 - t) * f / a["factor"]
        freq.append(f)
    turn = torch.outer(positions.double(), torch.tensor(freq, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.ones_like(turn), turn)[:, None, :]
    if case["interleaved"]:
        return torch.view_as_real(torch.view_as_complex(z.unflatten(-1, (D // 2, 2)).contiguous()) * turn).flatten(-2)
    w = torch.complex(z[..., :D // 2].contiguous(), z[..., D // 2:].contiguous()) * turn
    return torch.cat([w.real, w.imag], -1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] in ("rotate", "append"):
        n = s["live"]
        pos = s["positions"][:n]
        q, k = s["q_out"].double(), s["k_out"].double()
        q[:n] = _exact_rows(s["q"][:n], s["q_weight"], pos, case)
        k[:n] = _exact_rows(s["k"][:n], s["k_weight"], pos, case)
        if case["op"] == "rotate":
            return q, k
        kc, vc = s["k_cache"][LAYER].double(), s["v_cache"][LAYER].double()
        for cache, rows in ((kc, k[:n]), (vc, s["v"][:n].double())):
            flat = cache.transpose(1, 2) if case["head_major"] else cache  # [blocks][B][H][D]
            flat[s["slots"][:n].div(case["block"], rounding_mode="floor"), s["slots"][:n].remainder(case["block"])] = rows
        out = dict(k_cache=kc, v_cache=vc)
        if case["with_q"]:
            out["q"] = q
        return out
    B, H, D, shared = case["block"], case["kv_heads"], case["dim"], case["shared"]
    G = case["q_heads"] // H
    kc, vc = s["k_cache"][LAYER], s["v_cache"][LAYER]
    if case["head_major"]:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    kc, vc = kc.reshape(-1, H, D), vc.reshape(-1, H, D)
    n, kv = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for r in range(case["requests"]):
        p = torch.arange(kv[r], device="cuda")
        slot = s["block_tables"][r].long()[p // B] * B + p % B
        if shared:
            slot[:shared] = s["shared_blocks"].long()[p[:shared] // B] * B + p[:shared] % B
        mine = slice(first, first + n[r])
        first += n[r]
        hidden = None
        if case["causal"]:
            hidden = p[None, :] > (kv[r] - n[r] + torch.arange(n[r], device="cuda"))[:, None]
        for h in range(H):
            kh, vh = kc[slot, h].double(), vc[slot, h].double()
            qh = s["q"][mine, h * G:(h + 1) * G].double()  # [n][G][D]
            x = torch.einsum("ngd,pd->ngp", qh, kh) / math.sqrt(D)
            if hidden is not None:
                x = x.masked_fill(hidden[:, None, :], -math.inf)
            out[mine, h * G:(h + 1) * G] = torch.einsum("ngp,pd->ngd", torch.softmax(x, -1), vh)
    return out
