"""Inputs and fp64 references of the query-side operators (rotate, append,
attend), shared by the GPU tests.  The references are written from the
definitions in include/inject_query.h, loop over requests, and use none of the
package's code; everything here runs on whatever device the tensors are on."""
from __future__ import annotations

import math

import torch

BF = torch.bfloat16


def inv_freq(D, theta, llama3=None):
    """fp64 RoPE frequencies; llama3 = (factor, low, high, original context)."""
    out = []
    for i in range(D // 2):
        f = theta ** (-2.0 * i / D)
        if llama3:
            factor, low, high, ctx = llama3
            wave = 2 * math.pi / f
            if wave > ctx / low:
                f /= factor
            elif wave >= ctx / high:
                w = (ctx / wave - low) / (high - low)
                f = (1 - w) * f / factor + w * f
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotated(x, weight, eps, positions, freq, interleaved):
    """fp64 norm and rotation of bf16 [T][heads][D], and the magnitude
    |a| + |b| of each output's input pair after the norm."""
    z = x.double()
    if weight is not None:
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * weight.double()
    ang = positions.double()[:, None] * freq.to(x.device)[None, :]
    c, s = torch.cos(ang)[:, None, :], torch.sin(ang)[:, None, :]
    if interleaved:
        a, b = z[..., 0::2], z[..., 1::2]
    else:
        a, b = z[..., : z.shape[-1] // 2], z[..., z.shape[-1] // 2:]
    ya, yb, m = a * c - b * s, b * c + a * s, a.abs() + b.abs()
    if interleaved:
        return torch.stack([ya, yb], -1).flatten(-2), torch.stack([m, m], -1).flatten(-2)
    return torch.cat([ya, yb], -1), torch.cat([m, m], -1)


def rotate_tolerance(ref, mag):
    """One bf16 rounding (half a step: 2^-8 of the value) of an fp32 result.
    The fp32 part, in units of 2^-24 of |a| + |b|: cos and sin 2 each, product
    and sum 2, the norm's factor at most 8 (mean of D squares in a tree of
    depth <= 16 + 5, halved by the root; rsqrt 2; two products): below
    2^-24 * 16 = 2^-20."""
    return 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag


def attend_reference(q, q_off, start, kv, tables, k_cache, v_cache, block, shared_blocks, shared_len, causal, scale):
    """fp64 attention, request by request.  k_cache and v_cache are one
    layer's [blocks][B][H][D] (bf16).  Returns (out, lse, tol) with tol the
    bound on |kernel - out|, elementwise:

      * the result's own rounding: 2^-8 |out|;
      * the probabilities rounded to bf16 before the product with v: each is
        off by at most 2^-8 of itself, together 2^-8 A with A = sum p |v|;
      * a score s summed in fp32 over D products in any order: off by at most
        (D + 2) 2^-24 S with S = scale sum |q k|, and exp2's argument and
        result by about 2^-22 (|s| + 2): each p is off by a factor
        exp(2 c), c = 2^-24 (D + 2) max S + 2^-22 (max |s| + 2), in numerator
        and denominator: 4 c A;
      * where a share of the exponentials is a polynomial within 2^-18 of them:
        2^-17 A, in numerator and denominator;
      * sums over n keys in fp32, in any order: 2 n 2^-24 A.
    """
    T, Hq, D = q.shape
    H = k_cache.shape[2]
    G = Hq // H
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for r in range(len(kv)):
        t0, t1, n = q_off[r], q_off[r + 1], kv[r]
        if n == 0 or t0 == t1:
            continue
        j = torch.arange(n)
        blk = tables[r].cpu()[(j // block).clamp(max=tables.shape[1] - 1)].long()
        if shared_len:
            sb = shared_blocks.cpu()
            blk = torch.where(j < shared_len, sb[(j // block).clamp(max=len(sb) - 1)].long(), blk)
        blk, off = blk.to(q.device), (j % block).to(q.device)
        K, V = k_cache[blk, off].double(), v_cache[blk, off].double()  # [n][H][D]
        jj = j.to(q.device)
        for t in range(t0, t1):
            lim = min(n, start[r] + t - t0 + 1) if causal else n
            if lim <= 0:
                continue
            x = q[t].double().view(H, G, D)
            s = torch.einsum("hgd,nhd->hgn", x, K[:lim]) * scale
            p = torch.softmax(s, -1)
            S = (torch.einsum("hgd,nhd->hgn", x.abs(), K[:lim].abs()) * scale).amax(-1)
            c = 2.0 ** -24 * (D + 2) * S + 2.0 ** -22 * (s.abs().amax(-1) + 2)
            o = torch.einsum("hgn,nhd->hgd", p, V[:lim])
            A = torch.einsum("hgn,nhd->hgd", p, V[:lim].abs())
            out[t] = o.reshape(Hq, D)
            tol[t] = (2.0 ** -8 * (o.abs() + A) + A * (4 * c[..., None] + 2.0 ** -17 + 2 * lim * 2.0 ** -24)).reshape(Hq, D)
            lse[t] = torch.logsumexp(s, -1).reshape(Hq)
        del jj
    return out, lse, tol


class Paged:
    """A paged cache with random values at the positions in use and NaN
    everywhere else, block tables, and the metadata of an attention call."""

    def __init__(self, seed, D, H, G, block, n, mem, shared=0, head_major=False, layers=2, layer=1, device="cuda",
                 qscale=1.0, kv=None, start=None, extra_rows=0, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.D, self.H, self.G, self.block, self.shared = D, H, G, block, shared
        self.n = list(n)
        self.kv = list(kv) if kv is not None else [shared + m + k for m, k in zip(mem, n)]
        self.start = list(start) if start is not None else [max(0, k - m) for k, m in zip(self.kv, n)]
        self.q_off = [sum(self.n[:i]) for i in range(len(self.n) + 1)]
        self.layer = layer
        T = self.q_off[-1] + extra_rows
        sb, first = -(-shared // block), shared // block
        own = [max(0, -(-k // block) - first) for k in self.kv]
        nb = sb + sum(own) + spare
        ids = torch.randperm(nb, generator=g).to(torch.int32)
        self.shared_blocks = ids[:sb].contiguous()
        self.width = max([-(-k // block) for k in self.kv] + [1])
        tables = torch.full((len(n), self.width), -7, dtype=torch.int32)  # entries that are not read are bad
        at = sb
        for r, c in enumerate(own):
            tables[r, first:first + c] = ids[at:at + c]
            at += c
        self.tables = tables
        k = torch.full((nb, block, H, D), math.nan)
        v = torch.full((nb, block, H, D), math.nan)
        if shared:
            j = torch.arange(min(shared, max(self.kv + [0])))
            k[self.shared_blocks[j // block].long(), j % block] = torch.randn(len(j), H, D, generator=g)
            v[self.shared_blocks[j // block].long(), j % block] = torch.randn(len(j), H, D, generator=g)
        for r, m in enumerate(self.kv):
            j = torch.arange(shared, max(shared, m))
            k[tables[r, j // block].long(), j % block] = torch.randn(len(j), H, D, generator=g)
            v[tables[r, j // block].long(), j % block] = torch.randn(len(j), H, D, generator=g)
        self.k, self.v = k.to(BF).to(device), v.to(BF).to(device)  # one layer, token-major: the reference's view
        shape = (layers, nb, H, block, D) if head_major else (layers, nb, block, H, D)
        self.k_cache = torch.full(shape, math.nan, dtype=BF, device=device)
        self.v_cache = torch.full(shape, math.nan, dtype=BF, device=device)
        self.head_major = head_major
        self.sync_cache()
        qkv = torch.randn(T, H * G + 2, D, generator=g).mul_(qscale).to(BF).to(device)
        self.q = qkv[:, 1:1 + H * G]  # a strided slice
        self.device = device

    def sync_cache(self):
        for cache, rows in ((self.k_cache, self.k), (self.v_cache, self.v)):
            cache[self.layer].copy_(rows.transpose(1, 2) if self.head_major else rows)

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.device)

    def reference(self, causal=True, scale=None):
        return attend_reference(self.q, self.q_off, self.start, self.kv, self.tables, self.k, self.v, self.block,
                                self.shared_blocks, self.shared, causal,
                                1 / math.sqrt(self.D) if scale is None else scale)

    def call(self, store, cache, causal=True, **kw):
        args = dict(max_q_len=max(self.n + [1]), causal=causal)
        if self.shared:
            args.update(shared_blocks=self.shared_blocks.to(self.device), shared_len=self.shared)
        args.update(kw)
        return store.attend(self.q, self.i32(self.q_off), self.i32(self.start), self.i32(self.kv),
                            self.tables.to(self.device), cache, self.layer, **args)
