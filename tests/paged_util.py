"""Shared helpers of the paged-cache tests: seeded caches whose unused
positions hold NaN, and the operator's definition in float64.

Error bounds of attn_paged_fwd, against the float64 result on the same
(rounded, dequantised) inputs; A = sum_j p_ij |V_jc|:
  output rounding: half a step, eps / 2 relative, of the output's type (below
    the smallest normal, half the smallest subnormal step);
  rounding of the probabilities in front of V (tensor-core kernels only):
    eps / 2 of the 16-bit operand type, relative to A. The operand type is the
    cache's, and fp16 in front of an e4m3 cache: 2^-11 for the probability, and
    where V's scale is in V's operand 2^-11 for the scale and 2^-11 for the
    product, below 2^-9 A together;
  the exponentials and the fp32 sums: scores come from d <= 576 products of
    magnitude at most |q||k| summed in fp32 (relative 2^-24 per step, so
    below 2^-15 absolute for |s| <= 16), and 2^x has a relative error of at
    most 3.1e-6 where a quartic stands in for it: 2^-12 relative to A covers
    both in numerator and denominator.
  LSE: 2^-12 absolute by the same two terms, plus 2^-20 of its magnitude.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import exact_tiled_attention_softmax_b200 as eta

E4M3 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": E4M3}


def quantise(x):
    """The e4m3 form of rows x (last dimension): codes and fp32 scales."""
    a = x.float().abs().amax(-1)
    s = a / 448.0
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (x.float() / s[..., None]).clamp(-448, 448).to(E4M3), s


def make_cache(lens, page, Hkv, d, dv, dtype, *, heads_first=True, seed=0, spare=3, src=None, device="cuda"):
    """A cache with N(0, 1) rows at every used position and NaN elsewhere;
    pages in random order. Returns (PagedCache, dense fp64 K list, V list):
    per sequence [L, Hkv, d] of the values the cache stands for."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = [-(-L // page) for L in lens]
    P = sum(pages) + spare
    order = torch.randperm(P, generator=g)
    M = max(pages + [1])
    table = torch.full((B, M), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    quant = dtype == E4M3
    store = torch.float32 if quant else dtype
    pools, scales, dense = [], [], []
    for width in (d, dv):
        x = torch.full((P, page, Hkv, width), math.nan, dtype=store)
        sc = torch.full((P, page, Hkv), math.nan)
        code = torch.full((P, page, Hkv, width), math.nan).to(E4M3)
        rows = []
        for b, L in enumerate(lens):
            r = torch.randn(L, Hkv, width, generator=g).to(src or store)
            pos = torch.arange(L)
            pg, off = table[b].long()[pos // page], pos % page
            if quant:
                c, s = quantise(r)
                code.view(torch.uint8)[pg, off] = c.view(torch.uint8)
                sc[pg, off] = s
                rows.append(c.double() * s.double()[..., None])
            else:
                x[pg, off] = r.to(store)
                rows.append(r.to(store).double())
        pools.append(code if quant else x)
        scales.append(sc if quant else None)
        dense.append(rows)

    def lay(t):
        if t is None:
            return None
        t = t.to(device)
        if not heads_first:
            return t
        if t.dtype == E4M3:
            return t.view(torch.uint8).transpose(1, 2).contiguous().view(E4M3).transpose(1, 2)
        return t.transpose(1, 2).contiguous().transpose(1, 2)

    cache = eta.PagedCache(lay(pools[0]), lay(pools[1]), table.to(device),
                           torch.tensor(lens, dtype=torch.int32, device=device), lay(scales[0]), lay(scales[1]))
    return cache, dense[0], dense[1]


def cu_of(new, device="cuda"):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=device)


def seen(n, L, *, causal=True, window=0, first=0):
    """[n, L] truth values: does new token i see key j?"""
    p = torch.arange(L - n, L)[:, None]
    j = torch.arange(L)[None]
    ok = torch.ones(n, L, dtype=torch.bool)
    if causal:
        ok &= j <= p
    if window:
        ok &= (j > p - window) | (j < first)
    return ok & (p >= 0)


def reference(q, K, V, new, lens, scale, *, sink=None, skip=None, **mask):
    """(o, lse, A) in float64, rows in order; A = sum_j p_ij |V_j|. skip: per
    sequence a set of positions that belong to no set."""
    rows, Hq, d = q.shape
    dv = V[0].shape[-1]
    o, A = torch.zeros(rows, Hq, dv, dtype=torch.float64), torch.zeros(rows, Hq, dv, dtype=torch.float64)
    lse = torch.full((rows, Hq), -math.inf, dtype=torch.float64)
    t = 0
    for b, (n, L) in enumerate(zip(new, lens)):
        g = Hq // K[b].shape[1]
        ok = seen(n, L, **mask)
        if skip and skip[b]:
            ok[:, sorted(skip[b])] = False
        for h in range(Hq):
            k, v = K[b][:, h // g].clone(), V[b][:, h // g].clone()
            s = (q[t:t + n, h].double().cpu() @ torch.where(torch.isnan(k), 0.0, k).T) * scale
            if torch.isnan(k).any():
                s[:, torch.isnan(k).any(1)] = math.nan
            s = torch.where(ok, s, torch.tensor(-math.inf, dtype=torch.float64))
            z = -math.inf if sink is None else float(sink[h])
            for i in range(n):
                a = ok[i]
                x = s[i][a]
                l = torch.logsumexp(torch.cat([x, torch.tensor([z], dtype=torch.float64)]), 0)
                lse[t + i, h] = l
                if a.any():
                    p = torch.exp(x - l)
                    o[t + i, h] = p @ v[a]
                    A[t + i, h] = p @ v[a].abs()
        t += n
    return o, lse, A


def check(got_o, got_lse, o, lse, A, *, tensor_core, cache="same"):
    """tensor_core: the output may come from the tensor-core kernels; cache: the
    cache's type where it is not the output's."""
    dt = got_o.dtype
    eps = torch.finfo(dt).eps / 2
    bound = eps * o.abs() + torch.finfo(dt).smallest_normal * eps + 2.0 ** -12 * A
    if tensor_core:
        bound = bound + (2.0 ** -9 if cache in ("e4m3", E4M3) else eps) * A
    err = (got_o.double().cpu() - o).abs()
    bad = ~(err <= bound * (1 + 1e-6))
    assert not bad.any(), f"o: {int(bad.sum())} of {bad.numel()} past the bound, worst {float((err - bound).max()):.3e}"
    gl = got_lse.double().cpu()
    assert torch.equal(torch.isinf(gl), torch.isinf(lse)), "empty rows differ"
    f = torch.isfinite(lse)
    el = (gl[f] - lse[f]).abs() - (2.0 ** -12 + 2.0 ** -20 * lse[f].abs())
    assert not f.any() or float(el.max()) <= 0, f"lse past its bound by {float(el.max()):.3e}"


def seeded_q(rows, Hq, d, dtype, seed=1, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, Hq, d, generator=g).to(dtype).to(device)


def run(q, cache, new=None, *, allowed=None, scale=None, max_q=0, status=0, **kw):
    """attn_paged_fwd with the workspace's status word checked afterwards."""
    ws = torch.empty(eta.attn_paged_workspace_size(q, cache, allowed), dtype=torch.uint8, device=q.device)
    cu = None if new is None else cu_of(new)
    o, lse = eta.attn_paged_fwd(q, cache, cu, allowed, scale, max_q=max_q, workspace=ws, **kw)
    assert eta.attn_get_status(ws) == status
    return o, lse
