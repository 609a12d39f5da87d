"""Host-side checks of the paged-cache entry points and of the first-token
set: what they refuse, before any launch. No kernel runs, so no GPU is needed."""
import ctypes
import os
import shutil
import subprocess

import pytest

from tests.test_abi import ROOT, _call_fwd, _t, lib  # noqa: F401  (lib is a fixture)

import exact_tiled_attention_softmax_b200 as eta


def _cache(dtype=1, pages=10, page=16, Hkv=2, d=128, dv=128, batch=3, max_pages=4):
    c = eta.AttnCacheC()
    c.k, c.v = _t([pages, page, Hkv, d], dtype), _t([pages, page, Hkv, dv], dtype)
    if dtype == eta.ATTN_E4M3:
        c.k_scale, c.v_scale = _t([pages, page, Hkv], 0), _t([pages, page, Hkv], 0)
    c.block_table, c.table_stride, c.max_pages, c.batch, c.seq_lens = 0x5000, max_pages, max_pages, batch, 0x6000
    return c


def _write(lib, c, k=None, v=None, cu=0x7000, ws=0x100008, n=256):  # noqa: F811
    """Stops at the misaligned workspace when every earlier check passes."""
    k = k or _t([6, 2, 128])
    v = v or _t([6, 2, 128])
    return lib.attn_cache_write(ctypes.byref(k), ctypes.byref(v), cu, ctypes.byref(c), ws, n, None)


def _fwd(lib, c, q=None, o=None, lse=None, mask=None, cu=0x7000, scale=0.1, max_q=0, ws=0x100008, n=1 << 30):  # noqa: F811
    q = q or _t([6, 4, 128])
    o = o or _t([6, 4, 128])
    lse = lse or _t([6, 4], 0)
    return lib.attn_paged_fwd(ctypes.byref(q), cu, ctypes.byref(c), ctypes.byref(mask) if mask else None,
                              ctypes.c_float(scale), max_q, ctypes.byref(o), ctypes.byref(lse), ws, n, None)


def _read(lib, c, k=None, v=None, ws=0x100008, n=256):  # noqa: F811
    k = k or _t([3, 2, 50, 128])
    v = v or _t([3, 2, 50, 128])
    return lib.attn_cache_read(ctypes.byref(c), ctypes.byref(k), ctypes.byref(v), ws, n, None)


def test_good_arguments_reach_the_workspace_check(lib):  # noqa: F811
    for dt in (0, 1, 2, 3):
        rows = dt if dt != 3 else 1
        c = _cache(dt)
        assert _write(lib, c, _t([6, 2, 128], rows), _t([6, 2, 128], rows)) == eta.ATTN_ERR_WORKSPACE
        assert _read(lib, c, _t([3, 2, 50, 128], rows), _t([3, 2, 50, 128], rows)) == eta.ATTN_ERR_WORKSPACE
        assert _fwd(lib, c, _t([6, 4, 128], rows), _t([6, 4, 128], rows)) == eta.ATTN_ERR_WORKSPACE
    assert _fwd(lib, _cache(), ws=0) == eta.ATTN_ERR_WORKSPACE
    assert _fwd(lib, _cache(), ws=0x100000, n=16) == eta.ATTN_ERR_WORKSPACE
    assert _write(lib, _cache(), ws=0x100000, n=16) == eta.ATTN_ERR_WORKSPACE


def _broken():
    """(what is wrong, descriptor, status)"""
    bad, uns = eta.ATTN_ERR_INVALID_ARG, eta.ATTN_ERR_UNSUPPORTED

    def c(**kw):
        x = _cache(**{k: v for k, v in kw.items() if k in ("dtype", "pages", "page", "Hkv", "d", "dv", "batch",
                                                           "max_pages")})
        for k, v in kw.items():
            if k in ("k", "v", "k_scale", "v_scale", "block_table", "table_stride", "seq_lens"):
                setattr(x, k, v)
        return x

    yield "rank", c(k=_t([10, 16, 128])), bad
    yield "pool shapes differ", c(v=_t([9, 16, 2, 128])), bad
    yield "pool types differ", c(v=_t([10, 16, 2, 128], 2)), bad
    yield "inner stride", c(k=_t([10, 16, 2, 128], stride=[8192, 512, 256, 2])), bad
    yield "broadcast pool", c(k=_t([10, 16, 2, 128], stride=[0, 256, 128, 1])), bad
    yield "no pool", c(k=_t([10, 16, 2, 128], data=0)), bad
    yield "odd address", c(k=_t([10, 16, 2, 128], data=0x1001)), bad
    yield "e4m3 without scales", c(dtype=3, k_scale=_t([10, 16, 2], 0, data=0)), bad
    yield "scales of another shape", c(dtype=3, v_scale=_t([10, 16, 3], 0)), bad
    yield "16-bit scales", c(dtype=3, v_scale=_t([10, 16, 2], 1)), bad
    yield "scales of a bf16 pool", c(k_scale=_t([10, 16, 2], 0)), bad
    yield "rows of the table overlap", c(table_stride=2), bad
    yield "no table", c(block_table=0), bad
    yield "no lengths", c(seq_lens=0), bad
    yield "negative batch", c(batch=-1), bad
    yield "unknown type", c(dtype=4), bad
    yield "wide head", c(d=640), uns
    yield "positions past 32 bits", c(max_pages=1 << 28), uns


def test_broken_descriptors_are_refused(lib):  # noqa: F811
    for what, c, want in _broken():
        dt = c.k.dtype if c.k.dtype < 3 else 1
        w = c.k.shape[c.k.ndim - 1]
        assert _write(lib, c, _t([6, 2, w], dt), _t([6, 2, 128], dt)) == want, what
        assert _read(lib, c, _t([max(c.batch, 0), 2, 50, w], dt), _t([max(c.batch, 0), 2, 50, 128], dt)) == want, what
        assert _fwd(lib, c, _t([6, 4, w], dt), _t([6, 4, 128], dt)) == want, what


def test_calls_that_do_not_fit_the_cache_are_refused(lib):  # noqa: F811
    bad, uns = eta.ATTN_ERR_INVALID_ARG, eta.ATTN_ERR_UNSUPPORTED
    c = _cache()
    assert _write(lib, c, _t([6, 2, 64])) == bad            # head width
    assert _write(lib, c, _t([6, 3, 128])) == bad           # heads
    assert _write(lib, c, _t([7, 2, 128])) == bad           # K and V rows differ
    assert _write(lib, c, _t([6, 2, 128], 2), _t([6, 2, 128], 2)) == bad  # fp16 rows, bf16 pool
    assert _write(lib, c, _t([7, 2, 128]), _t([7, 2, 128]), cu=None) == bad  # 7 tokens, 3 sequences alike
    assert _write(lib, c, _t([6, 2, 128], data=0)) == bad
    assert _write(lib, _cache(batch=0), cu=None) == bad
    assert _write(lib, _cache(3), _t([6, 2, 128], 3), _t([6, 2, 128], 3)) == bad  # e4m3 rows
    assert _read(lib, c, _t([2, 2, 50, 128])) == bad        # batch
    assert _read(lib, c, _t([3, 2, 50, 128], 0), _t([3, 2, 50, 128], 0)) == bad  # fp32 out of a bf16 pool
    assert _read(lib, c, _t([3, 2, 50, 128], stride=[0, 6400, 128, 1])) == bad
    assert _read(lib, _cache(3), _t([3, 2, 50, 128], 3), _t([3, 2, 50, 128], 3)) == bad
    assert _fwd(lib, c, _t([6, 3, 128]), _t([6, 3, 128]), _t([6, 3], 0)) == bad  # 3 heads over 2
    assert _fwd(lib, c, _t([6, 4, 64])) == bad
    assert _fwd(lib, c, o=_t([6, 4, 64])) == bad
    assert _fwd(lib, c, o=_t([6, 4, 128], 2)) == bad
    assert _fwd(lib, c, lse=_t([6, 4], 1)) == bad
    assert _fwd(lib, c, lse=_t([6, 5], 0)) == bad
    assert _fwd(lib, c, o=_t([6, 4, 128], stride=[0, 128, 1])) == bad
    assert _fwd(lib, c, scale=float("inf")) == bad
    assert _fwd(lib, c, max_q=-1) == bad
    for kw, want in ((dict(dropout_p=0.5), uns), (dict(causal=True, window_left=4, window_first=2), None),
                     (dict(window_first=2), bad), (dict(window_left=4, window_first=-2), bad)):
        m = eta.AllowedSet(**kw).to_c()
        assert _fwd(lib, c, mask=m) == (eta.ATTN_ERR_WORKSPACE if want is None else want), kw
    for flag in (eta.ATTN_MASK_BLOCK, eta.ATTN_MASK_LENGTHS, eta.ATTN_MASK_STARTS):
        m = eta.AttnMaskC()
        m.flags, m.block_mask, m.lengths, m.starts, m.block_q, m.block_k = flag, 0x100, 0x100, 0x100, 1, 1
        assert _fwd(lib, c, mask=m) == uns


def test_first_tokens_need_a_window_and_no_starts(lib):  # noqa: F811
    q, o, lse = _t([1, 4, 64, 128]), _t([1, 4, 64, 128]), _t([1, 4, 64], dtype=0)

    def call(m):
        return _call_fwd(lib, q, q, q, o, lse, mask=m, ws=0x100010)

    assert call(eta.AllowedSet(causal=True, window_left=8, window_first=2).to_c()) == eta.ATTN_ERR_WORKSPACE
    assert call(eta.AllowedSet(causal=True, window_first=2).to_c()) == eta.ATTN_ERR_INVALID_ARG
    assert call(eta.AllowedSet(causal=True, window_left=8, window_first=-1).to_c()) == eta.ATTN_ERR_INVALID_ARG
    m = eta.AllowedSet(causal=True, window_left=8, window_first=2).to_c()
    m.flags |= eta.ATTN_MASK_STARTS
    m.starts = 0x4000
    assert call(m) == eta.ATTN_ERR_UNSUPPORTED
    m = eta.AllowedSet(causal=True, window_left=8).to_c()
    m.window_first = -5  # not read without its flag
    assert call(m) == eta.ATTN_ERR_WORKSPACE


def test_cache_struct_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "attn.h"', "int main(void) {",
             '  printf("size %zu\\n", sizeof(attn_cache));']
    lines += [f'  printf("{f} %zu\\n", offsetof(attn_cache, {f}));' for f, _ in eta.AttnCacheC._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split("\n")
    got = {x.split()[0]: int(x.split()[1]) for x in out if x}
    assert got.pop("size") == ctypes.sizeof(eta.AttnCacheC)
    assert got == {f: getattr(eta.AttnCacheC, f).offset for f, _ in eta.AttnCacheC._fields_}


def test_binding_refuses_host_tensors_and_wrong_tables():
    torch = pytest.importorskip("torch")
    pool = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        eta.PagedCache(pool, pool, table, lens).to_c()
    with pytest.raises(ValueError, match="block_table"):
        eta.PagedCache(pool, pool, table.long(), lens).to_c()
    with pytest.raises(ValueError, match="different numbers"):
        eta.PagedCache(pool, pool, table, lens[:1]).to_c()


def test_binding_refuses_a_sink_shorter_than_the_heads():
    """The library reads a logit, and writes a gradient, per query head; the
    binding sees how many there are."""
    torch = pytest.importorskip("torch")
    z = torch.zeros(3)
    a = eta.AllowedSet(causal=True, sink=z)
    q, o, lse = torch.zeros(1, 4, 8, 16), torch.zeros(1, 4, 8, 16), torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="sink: 3 entries for 4"):
        eta.attn_fwd(q, q, q, a)
    with pytest.raises(ValueError, match="sink: 3 entries for 4"):
        eta.attn_bwd(q, q, q, o, o, lse, a, dsink=torch.zeros(4))
    full = eta.AllowedSet(causal=True, sink=torch.zeros(4))
    with pytest.raises(ValueError, match="dsink: 3 entries for 4"):
        eta.attn_bwd(q, q, q, o, o, lse, full, dsink=z)
    with pytest.raises(ValueError, match="dsink: 3 entries for 4"):
        eta.attn_bwd_noalloc(q, q, q, o, o, lse, full, dq=q, dk=q, dv=q, dsink=z)
    topk = eta.AllowedSet(topk_idxs=torch.zeros(6, 2, dtype=torch.int32), sink=z)
    with pytest.raises(ValueError, match="sink: 3 entries for 4"):
        eta.attn_fwd(torch.zeros(6, 4, 16), torch.zeros(9, 16), torch.zeros(9, 16), topk)
    pool = torch.zeros(4, 16, 2, 16)
    cache = eta.PagedCache(pool, pool, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="sink: 3 entries for 4"):
        eta.attn_paged_fwd(torch.zeros(6, 4, 16), cache, None, a)
    # one that is long enough goes on to the next check
    with pytest.raises(ValueError, match="CUDA"):
        eta.attn_paged_fwd(torch.zeros(6, 4, 16), cache, None, full)


def test_quartic_exponential():
    """The quartic that stands in for some exponentials where the sum's logarithm
    is an fp32 output: the kernel's fp32 steps in NumPy, and its coefficients
    from the generator."""
    import importlib.util

    import numpy as np
    path = os.path.join(ROOT, "exact_tiled_attention_softmax_b200", "csrc", "gen_exp2_poly.py")
    spec = importlib.util.spec_from_file_location("gen_exp2_poly", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    coeffs, err = mod.fit(4)
    text = open(os.path.join(os.path.dirname(path), "sm100_ptx.cuh")).read()
    for c in coeffs[1:]:
        assert f"{float(np.float32(c))!r}f" in text
    assert err < 3.1e-6
    x = np.linspace(-120.0, 8.0, 500_001, dtype=np.float32)
    t = (x + np.float32(12582912.0)).astype(np.float32)
    f = (x - (t - np.float32(12582912.0))).astype(np.float32)
    p = np.float32(coeffs[4])
    for c in coeffs[3::-1]:
        p = (p * f + np.float32(c)).astype(np.float32)
    n = t.view(np.int32) - np.int32(0x4B400000)
    got = (p.view(np.int32) + (n << 23)).view(np.float32).astype(np.float64)
    # the fit's error, and four roundings of 2^-24 (one is relative to terms below 1)
    assert np.abs(got / np.exp2(x.astype(np.float64)) - 1).max() < 3.1e-6 + 4 * 2.0 ** -23


def test_addresses_between_elements_are_refused(lib):  # noqa: F811
    bad = eta.ATTN_ERR_INVALID_ARG
    odd = _t([6, 2, 128], data=0x1001)
    assert _write(lib, _cache(), odd) == bad
    assert _write(lib, _cache(), v=odd) == bad
    half = _t([6, 2, 128], 0, data=0x1002)  # fp32 rows at a 2-byte boundary
    assert _write(lib, _cache(3), half, _t([6, 2, 128], 0)) == bad
    assert _fwd(lib, _cache(), _t([6, 4, 128], data=0x1001)) == bad
    for field in ("block_table", "seq_lens"):
        c = _cache()
        setattr(c, field, 0x5002)
        assert _write(lib, c) == bad and _fwd(lib, c) == bad and _read(lib, c) == bad
    assert _write(lib, _cache(), cu=0x7001) == bad
    assert _fwd(lib, _cache(), cu=0x7001) == bad


def test_more_sequences_than_positions_are_refused(lib):  # noqa: F811
    c = _cache(batch=(1 << 30) + 1)
    assert _write(lib, c) == eta.ATTN_ERR_UNSUPPORTED
    assert _fwd(lib, c) == eta.ATTN_ERR_UNSUPPORTED


def test_quartic_exponential_at_its_lower_end():
    """The kernels clamp its argument at -127, where it is exactly 0, so that a
    score of -inf has no share; above that it is small and not negative."""
    import numpy as np
    f32 = np.float32
    c = [f32(x) for x in (1.0, 0.6931219696998596, 0.24023719131946564, 0.05591689422726631, 0.00960039533674717)]
    text = open(os.path.join(ROOT, "exact_tiled_attention_softmax_b200", "csrc", "sm100_ptx.cuh")).read()
    assert all(f"{float(x)!r}f" in text for x in c[1:])
    x = np.concatenate([[f32(-127)], np.linspace(-127, -124, 100_001, dtype=f32)])
    t = (x + f32(12582912.0)).astype(f32)
    f = (x - (t - f32(12582912.0))).astype(f32)
    p = np.full_like(f, c[4])
    for a in c[3::-1]:
        p = (p * f + a).astype(f32)
    n = t.view(np.int32) - np.int32(0x4B400000)
    got = (p.view(np.int32) + (n << 23)).view(f32)
    assert got[0] == 0 and not np.signbit(got[0])
    assert (got >= 0).all() and (got[x <= -125] <= f32(2.0) ** -124).all()
