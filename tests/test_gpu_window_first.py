"""Sliding window with first keys that stay visible (ATTN_MASK_FIRST): forward
and reverse of every dense path against the float64 oracle, and the gradients
against differences."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import exact_tiled_attention_softmax_b200 as eta  # noqa: E402
import oracle  # noqa: E402
from exact_tiled_attention_softmax_b200 import workloads as W  # noqa: E402
from oracle import philox as P  # noqa: E402
from tests.parity_util import check_close, to_dev, to_np  # noqa: E402

TORCH_DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    eta.load_library()


def allow_grid(Tq, Tk, *, causal=True, window, first, lengths=None, bm=None, block=0):
    """[B or 1, H or 1, Tq, Tk] truth values of the definition."""
    p = np.arange(Tq)[:, None] + Tk - Tq
    j = np.arange(Tk)[None]
    ok = (j > p - window) | (j < first)
    if causal:
        ok = ok & (j <= p)
    ok = ok[None, None]
    if lengths is not None:
        L = np.asarray(lengths)[:, None, None, None]
        ok = ok & (np.arange(Tq)[:, None] < L) & (j < L)
    if bm is not None:
        ok = ok & (np.repeat(np.repeat(bm, block, 2), block, 3)[:, :, :Tq, :Tk] != 0)
    return ok


CASES = {
    # the gap between first keys and window spans no tile, one tile, many tiles
    "short": dict(shape=(1, 2, 2, 100, 100), window=30, first=4),
    "ragged": dict(shape=(2, 4, 2, 333, 333), window=64, first=1),
    "many_tiles": dict(shape=(1, 2, 1, 1100, 1100), window=130, first=4),
    "aligned": dict(shape=(1, 2, 1, 1024, 1024), window=128, first=128),
    "first_past_a_tile": dict(shape=(1, 2, 1, 1100, 1100), window=100, first=140),
    "first_past_everything": dict(shape=(1, 1, 1, 300, 300), window=5, first=1000),
    "window_of_one": dict(shape=(1, 1, 1, 700, 700), window=1, first=3),
    "window_past_everything": dict(shape=(1, 1, 1, 300, 300), window=5000, first=3),
    "longer_keys": dict(shape=(1, 4, 1, 150, 900), window=90, first=7),
    "shorter_keys": dict(shape=(1, 1, 1, 300, 200), window=90, first=7),
    "open": dict(shape=(1, 2, 1, 400, 600), window=60, first=9, causal=False),
    "lengths": dict(shape=(3, 2, 1, 600, 600), window=60, first=9, lengths=[600, 0, 333]),
    "block": dict(shape=(2, 2, 2, 520, 520), window=200, first=70, block=64),
    "block_odd": dict(shape=(1, 2, 2, 400, 400), window=100, first=30, block=48),
    "sink_dropout": dict(shape=(2, 4, 2, 460, 460), window=90, first=5, sink=True, dropout=0.1),
    "grouped_long": dict(shape=(1, 8, 1, 2100, 2100), window=150, first=4, sink=True),
}


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", list(CASES))
def test_matches_the_oracle(kind, dtype, deterministic):
    c = CASES[kind]
    B, Hq, Hkv, Tq, Tk = c["shape"]
    if dtype == "f32" and (deterministic or Tq > 1100):
        pytest.skip("one fp32 path: the row kernels")
    d = 128 if dtype != "f32" else 40
    rng = np.random.default_rng(11)
    f = lambda s: W.round_to_storage(rng.standard_normal(s, dtype=np.float32), dtype)  # noqa: E731
    q, k, v, g = f((B, Hq, Tq, d)), f((B, Hkv, Tk, d)), f((B, Hkv, Tk, d)), f((B, Hq, Tq, d))
    block, bm = c.get("block", 0), None
    if block:
        bm = (rng.random((B, Hq, -(-Tq // block), -(-Tk // block))) < 0.6).astype(np.uint8)
    sink = rng.standard_normal(Hq).astype(np.float32) if c.get("sink") else None
    rho, seed = c.get("dropout", 0.0), 77
    tdt = TORCH_DTYPE[dtype]
    allowed = eta.AllowedSet(
        causal=c.get("causal", True), window_left=c["window"], window_first=c["first"],
        block_mask=to_dev(bm, torch.uint8) if block else None, block_q=block or 128, block_k=block or 128,
        lengths=torch.tensor(c["lengths"], dtype=torch.int32, device="cuda") if "lengths" in c else None,
        sink=to_dev(sink, torch.float32) if sink is not None else None, dropout_p=rho, dropout_seed=seed,
        deterministic=deterministic)
    tq, tk, tv, tg = (to_dev(x, tdt) for x in (q, k, v, g))
    scale = d ** -0.5
    wf = torch.empty(eta.attn_fwd_workspace_size(tq, tk, tv, allowed), dtype=torch.uint8, device="cuda")
    wb = torch.empty(eta.attn_bwd_workspace_size(tq, tk, tv, allowed), dtype=torch.uint8, device="cuda")
    o, lse = eta.attn_fwd(tq, tk, tv, allowed, scale, workspace=wf)
    dq, dk, dv, dsink = eta.attn_bwd(tq, tk, tv, o, tg, lse, allowed, scale, workspace=wb)
    assert eta.attn_get_status(wf) == 0 and eta.attn_get_status(wb) == 0

    allow = allow_grid(Tq, Tk, causal=c.get("causal", True), window=c["window"], first=c["first"],
                       lengths=c.get("lengths"), bm=bm, block=block)
    keep = P.dropout_keep(seed, rho, B, Hq, Tq, Tk) if rho else None
    q, k, v, g = (x.astype(np.float64) for x in (q, k, v, g))
    z = sink.astype(np.float64) if sink is not None else None
    fw = oracle.forward(q, k, v, allow, scale, sink=z, keep=keep, rho=rho)
    bw = oracle.backward(q, k, v, g, allow, scale, sink=z, keep=keep, rho=rho, y=fw.y)
    fp32 = dtype == "f32"
    check_close("o", to_np(o), fw.y, fp32=fp32, grad=False, storage=dtype)
    for name, got, want in (("dq", dq, bw.dq), ("dk", dk, bw.dk), ("dv", dv, bw.dv)):
        check_close(name, to_np(got), want, fp32=False, grad=True, storage=dtype)
    got_lse = to_np(lse)
    assert np.array_equal(np.isinf(got_lse), np.isinf(fw.lse))
    live = np.isfinite(fw.lse)
    assert np.abs(got_lse[live] - fw.lse[live]).max() <= 2.0 ** -12 + 2.0 ** -20 * np.abs(fw.lse[live]).max()
    if sink is not None:
        check_close("dsink", to_np(dsink), bw.dsink, fp32=False, grad=True)
    if deterministic:
        again = eta.attn_bwd(tq, tk, tv, o, tg, lse, allowed, scale)
        for a, b in zip((dq, dk, dv), again):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sink_gradient_is_fp32_accurate(dtype):
    """dz_h = -sum_i p_i delta_i with delta in fp32: each term's error is 2^-18
    of sum_j p_ij |dP_ij| at most (scores and dP are fp32 sums of 128
    products, the LSE is off by 4e-6 at most), so the sum's is 2^-18 of the
    terms' magnitudes."""
    B, Hq, Hkv, T, W_, F = 2, 4, 2, 700, 96, 5
    rng = np.random.default_rng(21)
    f = lambda s: W.round_to_storage(rng.standard_normal(s, dtype=np.float32), dtype)  # noqa: E731
    q, k, v, g = f((B, Hq, T, 128)), f((B, Hkv, T, 128)), f((B, Hkv, T, 128)), f((B, Hq, T, 128))
    sink = rng.standard_normal(Hq).astype(np.float32)
    tq, tk, tv, tg = (to_dev(x, TORCH_DTYPE[dtype]) for x in (q, k, v, g))
    allowed = eta.AllowedSet(causal=True, window_left=W_, window_first=F, sink=to_dev(sink, torch.float32))
    o, lse = eta.attn_fwd(tq, tk, tv, allowed)
    dsink = eta.attn_bwd(tq, tk, tv, o, tg, lse, allowed)[3]
    allow = allow_grid(T, T, window=W_, first=F)
    q, k, v, g = (x.astype(np.float64) for x in (q, k, v, g))
    fw = oracle.forward(q, k, v, allow, 128 ** -0.5, sink=sink.astype(np.float64))
    bw = oracle.backward(q, k, v, g, allow, 128 ** -0.5, sink=sink.astype(np.float64), y=fw.y)
    kk, vv = np.repeat(k, Hq // Hkv, 1), np.repeat(v, Hq // Hkv, 1)
    s = np.where(allow, np.einsum("bhid,bhjd->bhij", q, kk) * 128 ** -0.5, -np.inf)
    p = np.exp(s - fw.lse[..., None])
    size = (np.exp(sink[:, None] - fw.lse) * (p * np.abs(np.einsum("bhid,bhjd->bhij", g, vv))).sum(-1)).sum((0, 2))
    assert (np.abs(to_np(dsink) - bw.dsink) <= 2.0 ** -17 * size).all(), (to_np(dsink) - bw.dsink, size)


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["lengths", "shorter_keys", "block"])
def test_sink_gradient_with_query_tiles_that_see_no_key(kind, dtype, deterministic):
    """Rows without a key give the sink all of their probability and no
    gradient (delta 0), whole 128-row tiles of them too: a batch row of length
    0, queries in front of the first key, an all-zero stripe of the block mask.
    The bound is test_sink_gradient_is_fp32_accurate's; such rows add nothing to it."""
    B, Hq, Hkv, W_, F, d = 3, 4, 2, 60, 9, 128
    Tq, Tk = (700, 350) if kind == "shorter_keys" else (600, 600)
    lengths = [600, 0, 200] if kind == "lengths" else None
    block, bm = 64, None
    rng = np.random.default_rng(31)
    if kind == "block":
        bm = (rng.random((B, Hq, -(-Tq // block), -(-Tk // block))) < 0.6).astype(np.uint8)
        bm[:, :, 2:6] = 0  # query rows 128 .. 383
    f = lambda s: W.round_to_storage(rng.standard_normal(s, dtype=np.float32), dtype)  # noqa: E731
    q, k, v, g = f((B, Hq, Tq, d)), f((B, Hkv, Tk, d)), f((B, Hkv, Tk, d)), f((B, Hq, Tq, d))
    sink = rng.standard_normal(Hq).astype(np.float32)
    tq, tk, tv, tg = (to_dev(x, TORCH_DTYPE[dtype]) for x in (q, k, v, g))
    allowed = eta.AllowedSet(
        causal=True, window_left=W_, window_first=F, sink=to_dev(sink, torch.float32), deterministic=deterministic,
        block_mask=to_dev(bm, torch.uint8) if bm is not None else None, block_q=block, block_k=block,
        lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda") if lengths else None)
    wb = torch.empty(eta.attn_bwd_workspace_size(tq, tk, tv, allowed), dtype=torch.uint8, device="cuda")
    o, lse = eta.attn_fwd(tq, tk, tv, allowed)
    dq, dk, dv, dsink = eta.attn_bwd(tq, tk, tv, o, tg, lse, allowed, workspace=wb)
    assert eta.attn_get_status(wb) == 0
    allow = allow_grid(Tq, Tk, window=W_, first=F, lengths=lengths, bm=bm, block=block)
    q, k, v, g = (x.astype(np.float64) for x in (q, k, v, g))
    z = sink.astype(np.float64)
    fw = oracle.forward(q, k, v, allow, d ** -0.5, sink=z)
    bw = oracle.backward(q, k, v, g, allow, d ** -0.5, sink=z, y=fw.y)
    for name, got, want in (("dq", dq, bw.dq), ("dk", dk, bw.dk), ("dv", dv, bw.dv)):
        check_close(name, to_np(got), want, fp32=False, grad=True, storage=dtype)
    kk, vv = np.repeat(k, Hq // Hkv, 1), np.repeat(v, Hq // Hkv, 1)
    s = np.where(allow, np.einsum("bhid,bhjd->bhij", q, kk) * d ** -0.5, -np.inf)
    assert np.isneginf(s).all(-1).reshape(B, Hq, -1)[:, :, :Tq // 128 * 128].reshape(B, Hq, -1, 128).all(-1).any()
    p = np.exp(s - fw.lse[..., None])
    size = (np.exp(sink[:, None] - fw.lse) * (p * np.abs(np.einsum("bhid,bhjd->bhij", g, vv))).sum(-1)).sum((0, 2))
    assert (np.abs(to_np(dsink) - bw.dsink) <= 2.0 ** -17 * size).all(), (to_np(dsink) - bw.dsink, size)


def test_gradients_against_differences():
    """fp32, autograd: <grad, u> against a central difference along u. With
    h = 2^-6 the difference's own error is h^2/6 times a third derivative
    (values of order one over 200 rows) and 2^-24 |L| / h of rounding: both
    stay below 2^-10 of |u||grad|."""
    torch.manual_seed(3)
    q, k, v = (torch.randn(1, h, 70, 16, device="cuda", requires_grad=True) for h in (2, 1, 1))
    sink = torch.randn(2, device="cuda", requires_grad=True)
    w = torch.randn(1, 2, 70, 16, device="cuda")

    def loss(q, k, v, z):
        o, _ = eta.attention(q, k, v, eta.AllowedSet(causal=True, window_left=9, window_first=3), 0.25, sink=z)
        return (o * w).double().sum()

    x = [q, k, v, sink]
    grads = torch.autograd.grad(loss(*x), x)
    for i, g in enumerate(grads):
        u = g / g.norm()
        h = 2.0 ** -6
        with torch.no_grad():
            up = loss(*[t + h * u if n == i else t for n, t in enumerate(x)])
            dn = loss(*[t - h * u if n == i else t for n, t in enumerate(x)])
        diff, want = float((up - dn) / (2 * h)), float((g * u).sum())
        assert math.isclose(diff, want, rel_tol=2.0 ** -8, abs_tol=2.0 ** -10 * float(g.norm())), (i, diff, want)
