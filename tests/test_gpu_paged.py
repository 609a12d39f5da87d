"""Paged caches on the GPU: the write, the read back and the attention over a
cache against their float64 definitions, at the sizes and masks where they can
go wrong, and a serving run of them together."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import exact_tiled_attention_softmax_b200 as eta  # noqa: E402
from tests.paged_util import (DT, E4M3, check, cu_of, make_cache, quantise, reference, run,  # noqa: E402
                              seeded_q)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    eta.load_library()


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


# ------------------------------------------------------------- write, read


WRITES = {
    "one_token_each": dict(lens=[1, 17, 40, 64], new=[1, 1, 1, 1], page=16, Hkv=8, d=128, dv=128),
    "ragged_with_none": dict(lens=[33, 20, 5, 130], new=[33, 0, 2, 70], page=32, Hkv=3, d=128, dv=128),
    "wide_and_narrow_heads": dict(lens=[50, 9], new=[30, 9], page=64, Hkv=2, d=576, dv=72),
    "odd_width": dict(lens=[50, 9], new=[30, 9], page=5, Hkv=2, d=33, dv=20),
}


@pytest.mark.parametrize("heads_first", [True, False])
@pytest.mark.parametrize("src,store", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"),
                                       ("f16", "e4m3"), ("f32", "e4m3")])
@pytest.mark.parametrize("kind", list(WRITES))
def test_write_then_read(kind, src, store, heads_first):
    c = WRITES[kind]
    cache, _, _ = make_cache(c["lens"], c["page"], c["Hkv"], c["d"], c["dv"], DT[store], heads_first=heads_first, seed=3)
    before = [bits(t) for t in cache.tensors()]
    rows = sum(c["new"])
    k, v = seeded_q(rows + 2, c["Hkv"], c["d"], DT[src], 5), seeded_q(rows + 2, c["Hkv"], c["dv"], DT[src], 6)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    eta.attn_cache_write(k, v, cache, cu_of(c["new"]), workspace=ws)
    assert eta.attn_get_status(ws) == 0
    # what the pool holds now: the new rows at their slots, all else as it was
    want = [t.clone() for t in before]
    table, at = cache.block_table.cpu(), 0
    for b, (n, L) in enumerate(zip(c["new"], c["lens"])):
        pos = torch.arange(L - n, L)
        pg, off = table[b].long()[pos // c["page"]], pos % c["page"]
        for i, new in enumerate((k, v)):
            r = new[at:at + n].cpu()
            if store == "e4m3":
                code, s = quantise(r)
                want[i][pg, off] = code.view(torch.uint8)
                want[4 + i][pg, off] = s.view(torch.int32)
            else:
                want[i][pg, off] = bits(r)
        at += n
    for got, w in zip(cache.tensors(), want):
        assert torch.equal(bits(got), w)
    # and back: every row the sequences hold, the rows past them untouched
    T = max(c["lens"]) + 3
    for out in (["bf16", "f16", "f32"] if store == "e4m3" else [store]):
        B = len(c["lens"])
        ok = torch.full((B, T, c["Hkv"], c["d"]), 7.0, dtype=DT[out], device="cuda").transpose(1, 2)
        ov = torch.full((B, c["Hkv"], T, c["dv"]), 7.0, dtype=DT[out], device="cuda")
        eta.attn_cache_read(cache, k=ok, v=ov, workspace=ws)
        assert eta.attn_get_status(ws) == 0
        for got, pool, scale in ((ok, cache.k, cache.k_scale), (ov, cache.v, cache.v_scale)):
            vals = pool.float().cpu() if scale is None else pool.float().cpu() * scale.cpu()[..., None]
            for b, L in enumerate(c["lens"]):
                pos = torch.arange(L)
                r = vals[table[b].long()[pos // c["page"]], pos % c["page"]].to(DT[out])
                assert torch.equal(got[b, :, :L].cpu(), r.transpose(0, 1))
                assert (got[b, :, L:] == 7).all()


def test_write_of_special_rows():
    """Zero rows, rows of the smallest values, and rows with an infinity or a
    NaN: zeros stay zeros, finite rows stay finite, the others read as NaN."""
    cache, _, _ = make_cache([6], 16, 1, 128, 128, E4M3, seed=1)
    k = torch.zeros(6, 1, 128, device="cuda")
    k[1, 0, 3] = 1e-45
    k[1, 0, 4] = -0.0
    k[2, 0, 5] = math.inf
    k[3, 0, 6] = math.nan
    k[4] = 3e38
    k[5] = torch.linspace(-448, 448, 128)
    eta.attn_cache_write(k, k, cache)
    for got in eta.attn_cache_read(cache, 6, dtype=torch.float32):
        got = got[0, 0].cpu()
        assert (got[0] == 0).all() and (got[1] == 0).all()
        assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
        # (3e38 / s) is 448 up to one rounding each way, and back times s
        assert torch.allclose(got[4], torch.full((128,), 3e38), rtol=2.0 ** -22)
        # e4m3: half a step relative, 2^-10 of the scale for the subnormal codes
        assert ((got[5] - k[5, 0].cpu()).abs() <= k[5, 0].cpu().abs() * 2.0 ** -4 + 2.0 ** -10).all()


@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
def test_codes_at_every_magnitude(src):
    """Codes and scales equal the correctly rounded quotients, bit for bit, for
    rows of every magnitude the type holds, values on borders among them."""
    g = torch.Generator().manual_seed(4)
    top = {"bf16": 127, "f16": 15, "f32": 127}[src]
    n = 2 * top + 10
    mag = 2.0 ** torch.linspace(-top - 8, top - 1, n).double()
    x = torch.randn(n, 2, 128, generator=g).double().clamp(-1, 1)
    x[:, 0, :64] = torch.randint(-448, 449, (n, 64), generator=g) / 448.0  # on and between codes
    x = (x * mag[:, None, None]).to(DT[src])
    cache, _, _ = make_cache([n], 16, 2, 128, 128, E4M3, seed=1)
    eta.attn_cache_write(x.cuda(), x.flip(0).contiguous().cuda(), cache)
    pos = torch.arange(n)
    at = cache.block_table[0].long().cpu()[pos // 16], pos % 16
    for pool, scale, rows in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, x.flip(0))):
        code, s = quantise(rows)
        assert torch.equal(bits(scale)[at], s.view(torch.int32))
        assert torch.equal(pool.view(torch.uint8).cpu()[at], code.view(torch.uint8))


def test_write_and_read_report_bad_pages_and_lengths():
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    cache, K, _ = make_cache([40, 20], 16, 2, 128, 128, torch.bfloat16, seed=2)
    cache.block_table[0, 1] = cache.k.shape[0]  # one past the pool: positions 16..31 of sequence 0
    before = bits(cache.k)
    k = seeded_q(60, 2, 128, torch.bfloat16)
    eta.attn_cache_write(k, k, cache, cu_of([40, 20]), workspace=ws)
    assert eta.attn_get_status(ws) == eta.ATTN_DEVERR_PAGE
    live = torch.zeros(cache.k.shape[0], 16, dtype=torch.bool)
    for b, p in ((0, list(range(16)) + list(range(32, 40))), (1, list(range(20)))):
        for x in p:
            live[int(cache.block_table[b, x // 16]), x % 16] = True
    assert torch.equal(bits(cache.k)[~live], before[~live])
    out = [torch.full((2, 2, 48, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    eta.attn_cache_read(cache, k=out[0], v=out[1], workspace=ws)
    assert eta.attn_get_status(ws) == eta.ATTN_DEVERR_PAGE
    assert (out[0][0, :, 16:32] == 9).all() and (out[0][0, :, 40:] == 9).all()
    assert torch.equal(out[0][0, :, 32:40].transpose(0, 1), k[32:40])
    # more new tokens than positions: the ones in front of position 0 go nowhere
    cache, _, _ = make_cache([3, 20], 16, 2, 128, 128, torch.bfloat16, seed=2)
    eta.attn_cache_write(k[:9], k[:9], cache, cu_of([5, 4]), workspace=ws)
    assert eta.attn_get_status(ws) == eta.ATTN_DEVERR_RAGGED
    got, _ = eta.attn_cache_read(cache, 3)
    assert torch.equal(got[0].transpose(0, 1), k[2:5])
    # lengths and offsets out of range are clamped
    for lens, cu in (([-4, 20], [0, 0, 2]), ([1000, 20], [0, 0, 2]), ([3, 20], [0, -1, 2]), ([3, 20], [0, 2, 1000]),
                     ([3, 20], [2, 1, 4])):
        cache.seq_lens.copy_(torch.tensor(lens))
        eta.attn_cache_write(k[:4], k[:4], cache, torch.tensor(cu, dtype=torch.int32, device="cuda"), workspace=ws)
        assert eta.attn_get_status(ws) & eta.ATTN_DEVERR_RAGGED


# --------------------------------------------------------------- attention


ATTN = {
    # every length from one key on, pages that end inside a tile, one token each
    "decode": dict(lens=[1, 2, 15, 16, 17, 127, 128, 129, 300], new=[1] * 9, page=16, Hq=8, Hkv=2),
    "decode_mha": dict(lens=[5, 260], new=[1, 1], page=32, Hq=4, Hkv=4),
    "decode_mqa": dict(lens=[100, 33], new=[1, 1], page=64, Hq=16, Hkv=1),
    "decode_wide_group": dict(lens=[100, 33], new=[1, 1], page=64, Hq=40, Hkv=1),
    "few_tokens": dict(lens=[70, 4, 260, 9], new=[3, 4, 2, 0], page=16, Hq=12, Hkv=4),
    "odd_group": dict(lens=[150, 40], new=[30, 40], page=16, Hq=9, Hkv=3),
    "chunk": dict(lens=[300, 129, 64], new=[130, 129, 1], page=64, Hq=8, Hkv=2),
    "chunk_page_128": dict(lens=[400], new=[257], page=128, Hq=4, Hkv=4),
    "page_48": dict(lens=[400, 20], new=[5, 20], page=48, Hq=4, Hkv=2),
    "page_256": dict(lens=[600, 20], new=[70, 2], page=256, Hq=4, Hkv=2),
    "page_7": dict(lens=[60, 20], new=[5, 20], page=7, Hq=4, Hkv=2),
    "page_1": dict(lens=[9, 3], new=[2, 1], page=1, Hq=4, Hkv=2),
    "widths": dict(lens=[60, 20], new=[5, 20], page=16, Hq=4, Hkv=2, d=80, dv=48),
    "wide": dict(lens=[40], new=[3], page=16, Hq=2, Hkv=1, d=576, dv=512),
}
MASKS = {
    "causal": dict(causal=True),
    "all_keys": dict(causal=False),
    "window": dict(causal=True, window=20),
    "window_first": dict(causal=True, window=33, first=5),
    "window_first_many": dict(causal=True, window=1, first=150),
    "open_window_first": dict(causal=False, window=7, first=3),
}


def allowed_of(mask, sink=None, **kw):
    return eta.AllowedSet(causal=mask["causal"], window_left=mask.get("window", 0), window_first=mask.get("first", 0),
                          sink=sink, **kw)


def one_case(kind, qd, cd, mask, *, heads_first=True, sink=False, max_q=True, seed=0):
    c = dict(dict(d=128, dv=128), **ATTN[kind])
    cache, K, V = make_cache(c["lens"], c["page"], c["Hkv"], c["d"], c["dv"], DT[cd], heads_first=heads_first,
                             seed=seed, src=DT[qd])
    q = seeded_q(sum(c["new"]), c["Hq"], c["d"], DT[qd], seed + 1)
    z = torch.randn(c["Hq"], generator=torch.Generator().manual_seed(seed)).cuda() if sink else None
    o, lse = run(q, cache, c["new"], allowed=allowed_of(mask, z), max_q=max(c["new"]) if max_q else 0)
    ref = reference(q, K, V, c["new"], c["lens"], c["d"] ** -0.5, sink=None if z is None else z.cpu(), **mask)
    check(o, lse, *ref, tensor_core=qd != "f32", cache=cd)
    return o, lse


@pytest.mark.parametrize("kind", list(ATTN))
@pytest.mark.parametrize("qd,cd", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "e4m3"), ("f16", "e4m3"),
                                   ("f32", "e4m3")])
def test_attention_types(kind, qd, cd):
    one_case(kind, qd, cd, MASKS["causal"])


@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("kind", ["decode", "few_tokens", "odd_group", "chunk", "page_7"])
@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
def test_attention_masks(kind, mask, cd):
    one_case(kind, "bf16", cd, MASKS[mask], heads_first=False, sink=mask != "causal", seed=4)


@pytest.mark.parametrize("kind", ["decode", "few_tokens", "chunk"])
def test_max_q_changes_no_set(kind):
    """Without the hint, and with a wrong one, the same tokens are attended."""
    one_case(kind, "bf16", "bf16", MASKS["causal"], max_q=False)
    c = ATTN[kind]
    cache, K, V = make_cache(c["lens"], c["page"], c["Hkv"], 128, 128, torch.bfloat16)
    q = seeded_q(sum(c["new"]), c["Hq"], 128, torch.bfloat16)
    o, lse = run(q, cache, c["new"], allowed=eta.AllowedSet(causal=True), max_q=1)
    check(o, lse, *reference(q, K, V, c["new"], c["lens"], 128 ** -0.5), tensor_core=True)


@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("new", [[5, 6, 0, 2], [8, 1, 7, 8], [9, 8, 12, 3]])  # up to 24, 32 and 48 rows a K/V head
@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
def test_several_row_blocks_of_drafted_tokens(new, mask, cd):
    lens = [70, 8, 260, 129]
    cache, K, V = make_cache(lens, 16, 2, 128, 128, DT[cd], seed=8, src=torch.bfloat16)
    q = seeded_q(sum(new), 8, 128, torch.bfloat16, 9)
    o, lse = run(q, cache, new, allowed=allowed_of(MASKS[mask]), max_q=max(new))
    check(o, lse, *reference(q, K, V, new, lens, 128 ** -0.5, **MASKS[mask]), tensor_core=True, cache=cd)


@pytest.mark.parametrize("kind,new", [("decode", 1), ("few_tokens", 3), ("chunk", 60)])
@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
def test_rows_outside_every_sequence_and_strides(kind, new, cd):
    """Rows in front of the first sequence and behind the last stay as they
    were; q, o and lse are strided views; cu_q does not start at 0."""
    lens = [max(L, new) for L in ATTN[kind]["lens"]]
    B, Hkv, Hq = len(lens), 2, 8
    cache, K, V = make_cache(lens, 16, Hkv, 128, 128, DT[cd], seed=9)
    rows = B * new + 5
    q = seeded_q(rows, 2 * Hq, 128, torch.bfloat16)[:, ::2]
    o = torch.full((Hq, rows, 136), 5.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)[..., :128]
    lse = torch.full((Hq, rows), 5.0, device="cuda").t()
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * new + 2
    ws = torch.empty(eta.attn_paged_workspace_size(q, cache), dtype=torch.uint8, device="cuda")
    eta.attn_paged_fwd(q, cache, cu, eta.AllowedSet(causal=True), out=o, lse=lse, workspace=ws, max_q=new)
    assert eta.attn_get_status(ws) == 0
    ref = reference(q[2:-3], K, V, [new] * B, lens, 128 ** -0.5)
    check(o[2:-3], lse[2:-3], *ref, tensor_core=True, cache=cd)
    for part in (o[:2], o[-3:], lse[:2], lse[-3:]):
        assert (part == 5).all()
    # without cu_q: the same number each
    o2, lse2 = run(q[2:-3], cache, allowed=eta.AllowedSet(causal=True), max_q=new)
    check(o2, lse2, *ref, tensor_core=True, cache=cd)


@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [64, 100, 128, 160, 256, 300])
def test_many_query_heads_over_one(group, cd):
    """Row blocks of two tokens, of one, of a token that fills them, and a group
    wider than a block; one new token and several."""
    new, lens = [1, 3, 5], [200, 3, 131]
    cache, K, V = make_cache(lens, 16, 1, 128, 128, DT[cd], seed=33, src=torch.bfloat16)
    q = seeded_q(sum(new), group, 128, torch.bfloat16, 34)
    mask = dict(causal=True, window=50, first=3)
    o, lse = run(q, cache, new, allowed=allowed_of(mask), max_q=max(new))
    check(o, lse, *reference(q, K, V, new, lens, 128 ** -0.5, **mask), tensor_core=True, cache=cd)


@pytest.mark.parametrize("max_q", [0, 1, 100])
def test_calls_with_nothing_to_do(max_q):
    """No tokens, no sequences, tables without pages, pools without pages."""
    a = eta.AllowedSet(causal=True)
    dt = torch.bfloat16
    cache, _, _ = make_cache([40, 20], 16, 2, 128, 128, dt, seed=2)
    q = seeded_q(4, 4, 128, dt)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    # no tokens: with cu_q and without
    for cu in (None, cu_of([0, 0])):
        o, lse = eta.attn_paged_fwd(q[:0], cache, cu, a, max_q=max_q)
        assert o.shape == (0, 4, 128) and lse.shape == (0, 4)
        eta.attn_cache_write(q[:0, :2], q[:0, :2], cache, cu, workspace=ws)
        assert eta.attn_get_status(ws) == 0
    # rows that belong to nobody: cu_q all zero, and no sequence at all
    none = eta.PagedCache(cache.k, cache.v, cache.block_table[:0], cache.seq_lens[:0])
    before = bits(cache.k)
    for c, cu in ((cache, cu_of([0, 0])), (none, cu_of([]))):
        o = torch.full((4, 4, 128), 3.0, dtype=dt, device="cuda")
        lse = torch.full((4, 4), 3.0, device="cuda")
        big = torch.full((eta.attn_paged_workspace_size(q, c, a),), 255, dtype=torch.uint8, device="cuda")
        eta.attn_paged_fwd(q, c, cu, a, max_q=max_q, out=o, lse=lse, workspace=big)
        assert eta.attn_get_status(big) == 0 and (o == 3).all() and (lse == 3).all()
        eta.attn_cache_write(q[:, :2], q[:, :2], c, cu, workspace=ws)
        assert eta.attn_get_status(ws) == 0
    assert torch.equal(bits(cache.k), before)
    assert eta.attn_cache_read(none, 5)[0].shape == (0, 2, 5, 128)
    # tables without pages: every length is past the table, every row empty
    flat = eta.PagedCache(cache.k, cache.v, cache.block_table[:, :0].contiguous(), cache.seq_lens)
    o, lse = run(q, flat, [2, 2], allowed=a, max_q=max_q, status=eta.ATTN_DEVERR_RAGGED)
    assert (o == 0).all() and (lse == -math.inf).all()
    assert eta.attn_cache_read(flat, 0)[0].shape == (2, 2, 0, 128) and eta.attn_cache_read(flat)[0].shape[2] == 0
    assert (eta.attn_cache_read(flat, 7, workspace=ws)[0] == 0).all()
    assert eta.attn_get_status(ws) == eta.ATTN_DEVERR_RAGGED
    # a pool without pages: every page number is outside it
    bare = eta.PagedCache(cache.k[:0], cache.v[:0], cache.block_table, cache.seq_lens)
    o, lse = run(q, bare, [2, 2], allowed=a, max_q=max_q, status=eta.ATTN_DEVERR_PAGE)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("fmt", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("kind", ["decode", "chunk", "page_7"])
def test_lse_formats(kind, fmt):
    c = ATTN[kind]
    cache, K, V = make_cache(c["lens"], c["page"], c["Hkv"], 128, 128, torch.float16)
    q = seeded_q(sum(c["new"]), c["Hq"], 128, torch.float16)
    z = torch.randn(c["Hq"], device="cuda")
    o, lse = run(q, cache, c["new"], allowed=eta.AllowedSet(causal=True, sink=z, lse_kv_only=fmt[0], lse_neg_log2=fmt[1]))
    o_ref, l_ref, A = reference(q, K, V, c["new"], c["lens"], 128 ** -0.5, sink=z.cpu())
    if fmt[0]:
        l_ref = reference(q, K, V, c["new"], c["lens"], 128 ** -0.5)[1]
    check(o, lse * -math.log(2) if fmt[1] else lse, o_ref, l_ref, A, tensor_core=True)


@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,new", [("decode", 1), ("few", 3), ("chunk", 140), ("any", 4)])
def test_empty_rows_and_bad_pages(kind, new, cd):
    """Sequences of length zero, tokens in front of position 0, pages outside
    the pool: empty rows are 0 and -inf (or the sink), the rest is exact."""
    page = 7 if kind == "any" else 16
    lens = [300, 2, 300]
    cache, K, V = make_cache(lens, page, 2, 128, 128, DT[cd], seed=5)
    q = seeded_q(3 * new, 4, 128, torch.bfloat16)
    bad = [1, 6]
    for p, v in zip(bad, (-1, cache.k.shape[0] + 5)):
        cache.block_table[2, p] = v
    skip = [None, None, {x for p in bad for x in range(p * page, p * page + page)}]
    cache.block_table[0] = -1
    cache.seq_lens[0] = 0
    want = eta.ATTN_DEVERR_PAGE | eta.ATTN_DEVERR_RAGGED
    for sink in (None, torch.randn(4, device="cuda")):
        o, lse = run(q, cache, [new] * 3, allowed=eta.AllowedSet(causal=True, sink=sink), max_q=new, status=want)
        z = torch.full((4,), -math.inf) if sink is None else sink.cpu()
        empty = new + max(0, new - 2)
        assert (o[:empty] == 0).all()
        assert torch.allclose(lse[:empty].cpu(), z.expand(empty, 4), rtol=2.0 ** -22, atol=0)
        t = reference(q[empty:], K[1:], V[1:], [min(new, 2), new], [2, 300], 128 ** -0.5,
                      sink=None if sink is None else sink.cpu(), skip=skip[1:])
        check(o[empty:], lse[empty:], *t, tensor_core=True, cache=cd)


@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (9, 3)])
@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
def test_many_row_blocks_without_keys(Hq, Hkv, cd):
    """Sequences of length 0 that bring thousands of tokens: every CTA walks
    several row blocks without a key, between blocks of a sequence that has
    keys. All are reported, none delays or disturbs the others."""
    new, lens = [16384, 600, 8192], [0, 900, 0]
    cache, K, V = make_cache(lens, 16, Hkv, 128, 128, DT[cd], seed=15, src=torch.bfloat16)
    q = seeded_q(sum(new), Hq, 128, torch.bfloat16, 16)
    a = eta.AllowedSet(causal=True)
    o, lse = run(q, cache, new, allowed=a, max_q=max(new), status=eta.ATTN_DEVERR_RAGGED)
    at = slice(new[0], new[0] + new[1])
    check(o[at], lse[at], *reference(q[at], K[1:2], V[1:2], new[1:2], lens[1:2], 128 ** -0.5), tensor_core=True, cache=cd)
    for part in (slice(0, new[0]), slice(new[0] + new[1], None)):
        assert (o[part] == 0).all() and (lse[part] == -math.inf).all()
    o2, lse2 = run(q, cache, new, allowed=a, max_q=max(new), status=eta.ATTN_DEVERR_RAGGED)
    assert torch.equal(bits(o), bits(o2)) and torch.equal(bits(lse), bits(lse2))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kind,new", [("decode", 1), ("few", 4), ("chunk", 150), ("any", 4)])
def test_masked_rows_hold_anything(kind, new, value):
    """NaN and infinities in K and V rows that a query does not see do not
    reach it; one that sees them is not finite."""
    page = 7 if kind == "any" else 16
    lens = [290, 290]
    cache, K, V = make_cache(lens, page, 2, 128, 128, torch.bfloat16, seed=6)
    hit = [100, 289, 270, 288]  # out of the window for all or some queries; after some queries
    for j in hit:
        pg, off = int(cache.block_table[0, j // page]), j % page
        (cache.v if value != value or j % 2 == 0 else cache.k)[pg, off, 1, 3] = value
        cache.v[pg, off, 1, 70] = value
        V[0][j, 1, 70] = value
    q = seeded_q(2 * new, 4, 128, torch.bfloat16)
    mask = dict(causal=True, window=16, first=3)
    o, lse = run(q, cache, [new, new], allowed=allowed_of(mask), max_q=new)
    ok = torch.zeros(2 * new, 4, dtype=torch.bool)
    for i in range(new):
        p = 290 - new + i
        ok[i] = not any(p - 16 < j <= p for j in hit)
    ok[new:] = True
    ok[:, :2] = True  # the first K/V head is clean
    clean, Kc, Vc = make_cache(lens, page, 2, 128, 128, torch.bfloat16, seed=6)
    ref = reference(q, Kc, Vc, [new, new], lens, 128 ** -0.5, **mask)
    check(o[ok.cuda()], lse[ok.cuda()], *[r[ok] for r in ref], tensor_core=True)
    assert not torch.isfinite(o[~ok.cuda()][:, 70]).any()


@pytest.mark.parametrize("kind,new", [("decode", 1), ("few", 4), ("chunk", 150), ("any", 4)])
def test_masked_e4m3_rows_hold_anything(kind, new):
    """NaN codes, and scales that are not finite, in e4m3 rows that a query does
    not see."""
    page = 7 if kind == "any" else 16
    L = 290
    cache, K, V = make_cache([L], page, 2, 128, 128, E4M3, seed=6, src=torch.bfloat16)
    hit = [100, 289, 270, 288]
    for j in hit:
        pg, off = int(cache.block_table[0, j // page]), j % page
        cache.v.view(torch.uint8)[pg, off, 1, 70] = 0x7F
        if j == 270:
            cache.v_scale[pg, off, 1] = math.inf
        if j == 100:
            cache.k_scale[pg, off, 1] = math.nan
    q = seeded_q(new, 4, 128, torch.bfloat16)
    mask = dict(causal=True, window=16, first=3)
    o, lse = run(q, cache, [new], allowed=allowed_of(mask), max_q=new)
    ok = torch.tensor([[h < 2 or not any(p - 16 < j <= p for j in hit) for h in range(4)]
                       for p in range(L - new, L)])
    ref = reference(q, K, V, [new], [L], 128 ** -0.5, **mask)
    check(o[ok.cuda()], lse[ok.cuda()], *[r[ok] for r in ref], tensor_core=True, cache=E4M3)
    assert not torch.isfinite(o[~ok.cuda()][:, 70]).any()


def causal_reference(q, K, V, new, lens, scale):
    """`reference` of causal rows that all see a key, whole matrices at a time."""
    o, lse, A = [], [], []
    for b, at in enumerate(cu_of(new, "cpu")[:-1].tolist()):
        n, L, g = new[b], lens[b], q.shape[1] // K[b].shape[1]
        k, v = (x[b].transpose(0, 1).repeat_interleave(g, 0) for x in (K, V))  # [Hq, L, d]
        s = q[at:at + n].double().cpu().transpose(0, 1) @ k.transpose(1, 2) * scale
        s = s.masked_fill(torch.arange(L) > torch.arange(L - n, L)[:, None], -math.inf)
        m = torch.logsumexp(s, -1)
        p = torch.exp(s - m[..., None])
        for x, y in ((o, p @ v), (A, p @ v.abs()), (lse, m)):
            x.append(y.transpose(0, 1))
    return torch.cat(o), torch.cat(lse), torch.cat(A)


@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (12, 4)])
@pytest.mark.parametrize("cd", ["bf16", "f16", "e4m3"])
def test_non_finite_values_where_a_cta_walks_many_blocks(Hq, Hkv, cd):
    """Hundreds of row blocks, of more and of less than 128 rows and many of one
    key tile, with NaN and infinities in the last (partly visible) tiles and in
    front of the new tokens of every third sequence: every row that sees one is
    not finite, every other row is within its bound."""
    g = torch.Generator().manual_seed(17)
    B = 100
    new = [int(x) for x in torch.randint(1, 60, (B,), generator=g)]
    lens = [n + int(x) for n, x in zip(new, torch.randint(0, 130, (B,), generator=g))]
    for b, (n, more) in enumerate([(300, 400), (140, 0), (257, 900), (131, 129)]):
        new[30 * b], lens[30 * b] = n, n + more
    qd = torch.float16 if cd == "f16" else torch.bfloat16
    cache, K, V = make_cache(lens, 16, Hkv, 128, 128, DT[cd], seed=18, src=qd)
    q = seeded_q(sum(new), Hq, 128, qd, 19)
    head, group = Hkv - 1, Hq // Hkv
    ok, at = torch.ones(sum(new), Hq, dtype=torch.bool), 0
    for b, (n, L) in enumerate(zip(new, lens)):
        if b % 3 == 0:
            for i, j in enumerate({L - 1, max(0, L - 7), max(0, L - n - 3)} if b % 2 else {L - 1 - n // 2}):
                pg, off = int(cache.block_table[b, j // 16]), j % 16
                if cd != "e4m3":
                    cache.v[pg, off, head, 70] = (math.nan, math.inf, -math.inf)[(i + b) % 3]
                elif (i + b) % 2:
                    cache.v.view(torch.uint8)[pg, off, head, 70] = 0xFF
                else:
                    cache.v_scale[pg, off, head] = math.inf
                first = max(0, j - (L - n))  # the first new token that sees key j
                ok[at + first:at + n, head * group:] = False
        at += n
    o, lse = run(q, cache, new, allowed=eta.AllowedSet(causal=True), max_q=max(new))
    ref = causal_reference(q, K, V, new, lens, 128 ** -0.5)
    check(o[ok.cuda()], lse[ok.cuda()], *[r[ok] for r in ref], tensor_core=True, cache=cd)
    assert not torch.isfinite(o[~ok.cuda()][:, 70]).any()


@pytest.mark.parametrize("kind,most", [("decode", 1), ("chunk", 40)])
@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
def test_thousands_of_sequences(kind, most, cd):
    """More sequences than a block has threads and than the plan's lists in
    shared memory hold; every fifth brings no token."""
    g = torch.Generator().manual_seed(30)
    B = 2500
    new = [0 if b % 5 == 3 else int(x) for b, x in enumerate(torch.randint(1, most + 1, (B,), generator=g))]
    lens = [n + int(x) for n, x in zip(new, torch.randint(1, 70, (B,), generator=g))]
    cache, K, V = make_cache(lens, 16, 1, 128, 128, DT[cd], seed=31, src=torch.bfloat16)
    q = seeded_q(sum(new), 2, 128, torch.bfloat16, 32)
    o, lse = run(q, cache, new, allowed=eta.AllowedSet(causal=True), max_q=most)
    check(o, lse, *causal_reference(q, K, V, new, lens, 128 ** -0.5), tensor_core=True, cache=cd)


@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
def test_one_nan_behind_a_million_keys(cd):
    """A row block that walks 2^20 keys by itself, with one NaN in the last
    page: only the rows that see it are NaN, and no wait runs out meanwhile.
    The cache is eight pages, each listed many times, and a last one. Beside
    check's bounds, fp32 sums over 2^16 steps of 16 keys: 2^-8 relative to A,
    and 2^-8 for the LSE."""
    heads = torch.cuda.get_device_properties(0).multi_processor_count  # an item for every CTA
    page, n, times, new = 128, 8, 1024, 40
    lens, last = [n * times * page], n
    cache, K, V = make_cache([(n + 1) * page], page, heads, 128, 128, DT[cd], seed=21, src=torch.bfloat16)
    order = cache.block_table[0, :n + 1].clone()
    cache.block_table = torch.cat([order[:n].repeat(times)[:-1], order[n:]])[None].contiguous()
    cache.seq_lens.fill_(lens[0])
    pg = int(order[last])
    hit, see = page - 30, 10  # visible to the last 30 of the 40 new tokens
    if cd == "e4m3":
        cache.v.view(torch.uint8)[pg, hit, 1, 70] = 0x7F
    else:
        cache.v[pg, hit, 1, 70] = math.nan
    q = seeded_q(new, heads, 128, torch.bfloat16, 22)
    o, lse = run(q, cache, [new], allowed=eta.AllowedSet(causal=True), max_q=new)
    assert torch.isnan(o[see:, 1, 70]).all()
    for h in (0, 1, heads - 1):
        k, v = K[0][:, h], V[0][:, h]
        count = torch.full((n * page,), float(times), dtype=torch.float64)
        count[-page:] -= 1  # its last listing is the last page
        count = torch.cat([count, torch.ones(page, dtype=torch.float64)]).expand(new, -1).clone()
        count[:, -page:] = (torch.arange(page) <= page - new + torch.arange(new)[:, None]).double()
        x = q[:, h].double().cpu() @ k.T * 128 ** -0.5 + torch.log(count)
        want_lse = torch.logsumexp(x, 1)
        p = torch.exp(x - want_lse[:, None])
        A = p @ v.abs()
        ok = torch.ones(new, 128, dtype=torch.bool)
        if h == 1:
            ok[see:, 70] = False
        err = (o[:, h].double().cpu() - p @ v).abs()
        assert (err <= 2.0 ** -8 * (p @ v).abs() + (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -12) * A)[ok].all()
        assert ((lse[:, h].double().cpu() - want_lse).abs() <= 2.0 ** -8).all()


@pytest.mark.parametrize("new,kind", [(1, "decode"), (20, "chunk")])
@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
def test_one_long_sequence_is_joined_from_many_shares(new, kind, cd):
    """One K/V head and one row block: its keys fall to dozens of CTAs."""
    L = 20011
    cache, K, V = make_cache([L], 64, 1, 128, 128, DT[cd], seed=12, src=torch.bfloat16)
    q = seeded_q(new, 4, 128, torch.bfloat16)
    o, lse = run(q, cache, [new], allowed=eta.AllowedSet(causal=True), max_q=new)
    check(o, lse, *reference(q, K, V, [new], [L], 128 ** -0.5), tensor_core=True, cache=cd)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_e4m3_with_other_score_factors(kind, scale):
    """Negative and zero factors, and one that spreads the scores; row scales
    that differ by up to 2^12 within a tile, for K and V."""
    c = ATTN[kind]
    cache, K, V = make_cache(c["lens"], c["page"], c["Hkv"], 128, 128, E4M3, seed=3, src=torch.bfloat16)
    g = torch.Generator().manual_seed(9)
    for b, L in enumerate(c["lens"]):
        pos = torch.arange(L)
        at = cache.block_table[b].long().cpu()[pos // c["page"]], pos % c["page"]
        for sc, dense, most in ((cache.k_scale, K, 3), (cache.v_scale, V, 12)):
            f = 2.0 ** -torch.randint(0, most + 1, (L, c["Hkv"]), generator=g).double()
            sc[at[0].cuda(), at[1].cuda()] *= f.float().cuda()
            dense[b] = dense[b] * f[..., None]
    q = seeded_q(sum(c["new"]), c["Hq"], 128, torch.bfloat16)
    o, lse = run(q, cache, c["new"], scale=scale, allowed=eta.AllowedSet(causal=True), max_q=max(c["new"]))
    o_ref, l_ref, A = reference(q, K, V, c["new"], c["lens"], scale)
    # Probabilities below fp16's normal range (2^-14 of the row's largest times
    # scale) are rounded to steps of 2^-24: with N keys, another N 2^-25 of the
    # largest value row.
    top = torch.stack([v.abs().amax() for v in V]).max() * max(c["lens"]) * 2.0 ** -25
    check(o, lse, o_ref, l_ref, A + top * 2.0 ** 9, tensor_core=True, cache=E4M3)


@pytest.mark.parametrize("other", [2.0 ** 20, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("kind,new", [("decode", 1), ("few", 4), ("chunk", 150), ("any", 4)])
def test_one_value_row_of_the_largest_scale(kind, new, other):
    """A value row near the end of fp32's range takes part of the probability,
    several hundred rows of scales within 2^100 of its own the rest: none of
    their shares is lost from the sum, though 2^(score - reference) is tiny."""
    page, L, big = 7 if kind == "any" else 16, 700, 333
    cache, K, V = make_cache([L], page, 1, 128, 128, E4M3, seed=27, src=torch.bfloat16)
    pos = torch.arange(L)
    at = cache.block_table[0].long().cpu()[pos // page].cuda(), (pos % page).cuda()
    k = torch.zeros(L, 1, 128)
    k[big, 0, 0] = 1
    cache.k.view(torch.uint8)[at[0], at[1]] = k.to(E4M3).view(torch.uint8).cuda()
    cache.k_scale[at] = 1.0
    V[0] = V[0] / cache.v_scale[at].double().cpu()[..., None]  # the codes
    scales = torch.full((L, 1), other)
    scales[big] = 2.0 ** 118
    cache.v_scale[at] = scales.cuda()
    q = torch.zeros(new, 4, 128, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 9  # 2^9 times another key's share, of which there are 2^9.4
    o, lse = run(q, cache, [new], allowed=eta.AllowedSet(causal=True), scale=math.log(2), max_q=new)
    K, V = [k.double()], [V[0] * scales.double()[..., None]]
    check(o, lse, *reference(q, K, V, [new], [L], math.log(2)), tensor_core=True, cache=E4M3)


@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_unaligned_tensors(kind, cd):
    """Rows that start off the 16-byte grid, in q, o or the pool, take the row
    kernels and give the same answers."""
    c = ATTN[kind]
    cache, K, V = make_cache(c["lens"], c["page"], c["Hkv"], 128, 128, DT[cd], src=torch.bfloat16)
    rows = sum(c["new"])
    q = seeded_q(rows, c["Hq"], 129, torch.bfloat16)[..., 1:]
    ref = reference(q, K, V, c["new"], c["lens"], 128 ** -0.5)
    o, lse = run(q, cache, c["new"], allowed=eta.AllowedSet(causal=True), max_q=max(c["new"]))
    check(o, lse, *ref, tensor_core=False)
    out = torch.empty(rows, c["Hq"], 131, dtype=torch.bfloat16, device="cuda")[..., 2:130]
    run(q, cache, c["new"], allowed=eta.AllowedSet(causal=True), max_q=max(c["new"]), out=out)
    check(out, lse, *ref, tensor_core=False)


def test_read_into_one_given_tensor():
    cache, K, V = make_cache([33], 16, 2, 128, 128, torch.bfloat16)
    k = torch.zeros(1, 2, 40, 128, dtype=torch.bfloat16, device="cuda")
    got_k, got_v = eta.attn_cache_read(cache, k=k)
    assert got_k is k and got_v.shape == k.shape
    assert torch.equal(got_v[0, :, :33].transpose(0, 1).double().cpu(), V[0]) and (got_v[0, :, 33:] == 0).all()


def test_read_into_as_many_rows_as_a_tensor_can_have():
    """2^31 - 1 rows a head, of which the table holds 48."""
    cache, K, _ = make_cache([33], 16, 1, 8, 8, torch.bfloat16)
    cache.v = cache.k
    T = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 34 GB of device memory")
    x = torch.empty(1, 1, T, 8, dtype=torch.bfloat16, device="cuda")
    x[:, :, :64] = 7
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    eta.attn_cache_read(cache, k=x, v=x, workspace=ws)
    assert eta.attn_get_status(ws) == 0
    assert torch.equal(x[0, 0, :33].double().cpu(), K[0][:, 0]) and (x[0, 0, 33:64] == 7).all()
    del x
    torch.cuda.empty_cache()


def test_nan_scores_make_the_row_nan():
    for new, page in ((1, 16), (150, 16), (2, 7)):
        cache, _, _ = make_cache([300], page, 2, 128, 128, torch.bfloat16)
        q = seeded_q(new, 4, 128, torch.bfloat16)
        q[0] = math.nan
        o, lse = run(q, cache, [new], allowed=eta.AllowedSet(causal=True), max_q=new)
        assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
        assert torch.isfinite(o[1:]).all() and torch.isfinite(lse[1:]).all()


@pytest.mark.parametrize("cd", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind,new,L,B", [("decode", 1, 300, 1), ("few", 4, 300, 1), ("any", 4, 300, 1),
                                          ("shares", 150, 3000, 1), ("whole", 40, 200, 300)])
def test_empty_rows_stay_empty_over_values_that_are_not_finite(kind, new, L, B, cd):
    """Scores of -inf throughout, and NaN in values of the last, partly visible
    tile: the rows are 0 and -inf, whether one CTA walks a row block or several."""
    page = 7 if kind == "any" else 16
    cache, _, _ = make_cache([L], page, 1, 128, 128, DT[cd], seed=25, src=torch.bfloat16)
    pos = torch.arange(L)
    cache.block_table, cache.seq_lens = cache.block_table.repeat(B, 1), cache.seq_lens.repeat(B)
    at = cache.block_table[0].long().cpu()[pos // page].cuda(), (pos % page).cuda()
    if cd == "e4m3":
        row = torch.zeros(128)
        row[0] = -1
        cache.k.view(torch.uint8)[at[0], at[1]] = row.to(E4M3).view(torch.uint8).cuda()
        cache.k_scale[at] = math.inf
        cache.v.view(torch.uint8)[at[0][-2], at[1][-2], 0, 70] = 0x7F
    else:
        cache.k[at[0], at[1], :, 0] = -math.inf
        cache.v[at[0][-2], at[1][-2], 0, 70] = math.nan
    q = seeded_q(B * new, 4, 128, torch.bfloat16, 26)
    q[..., 0] = 1
    o, lse = run(q, cache, [new] * B, allowed=eta.AllowedSet(causal=True), max_q=new)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("cd", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("kind,new", [("decode", 1), ("few", 4), ("chunk", 150), ("any", 4)])
def test_rows_whose_scores_are_all_minus_infinity(kind, new, cd, sink):
    """They count as empty, over tiles that are seen whole and in part alike;
    those of the other sequence and the other K/V head keep their results."""
    page = 7 if kind == "any" else 16
    lens, head = [600, 290], 1
    qd = torch.float16 if cd == "f16" else torch.bfloat16
    cache, K, V = make_cache(lens, page, 2, 128, 128, DT[cd], seed=23, src=qd)
    pos = torch.arange(lens[0])
    at = cache.block_table[0].long().cpu()[pos // page].cuda(), (pos % page).cuda()
    if cd == "e4m3":  # every score is negative and its scale infinite
        row = torch.zeros(128)
        row[0] = -1
        cache.k.view(torch.uint8)[at[0], at[1], head] = row.to(E4M3).view(torch.uint8).cuda()
        cache.k_scale[at[0], at[1], head] = math.inf
    else:
        cache.k[at[0], at[1], head, 0] = -math.inf
    q = seeded_q(2 * new, 4, 128, qd, 24)
    q[..., 0] = 1
    z = torch.randn(4, device="cuda") if sink else None
    o, lse = run(q, cache, [new, new], allowed=eta.AllowedSet(causal=True, sink=z), max_q=new)
    assert (o[:new, 2:] == 0).all()
    empty = torch.full((2,), -math.inf) if z is None else z[2:].cpu()
    assert torch.allclose(lse[:new, 2:].cpu(), empty.expand(new, 2), rtol=2.0 ** -22, atol=0)
    ref = reference(q, K, V, [new, new], lens, 128 ** -0.5, sink=None if z is None else z.cpu())
    ok = torch.ones(2 * new, 4, dtype=torch.bool)
    ok[:new, 2:] = False
    check(o[ok.cuda()], lse[ok.cuda()], *[r[ok] for r in ref], tensor_core=True, cache=cd)


@pytest.mark.parametrize("kind,new", [("decode", 1), ("chunk", 140)])
def test_scores_of_large_spread(kind, new):
    """Scores that grow along the keys move the running maximum in every tile;
    scales of both signs."""
    lens = [600, 350]
    cache, K, V = make_cache(lens, 16, 2, 128, 128, torch.bfloat16, seed=8)
    cache.k.zero_()
    for b, L in enumerate(lens):
        pos = torch.arange(L)
        r = torch.zeros(L, 2, 128)
        r[..., 0] = (pos.float() / 4).to(torch.bfloat16).float()[:, None]
        K[b] = r.double()
        cache.k[cache.block_table[b].long().cpu()[pos // 16].cuda(), (pos % 16).cuda()] = r.to(torch.bfloat16).cuda()
    q = torch.zeros(2 * new, 4, 128, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    for scale in (1.0, -1.0):
        o, lse = run(q, cache, [new, new], scale=scale, allowed=eta.AllowedSet(causal=True), max_q=new)
        check(o, lse, *reference(q, K, V, [new, new], lens, scale), tensor_core=True)


# ----------------------------------------------------- streams, graphs, runs


def test_repeats_bitwise_and_on_other_streams():
    for new in (1, 5, 200):
        lens = [700, 301, 256]
        cache, _, _ = make_cache(lens, 16, 2, 128, 128, torch.bfloat16)
        q = seeded_q(3 * new, 8, 128, torch.bfloat16)
        a = eta.AllowedSet(causal=True)
        o, lse = run(q, cache, [new] * 3, allowed=a, max_q=new)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = []
        for s in streams:  # three at once, workspaces of their own
            got.append(eta.attn_paged_fwd(q, cache, cu_of([new] * 3), a, max_q=new, stream=s))
        torch.cuda.synchronize()
        for o2, lse2 in got:
            assert torch.equal(bits(o), bits(o2)) and torch.equal(bits(lse), bits(lse2))


@pytest.mark.parametrize("new", [1, 3, 140])
def test_captured_step_replays_with_new_lengths(new):
    """Write and attention captured once; two graphs share one workspace; the
    lengths, tables and tokens change between replays."""
    page, Hq, Hkv, B = 16, 8, 2, 2
    cache, K, V = make_cache([400, 300], page, Hkv, 128, 128, E4M3, src=torch.bfloat16)
    nk, nv = (torch.zeros(B * new, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B * new, Hq, 128, dtype=torch.bfloat16, device="cuda")
    a = eta.AllowedSet(causal=True, window_left=200, window_first=4)
    ws = torch.empty(eta.attn_paged_workspace_size(q, cache, a), dtype=torch.uint8, device="cuda")
    out = [(torch.empty_like(q), torch.empty(B * new, Hq, device="cuda")) for _ in range(2)]

    def step(i):
        eta.attn_cache_write(nk, nv, cache)
        eta.attn_paged_fwd(q, cache, None, a, out=out[i][0], lse=out[i][1], workspace=ws, max_q=new)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(0)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(i)
        graphs.append(g)
    for t, (g, lens) in enumerate(zip(graphs * 2, ([400, 300], [150, 299], [new, 211], [399, 160]))):
        cache.seq_lens.copy_(torch.tensor(lens))
        for x, seed in ((nk, 50 + t), (nv, 60 + t), (q, 70 + t)):
            x.copy_(seeded_q(*x.shape, torch.bfloat16, seed))
        g.replay()
        torch.cuda.synchronize()
        for b in range(B):
            for x, dense in ((nk, K), (nv, V)):
                c, sc = quantise(x[b * new:(b + 1) * new].cpu())
                dense[b][lens[b] - new:lens[b]] = c.double() * sc.double()[..., None]
        ref = reference(q, [k[:L] for k, L in zip(K, lens)], [v[:L] for v, L in zip(V, lens)], [new] * B, lens,
                        128 ** -0.5, window=200, first=4)
        check(*out[t % 2], *ref, tensor_core=True, cache=E4M3)
    assert eta.attn_get_status(ws) == 0


@pytest.mark.parametrize("store", ["bf16", "e4m3"])
def test_serving_run(store):
    """A prompt in chunks, then single tokens, each step written and attended,
    against one dense forward pass over the rows read back at the end."""
    B, Hq, Hkv, d, page = 2, 8, 2, 128, 16
    total = [220, 90]
    steps = [[100, 80], [90, 0], [27, 7]] + [[1, 1]] * 3
    cache = eta.PagedCache.allocate(24, page, Hkv, d, B, 14, dtype=DT[store])
    cache.block_table.copy_(torch.randperm(24, generator=torch.Generator().manual_seed(1))[:28 - 4].to(torch.int32)
                            .repeat(2)[:28].reshape(2, 14).cuda())
    cache.block_table[0] = torch.arange(0, 14)
    cache.block_table[1] = torch.cat([torch.arange(14, 24), torch.arange(4) * 0 - 1])
    g = torch.Generator().manual_seed(2)
    qkv = [[torch.randn(L, h, d, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv)] for L in total]
    a = eta.AllowedSet(causal=True, window_left=64, window_first=4)
    done, outs = [0, 0], [[], []]
    for new in steps:
        cat = [torch.cat([qkv[b][i][done[b]:done[b] + new[b]] for b in range(B)]) for i in range(3)]
        cache.seq_lens.add_(torch.tensor(new, dtype=torch.int32, device="cuda"))
        cu = cu_of(new)
        eta.attn_cache_write(cat[1], cat[2], cache, cu)
        o, _ = eta.attn_paged_fwd(cat[0], cache, cu, a, max_q=max(new))
        at = 0
        for b in range(B):
            outs[b].append(o[at:at + new[b]])
            at += new[b]
            done[b] += new[b]
    assert done == total
    k, v = eta.attn_cache_read(cache, max(total), dtype=torch.float32 if store == "e4m3" else None)
    for b in range(B):
        L = total[b]
        q = qkv[b][0].transpose(0, 1)[None]
        kk, vv = k[b:b + 1, :, :L].float(), v[b:b + 1, :, :L].float()
        want, lse = eta.attn_fwd(q.float(), kk.contiguous(), vv.contiguous(), a)
        A, _ = eta.attn_fwd(q.float(), kk.contiguous(), vv.abs().contiguous(), a)
        got = torch.cat(outs[b])
        # the float32 dense pass stands 1e-5 from the definition (its own tests)
        eps = 2.0 ** -8
        want, A = want[0].transpose(0, 1), A[0].transpose(0, 1)
        assert ((got.float() - want).abs() <= eps * want.abs() + (eps + 2.0 ** -12) * A + 2e-5).all()
