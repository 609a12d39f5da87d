"""What is measured of the paged-cache operators and of the sliding window with first tokens.

Four operators: writing new tokens into a paged K/V cache (as they are, or quantised to e4m3 with one fp32 scale per
cached row), reading a cache back into the dense [B, Hkv, T, d] layout, attention of a ragged chunk of new tokens over
the cache, and the forward and reverse pass of a sliding window whose first keys stay visible.

`own` False computes them from elementary torch operations in fp32; `own` True calls the library.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": E4M3}
D = 128


def listed():
    return [
        # One new token of each of 64 sequences goes into the cache: a step of batched decoding.
        dict(name="write_step_b64_bf16", op="write", B=64, new=1, ctx=2048, ragged=True, page=16, Hkv=8, src="bf16",
             store="bf16", heads_first=True),
        # A long prompt's 8192 tokens, quantised as they are written.
        dict(name="write_prompt_8k_e4m3", op="write", B=1, new=8192, ctx=8192, ragged=False, page=64, Hkv=8, src="bf16",
             store="e4m3", heads_first=True),
        # One short cached prompt read back, for instance to score it with the dense reverse pass.
        dict(name="read_1k_f16", op="read", B=1, ctx=1000, ragged=False, page=16, Hkv=8, src="f16", store="f16",
             heads_first=False),
        # A batch of quantised, ragged caches read back.
        dict(name="read_b8_4k_e4m3", op="read", B=8, ctx=4096, ragged=True, page=64, Hkv=8, src="bf16", store="e4m3",
             heads_first=True),
        # The latency of one user's decoding step.
        dict(name="decode_b1_2k_bf16", op="paged", B=1, new=1, ctx=2000, ragged=False, page=16, Hq=32, Hkv=8,
             src="bf16", store="bf16", heads_first=True, window=0, first=0, sink=False),
        # A full batch's decoding step over quantised caches of different lengths.
        dict(name="decode_b64_8k_e4m3", op="paged", B=64, new=1, ctx=8192, ragged=True, page=64, Hq=32, Hkv=8,
             src="bf16", store="e4m3", heads_first=True, window=0, first=0, sink=False),
        # Decoding with a window, four first tokens and a sink logit: most of each long cache is not read.
        dict(name="decode_b32_16k_window_first", op="paged", B=32, new=1, ctx=16384, ragged=True, page=32, Hq=32,
             Hkv=8, src="f16", store="f16", heads_first=False, window=1024, first=4, sink=True),
        # A scheduler's mixed step: eight sequences bring 1 to 256 new tokens each.
        dict(name="chunk_b8_mixed_bf16", op="paged", B=8, new=256, ctx=4096, ragged=True, page=64, Hq=32, Hkv=8,
             src="bf16", store="bf16", heads_first=True, window=0, first=0, sink=False),
        # The last chunk of a 16384-token prompt, bf16 and quantised.
        dict(name="chunk_2k_of_16k_bf16", op="paged", B=1, new=2048, ctx=16384, ragged=False, page=64, Hq=32, Hkv=8,
             src="bf16", store="bf16", heads_first=True, window=0, first=0, sink=False),
        dict(name="chunk_2k_of_16k_e4m3", op="paged", B=1, new=2048, ctx=16384, ragged=False, page=128, Hq=32, Hkv=8,
             src="bf16", store="e4m3", heads_first=True, window=0, first=0, sink=False),
        # Training steps with a window and visible first tokens: a short odd length with grouped heads, and the
        # 8192-token length of the library's own window workload.
        dict(name="window_first_1k_gqa", op="train", B=2, T=1000, Hq=16, Hkv=4, src="bf16", window=256, first=4,
             sink=True),
        dict(name="window_first_8k", op="train", B=1, T=8192, Hq=32, Hkv=32, src="bf16", window=1024, first=4,
             sink=False),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def one():
        op = rng.choice(["write", "read", "paged", "paged", "train"])
        src = rng.choice(["bf16", "bf16", "f16"])
        store = rng.choice([src, "e4m3"])
        page = rng.choice([16, 32, 64, 128])
        heads_first = rng.random() < 0.6
        if op == "write":
            new = rng.choice([1, logint(2, 8192)])
            return dict(op=op, B=logint(1, 64), new=new, ctx=new + logint(1, 4096), ragged=rng.random() < 0.7, page=page,
                        Hkv=rng.choice([1, 2, 4, 8, 16]), src=src, store=store, heads_first=heads_first)
        if op == "read":
            return dict(op=op, B=logint(1, 32), ctx=logint(60, 16384), ragged=rng.random() < 0.7, page=page,
                        Hkv=rng.choice([1, 2, 4, 8, 16]), src=src, store=store, heads_first=heads_first)
        window, first = rng.choice([(0, 0), (logint(64, 2048), 0), (logint(64, 2048), rng.randint(1, 64))])
        if op == "paged":
            Hq, Hkv = rng.choice([(32, 8), (32, 4), (32, 32), (16, 16), (16, 2), (12, 4), (8, 1)])
            new = rng.choice([1, 1, logint(2, 16), logint(16, 2048)])
            return dict(op=op, B=logint(1, 64), new=new, ctx=new + logint(30, 16384), ragged=rng.random() < 0.7,
                        page=page, Hq=Hq, Hkv=Hkv, src=src, store=store, heads_first=heads_first, window=window,
                        first=first, sink=rng.random() < 0.3)
        Hq, Hkv = rng.choice([(32, 32), (32, 8), (16, 16), (16, 4), (8, 8), (8, 1)])
        return dict(op=op, B=rng.choice([1, 1, 2, 4]), T=logint(300, 8192), Hq=Hq, Hkv=Hkv, src=src,
                    window=logint(64, 2048), first=rng.randint(1, 64), sink=rng.random() < 0.3)

    most = max(_cost(c) for c in listed())
    while True:
        c = one()
        if _cost(c) > most:
            continue
        if c["op"] == "paged" and c["B"] * c["Hq"] * c["new"] * c["ctx"] > 32 * 2048 * 16384:
            continue  # the plain form's scores would not fit
        if c["op"] == "paged" and c["B"] * c["Hkv"] * c["ctx"] > 64 * 8 * 16384:
            continue
        if c["op"] == "train" and c["B"] * c["Hq"] * c["T"] ** 2 > 32 * 8192 ** 2:
            continue
        if c["op"] in ("write", "read") and c["B"] * c["ctx"] * c["Hkv"] > 16 * 16384 * 8:
            continue
        return c


# ---------------------------------------------------------------- sizes


def _lengths(case):
    """Per sequence: the new tokens and the cached length (new ones included), from the sizes alone."""
    B, ctx, new = case["B"], case["ctx"], case.get("new", 1)
    r = np.random.RandomState(B * 7919 + ctx * 31 + new)
    n = np.full(B, new, np.int64)
    L = np.full(B, ctx, np.int64)
    if case["ragged"]:
        if new > 1:
            n = r.randint(1, new + 1, B)
            n[r.randint(B)] = new
        L = r.randint(max(1, ctx // 4), ctx + 1, B)
        L[r.randint(B)] = ctx
        L = np.maximum(L, n)
    return n, L


def _pairs(n, L, window, first):
    """Allowed (query, key) pairs of n queries at the end of L keys: causal, window, first tokens."""
    p = np.arange(L - n, L, dtype=np.int64)
    if not window:
        return int((p + 1).sum()), int(L)
    lo = np.maximum(0, p - window + 1)
    kept = np.minimum(first, lo)
    seen = L - lo[0] + kept[-1 if lo[-1] < first else 0] if len(p) else 0
    return int((p - lo + 1 + kept).sum()), int(min(L, seen))


def work(case):
    el = 2
    if case["op"] == "train":
        pairs, _ = _pairs(case["T"], case["T"], case["window"], case["first"])
        q, kv = case["B"] * case["Hq"] * case["T"] * D, case["B"] * case["Hkv"] * case["T"] * D
        return {"bytes": el * (4 * q + 4 * kv) + 8 * q // D, "flops": 14 * D * pairs * case["B"] * case["Hq"]}
    n, L = _lengths(case)
    store = D * el if case["store"] != "e4m3" else D + 4  # bytes of one cached row
    if case["op"] == "write":
        rows = 2 * int(n.sum()) * case["Hkv"]
        return {"bytes": rows * (D * el + store), "flops": rows * D}
    if case["op"] == "read":
        rows = 2 * int(L.sum()) * case["Hkv"]
        return {"bytes": rows * (D * el + store), "flops": rows * D}
    got = [_pairs(int(a), int(b), case["window"], case["first"]) for a, b in zip(n, L)]
    rows = 2 * sum(s for _, s in got) * case["Hkv"]
    q = int(n.sum()) * case["Hq"]
    return {"bytes": rows * store + q * (2 * D * el + 4), "flops": 4 * D * case["Hq"] * sum(p for p, _ in got)}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# --------------------------------------------------------------- inputs


def _quantised(x):
    """Rows of x as e4m3 codes and one fp32 scale each: the largest magnitude at 448, a zero row with scale 1."""
    a = x.float().abs().amax(-1)
    s = torch.where(a == 0, torch.ones_like(a), a / E4M3_MAX)
    return (x.float() / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), s


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    src = DTYPES[case["src"]]
    s = dict(case=case, op=case["op"], scale=D ** -0.5)
    if case["op"] == "train":
        B, T, Hq, Hkv = case["B"], case["T"], case["Hq"], case["Hkv"]
        s.update(q=randn(B, Hq, T, D, dtype=src), k=randn(B, Hkv, T, D, dtype=src), v=randn(B, Hkv, T, D, dtype=src),
                 do=randn(B, Hq, T, D, dtype=src), sink=randn(Hq) if case["sink"] else None)
        return s
    n, L = _lengths(case)
    B, page, Hkv = case["B"], case["page"], case["Hkv"]
    pages = -(-L // page)
    M, P = int(pages.max()), int(pages.sum()) + 3
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    at = np.concatenate([[0], np.cumsum(pages)])
    take = np.minimum(at[:-1, None] + np.arange(M)[None], P - 1)
    s["block_table"] = order[torch.from_numpy(take).to("cuda")].contiguous()
    s["seq_lens"] = torch.from_numpy(L.astype(np.int32)).to("cuda")
    s["cu_q"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to("cuda")
    s["total"], s["max_new"], s["max_len"] = int(n.sum()), int(n.max()), int(L.max())

    def pool(dtype):  # [pages, page, Hkv, d], the head's rows of a page next to each other or the token's heads
        x = randn(P, Hkv, page, D).to(dtype) if case["heads_first"] else randn(P, page, Hkv, D).to(dtype)
        return x.transpose(1, 2) if case["heads_first"] else x

    s["k"], s["v"], s["k_scale"], s["v_scale"] = pool(src), pool(src), None, None
    if case["store"] == "e4m3":
        for x in ("k", "v"):
            # quantised in the pool's own memory order
            c, sc = _quantised(s[x].transpose(1, 2) if case["heads_first"] else s[x])
            s[x], s[x + "_scale"] = (c.transpose(1, 2), sc.transpose(1, 2)) if case["heads_first"] else (c, sc)
    if case["op"] == "write":
        s["new_k"], s["new_v"] = randn(s["total"], Hkv, D, dtype=src), randn(s["total"], Hkv, D, dtype=src)
    if case["op"] == "paged":
        s["q"] = randn(s["total"], case["Hq"], D, dtype=src)
        s["sink"] = randn(case["Hq"]) if case["sink"] else None
    if case["op"] == "read":
        T = s["max_len"]
        s["out_k"] = torch.zeros(B, Hkv, T, D, dtype=src, device="cuda")
        s["out_v"] = torch.zeros(B, Hkv, T, D, dtype=src, device="cuda")
    return s


# ---------------------------------------------------------- the library


def _own(s):
    import exact_tiled_attention_softmax_b200 as eta
    case = s["case"]
    if s["op"] == "train":
        allowed = eta.AllowedSet(causal=True, window_left=case["window"], window_first=case["first"], sink=s["sink"])
        o, lse = eta.attn_fwd(s["q"], s["k"], s["v"], allowed, s["scale"])
        dq, dk, dv, dsink = eta.attn_bwd(s["q"], s["k"], s["v"], o, s["do"], lse, allowed, s["scale"])
        return [o, lse, dq, dk, dv] + ([dsink] if dsink is not None else [])
    cache = eta.PagedCache(s["k"], s["v"], s["block_table"], s["seq_lens"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "write":
        eta.attn_cache_write(s["new_k"], s["new_v"], cache, s["cu_q"])
        return _cache_of(s)
    if s["op"] == "read":
        eta.attn_cache_read(cache, k=s["out_k"], v=s["out_v"])
        return [s["out_k"], s["out_v"]]
    allowed = eta.AllowedSet(causal=True, window_left=case["window"], window_first=case["first"], sink=s["sink"])
    return list(eta.attn_paged_fwd(s["q"], cache, s["cu_q"], allowed, s["scale"], max_q=s["max_new"]))


def _cache_of(s):
    return [s[x] for x in ("k", "v", "k_scale", "v_scale") if s[x] is not None]


# ---------------------------------------------------------- plain forms


def _tokens(s):
    """Of each new token: its sequence, its index in the chunk and its position in the sequence."""
    t = torch.arange(s["total"], device="cuda")
    cu = s["cu_q"].long()
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    return b, i, s["seq_lens"].long()[b] - (cu[b + 1] - cu[b]) + i


def _plain_write(s):
    b, _, pos = _tokens(s)
    page = s["case"]["page"]
    pg, off = s["block_table"].long()[b, pos // page], pos % page

    def put(x, new, scale):
        if scale is None:
            x[pg, off] = new.to(x.dtype)
            return
        c, sc = _quantised(new)
        x.view(torch.uint8)[pg, off] = c.view(torch.uint8)
        scale[pg, off] = sc

    put(s["k"], s["new_k"], s["k_scale"])
    put(s["v"], s["new_v"], s["v_scale"])
    return _cache_of(s)


def _gathered(s, x):
    """The cached rows of every sequence as fp32 [B, Hkv, max_len, d]."""
    page, Lm = s["case"]["page"], s["max_len"]
    table = s["block_table"].long()

    def rows(t):
        got = t[table]
        return got.reshape(got.shape[0], -1, *got.shape[3:])[:, :Lm].transpose(1, 2)

    r = rows(s[x].view(torch.uint8)).contiguous().view(E4M3).float() if s[x].dtype == E4M3 else rows(s[x]).float()
    return r if s[x + "_scale"] is None else r * rows(s[x + "_scale"])[..., None]


def _plain_read(s):
    live = (torch.arange(s["max_len"], device="cuda") < s["seq_lens"][:, None])[:, None, :, None]
    s["out_k"].copy_(torch.where(live, _gathered(s, "k").to(s["out_k"].dtype), s["out_k"]))
    s["out_v"].copy_(torch.where(live, _gathered(s, "v").to(s["out_v"].dtype), s["out_v"]))
    return [s["out_k"], s["out_v"]]


def _seen(pos, keys, window, first):
    """Whether a query at `pos` sees each key: causal, and inside the window or among the first ones."""
    ok = keys <= pos
    return ok & ((keys > pos - window) | (keys < first)) if window else ok


def _softmax(scores, ok, z):
    """Probabilities over the allowed keys (and the sink logit z), and the log of the denominator."""
    sc = scores.masked_fill(~ok, -math.inf)
    m = sc.amax(-1, keepdim=True)
    if z is not None:
        m = torch.maximum(m, z)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(sc - m)
    den = p.sum(-1, keepdim=True)
    if z is not None:
        den = den + torch.exp(z - m)
    return p / torch.where(den == 0, torch.ones_like(den), den), (m + torch.log(den))[..., 0]


def _plain_paged(s):
    case = s["case"]
    Hq, Hkv, nq = case["Hq"], case["Hkv"], s["max_new"]
    g = Hq // Hkv
    cu = s["cu_q"].long()
    rows = (cu[:-1, None] + torch.arange(nq, device="cuda")).clamp(max=s["total"] - 1)
    q = s["q"].float()[rows].reshape(-1, nq, Hkv, g, D).permute(0, 2, 3, 1, 4)          # [B, Hkv, g, nq, d]
    k, v = _gathered(s, "k"), _gathered(s, "v")
    pos = s["seq_lens"].long()[:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(nq, device="cuda")
    keys = torch.arange(s["max_len"], device="cuda")
    ok = _seen(pos[:, :, None], keys, case["window"], case["first"]) & (keys < s["seq_lens"].long()[:, None, None])
    sc = torch.matmul(q, k[:, :, None].transpose(-1, -2)) * s["scale"]
    z = None if s["sink"] is None else s["sink"].reshape(1, Hkv, g, 1, 1)
    p, lse = _softmax(sc, ok[:, None, None], z)
    # a row past the cache's end may hold anything: only rows that some query sees take part
    v = torch.where((keys < s["seq_lens"].long()[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v[:, :, None]).permute(0, 3, 1, 2, 4).reshape(-1, nq, Hq, D)
    lse = lse.permute(0, 3, 1, 2).reshape(-1, nq, Hq)
    b, i, _ = _tokens(s)
    return [o[b, i].to(s["q"].dtype), lse[b, i]]


def _plain_train(s):
    case = s["case"]
    B, T, Hq, Hkv = case["B"], case["T"], case["Hq"], case["Hkv"]
    c = s["scale"]
    q, do = s["q"].float().reshape(B, Hkv, -1, T, D), s["do"].float().reshape(B, Hkv, -1, T, D)
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    t = torch.arange(T, device="cuda")
    ok = _seen(t[:, None], t, case["window"], case["first"])
    z = None if s["sink"] is None else s["sink"].reshape(1, Hkv, -1, 1, 1)
    p, lse = _softmax(torch.matmul(q, k.transpose(-1, -2)) * c, ok, z)
    o = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    delta = (o * do).sum(-1, keepdim=True)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_(delta).mul_(p)
    dq = torch.matmul(ds, k) * c
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2) * c
    dt = s["q"].dtype
    out = [o.reshape(B, Hq, T, D).to(dt), lse.reshape(B, Hq, T), dq.reshape(B, Hq, T, D).to(dt), dk.to(dt), dv.to(dt)]
    if z is not None:
        out.append(-(torch.exp(z[..., 0] - lse) * delta[..., 0]).sum((0, 3)).reshape(Hq))
    return out


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "paged": _plain_paged, "train": _plain_train}[state["op"]](state)


# ------------------------------------------------------------ in 64 bits


def _exact_rows(s, x, b, h):
    """Sequence b's cached rows of head h, as the values they stand for."""
    page, L = s["case"]["page"], int(s["seq_lens"][b])
    ids = s["block_table"][b, : -(-L // page)].tolist()
    rows = torch.stack([s[x][p, :, h] for p in ids]).reshape(-1, D)[:L].double()
    if s[x + "_scale"] is not None:
        rows = rows * torch.stack([s[x + "_scale"][p, :, h] for p in ids]).reshape(-1)[:L].double()[:, None]
    return rows


def exact(case, seed):
    s = prepare(case, seed)
    f64 = dict(dtype=torch.float64, device="cuda")
    if case["op"] == "train":
        return _exact_train(case, s, f64)
    n, L = _lengths(case)
    cu = np.concatenate([[0], np.cumsum(n)])
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    if case["op"] == "read":
        out = [s["out_k"].double(), s["out_v"].double()]
        for b in range(B):
            for h in range(Hkv):
                out[0][b, h, : L[b]] = _exact_rows(s, "k", b, h)
                out[1][b, h, : L[b]] = _exact_rows(s, "v", b, h)
        return out
    if case["op"] == "write":
        if s["total"] > 16384:
            return None
        vals, scales = [], []
        table = s["block_table"].cpu().numpy()
        pos = np.concatenate([np.arange(L[b] - n[b], L[b]) for b in range(B)])
        seq = np.repeat(np.arange(B), n)
        at = torch.from_numpy(table[seq, pos // page].astype(np.int64) * page + pos % page).to("cuda")
        for x in ("k", "v"):
            whole = s[x].double().reshape(-1, Hkv, D)
            new = s["new_" + x].double()
            if s[x + "_scale"] is not None:
                sc = s[x + "_scale"].double().reshape(-1, Hkv)
                a = new.abs().amax(-1) / E4M3_MAX
                a[a == 0] = 1
                y = new / a[..., None]
                # e4m3: 3 fraction bits, the smallest exponent -6; halves go to the even neighbour
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                whole[at], sc[at] = torch.round(y / step) * step, a
                scales.append(sc.reshape(s[x + "_scale"].shape))
            else:
                whole[at] = new
            vals.append(whole.reshape(s[x].shape))
        return vals + scales
    out, lse = torch.zeros(s["total"], case["Hq"], D, **f64), torch.zeros(s["total"], case["Hq"], **f64)
    g = case["Hq"] // Hkv
    for b in range(B):
        p = torch.arange(int(L[b] - n[b]), int(L[b]), device="cuda")
        t = slice(int(cu[b]), int(cu[b + 1]))
        j = torch.arange(int(L[b]), device="cuda")
        hidden = j[None] > p[:, None]
        if case["window"]:
            hidden |= (j[None] <= p[:, None] - case["window"]) & (j[None] >= case["first"])
        for h in range(Hkv):
            k, v = _exact_rows(s, "k", b, h), _exact_rows(s, "v", b, h)
            for hh in range(h * g, h * g + g):
                x = (s["q"][t, hh].double() @ k.T) * s["scale"]
                x[hidden] = -math.inf
                l = torch.logsumexp(x, 1)
                if s["sink"] is not None:
                    l = torch.logaddexp(l, s["sink"][hh].double())
                out[t, hh], lse[t, hh] = torch.exp(x - l[:, None]) @ v, l
    return [out, lse]


def _exact_train(case, s, f64):
    B, T, Hq, Hkv = case["B"], case["T"], case["Hq"], case["Hkv"]
    g, c = Hq // Hkv, s["scale"]
    t = torch.arange(T, device="cuda")
    hidden = (t[None] > t[:, None]) | ((t[None] <= t[:, None] - case["window"]) & (t[None] >= case["first"]))
    o, dq = torch.zeros(B, Hq, T, D, **f64), torch.zeros(B, Hq, T, D, **f64)
    dk, dv = torch.zeros(B, Hkv, T, D, **f64), torch.zeros(B, Hkv, T, D, **f64)
    lse, dz = torch.zeros(B, Hq, T, **f64), torch.zeros(Hq, **f64)
    for b in range(B):
        for h in range(Hq):
            q, do = s["q"][b, h].double(), s["do"][b, h].double()
            k, v = s["k"][b, h // g].double(), s["v"][b, h // g].double()
            x = q @ k.T * c
            x[hidden] = -math.inf
            l = torch.logsumexp(x, 1)
            if s["sink"] is not None:
                l = torch.logaddexp(l, s["sink"][h].double())
            p = torch.exp(x - l[:, None])
            y = p @ v
            delta = (y * do).sum(1)
            ds = p * (do @ v.T - delta[:, None])
            o[b, h], lse[b, h], dq[b, h] = y, l, ds @ k * c
            dk[b, h // g] += ds.T @ q * c
            dv[b, h // g] += p.T @ do
            if s["sink"] is not None:
                dz[h] -= (torch.exp(s["sink"][h].double() - l) * delta).sum()
    return [o, lse, dq, dk, dv] + ([dz] if s["sink"] is not None else [])
