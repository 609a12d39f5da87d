"""Calls on another stream than the current one: what the binding allocates is
ordered with the kernels that write it, and takes no memory that the current
stream still reads."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import exact_tiled_attention_softmax_b200 as eta  # noqa: E402
from tests.paged_util import cu_of, make_cache, seeded_q  # noqa: E402

BUSY = 100_000_000  # clocks of a kernel that keeps a stream busy: 50 ms


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    eta.load_library()


def held_back(call, *sizes):
    """call(stream)'s result while the current stream is busy and, behind that,
    still has to read freed blocks of the sizes (bytes) that the call allocates;
    checks that what it reads is what was there."""
    s = torch.cuda.Stream()
    call(s)  # (loads the kernels, which waits for the device)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.full((n,), i + 1, dtype=torch.uint8, device="cuda") for i, n in enumerate(sizes)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    reads = [x.clone() for x in blocks]
    del blocks
    got = call(s)
    s.synchronize()
    torch.cuda.synchronize()
    for i, r in enumerate(reads):
        assert (r == i + 1).all(), f"block {i} was taken while the current stream still read it"
    return got


@pytest.mark.parametrize("given", ["none", "k", "v"])
def test_cache_read_into_new_tensors(given):
    lens, T = [700, 301], 720
    cache, K, V = make_cache(lens, 16, 4, 128, 128, torch.bfloat16, seed=2)
    size = 2 * 4 * T * 128 * 2
    kept = torch.zeros(2, 4, T, 128, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()

    def call(s):
        return eta.attn_cache_read(cache, T, stream=s, **({} if given == "none" else {given: kept}))

    for got, want in zip(held_back(call, *[size] * (2 if given == "none" else 1)), (K, V)):
        for b, L in enumerate(lens):
            assert torch.equal(got[b, :, :L].transpose(0, 1).double().cpu(), want[b])
            assert (got[b, :, L:] == 0).all()


@pytest.mark.parametrize("new", [1, 300])
def test_paged_attention(new):
    lens = [700, 301, 512]
    cache, _, _ = make_cache(lens, 16, 8, 128, 128, torch.bfloat16, seed=3)
    q, cu, a = seeded_q(3 * new, 64, 128, torch.bfloat16), cu_of([new] * 3), eta.AllowedSet(causal=True)
    want = eta.attn_paged_fwd(q, cache, cu, a, max_q=new)
    sizes = [q.numel() * 2, q.numel() // 128 * 4, eta.attn_paged_workspace_size(q, cache, a)]
    for x, y in zip(held_back(lambda s: eta.attn_paged_fwd(q, cache, cu, a, max_q=new, stream=s), *sizes), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("sink", [False, True])
def test_dense_forward_and_reverse(sink):
    B, Hq, Hkv, T, d = 2, 8, 4, 600, 128
    q, k, v, g = (seeded_q(B * h, T, d, torch.bfloat16, i).view(B, h, T, d) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    z = torch.randn(Hq, device="cuda") if sink else None
    # (with lengths the forward's workspace holds a table that its kernel reads)
    a = eta.AllowedSet(causal=True, lengths=torch.tensor([600, 333], dtype=torch.int32, device="cuda"), sink=z,
                       deterministic=True)
    o, lse = eta.attn_fwd(q, k, v, a)
    want = eta.attn_bwd(q, k, v, o, g, lse, a)
    sizes = [q.numel() * 2, lse.numel() * 4, eta.attn_fwd_workspace_size(q, k, v, a)]
    for x, y in zip(held_back(lambda s: eta.attn_fwd(q, k, v, a, stream=s), *sizes), (o, lse)):
        assert torch.equal(x, y)
    sizes = [q.numel() * 2, k.numel() * 2, k.numel() * 2, eta.attn_bwd_workspace_size(q, k, v, a)]
    got = held_back(lambda s: eta.attn_bwd(q, k, v, o, g, lse, a, stream=s), *sizes)
    for x, y in zip(got[:3], want[:3]):
        assert torch.equal(x, y)
    assert sink == (got[3] is not None) and (not sink or torch.equal(got[3], want[3]))


def test_a_dropped_workspace_is_not_taken_by_the_current_stream():
    """The workspace that a call makes for itself goes back to its own stream's
    memory: what the current stream allocates and fills next is not it."""
    B, H, T, d = 1, 16, 2048, 128
    q, k, v, g = (seeded_q(B * H, T, d, torch.bfloat16, i).view(B, H, T, d) for i in range(4))
    a = eta.AllowedSet(causal=True, deterministic=True)
    o, lse = eta.attn_fwd(q, k, v, a)
    want = eta.attn_bwd(q, k, v, o, g, lse, a)
    n = eta.attn_bwd_workspace_size(q, k, v, a)
    s = torch.cuda.Stream()
    for _ in range(20):
        torch.cuda.synchronize()
        got = eta.attn_bwd(q, k, v, o, g, lse, a, stream=s)
        for _ in range(4):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7F)
        torch.cuda.synchronize()
        for x, y in zip(got[:3], want[:3]):
            assert torch.equal(x, y)
