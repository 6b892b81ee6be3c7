"""NaN queries, NaN rows and logits that are all -inf, in heads that one CTA serves and in heads that are cut over
several and joined: the results are the same."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(gpu_device):
    import __graft_entry__
    __graft_entry__.build()
    return gpu_device


def made(g, B, Hq, H, cap, d, dtype, q4, dev):
    """A queries tensor, a score, a cache and a call of (q, len, score) over it, on the GPU."""
    import kv_cache_compression_gb300 as kv
    q = (torch.randn(B, Hq, d, generator=g) * 1.5).to(dtype).to(dev)
    score = torch.rand(B, H, cap, generator=g).to(dev)
    rows = [torch.randn(B, H, cap, d, generator=g).to(dtype).to(dev) for _ in "kv"]
    if not q4:
        return q, score, rows[0], lambda q, n, s: kv.decode_attend_scored(q, *rows, n, s, decay=0.5)
    cache = kv.Q4Cache.empty(B, H, cap, d, dev)
    kv.q4_append(cache, *rows, torch.zeros(B, dtype=torch.int32, device=dev))
    return q, score, cache.k_meta, lambda q, n, s: kv.q4_decode_attend(q, cache, n, s, decay=0.5)


SHAPES = [(2, 2, 100),        # one CTA a head
          (1, 2, 40000),      # heads cut over hundreds of CTAs
          (1, 1, 3001),       # over some twenty
          (40, 8, 1200)]      # whole heads, and heads cut in two
CALLS = [(torch.bfloat16, 3), (torch.bfloat16, 6), (torch.bfloat16, 11), (torch.float32, 3), (torch.float32, 11)]


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("B,H,cap", SHAPES)
@pytest.mark.parametrize("dtype,G", CALLS)
def test_a_nan_query_gives_nan_and_spares_the_others(dev, B, H, cap, dtype, G, q4):
    g = torch.Generator().manual_seed(cap + G)
    d = 64
    q, score, _, call = made(g, B, G * H, H, cap, d, dtype, q4, dev)
    lens = torch.tensor([cap - b for b in range(B)], dtype=torch.int32, device=dev)
    want_s, s = score.clone(), score.clone()
    want = call(q, lens, want_s)
    heads = [(b, h) for b in range(B) for h in range(H) if (b + h) % 3 == 0]
    for b, h in heads:
        q[b, h * G + G // 2, 5] = float("nan")
        want[b, h * G + G // 2] = float("nan")
        want_s[b, h, :lens[b]] = float("nan")
    out = call(q, lens, s)
    plain = call(q, lens, None)
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isnan(s), torch.isnan(want_s))
    assert torch.equal(out.nan_to_num(), want.nan_to_num()) and torch.equal(s.nan_to_num(), want_s.nan_to_num())
    assert torch.equal(plain.nan_to_num(), out.nan_to_num()) and torch.equal(torch.isnan(plain), torch.isnan(out))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("B,H,cap", SHAPES)
@pytest.mark.parametrize("dtype,G", CALLS)
def test_parts_of_nan_rows_reach_the_whole_head(dev, B, H, cap, dtype, G, q4):
    """The first half of a head's rows is NaN: whole CTAs see nothing else."""
    g = torch.Generator().manual_seed(cap + G + 1)
    q, score, keys, call = made(g, B, G * H, H, cap, 64, dtype, q4, dev)
    lens = torch.tensor([cap - b for b in range(B)], dtype=torch.int32, device=dev)
    want_s, s = score.clone(), score.clone()
    want = call(q, lens, want_s)
    keys[0, 0, :cap // 2] = float("nan")
    want[0, :G] = float("nan")
    want_s[0, 0, :lens[0]] = float("nan")
    out = call(q, lens, s)
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isnan(s), torch.isnan(want_s))
    assert torch.equal(out.nan_to_num(), want.nan_to_num()) and torch.equal(s.nan_to_num(), want_s.nan_to_num())


@pytest.mark.parametrize("B,H,cap", SHAPES)
@pytest.mark.parametrize("dtype,G", CALLS)
def test_logits_that_are_all_minus_infinity_add_nothing(dev, B, H, cap, dtype, G):
    """Finite rows and a finite query whose products pass fp32's range: o = 0, and no weight for any row."""
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(cap + G + 2)
    d = 64
    q = (torch.randn(B, G * H, d, generator=g) * 1.5).to(dtype)
    k, v = (torch.randn(B, H, cap, d, generator=g).to(dtype) for _ in "kv")
    q[..., 0] = 0.0
    k[..., 0] = -2.0 ** 100
    score = torch.rand(B, H, cap, generator=g).to(dev)
    n = torch.full((B,), cap, dtype=torch.int32, device=dev)
    k, v = k.to(dev), v.to(dev)
    want_s, s = score.clone(), score.clone()
    want = kv.decode_attend_scored(q.to(dev), k, v, n, want_s, decay=0.0)
    q[0, :G] = 0.0                                        # of head 0, all queries; the others are as they were
    q[0, :G, 0] = 2.0 ** 100
    want[0, :G] = 0.0
    want_s[0, 0] = 0.0
    out = kv.decode_attend_scored(q.to(dev), k, v, n, s, decay=0.0)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(s, want_s)
