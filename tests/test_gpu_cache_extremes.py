"""The cache operators at the largest batches that a call may have, and evictions beyond 2^32 bytes."""
import pytest
import torch

from tests.cache_cases import check_attend, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(gpu_device):
    import __graft_entry__
    __graft_entry__.build()
    return gpu_device


def check_evicted(head, before, after, score0, score, idx, length, keep, recent):
    """One head (b, h) of an eviction from `length` rows: the slots that stay and what moved into them."""
    b, h = head
    n, left = length - recent, keep + recent
    i = idx[b, h].long()
    top = torch.topk(score0[b, h, :n], keep).indices.sort().values          # (random scores: no ties)
    assert torch.equal(i[:keep].sort().values, top)
    still = top[top < keep]
    assert torch.equal(i[still], still)                                      # those below `keep` stay in place
    holes = torch.ones(keep, dtype=torch.bool, device=i.device)
    holes[still] = False
    assert torch.equal(i[:keep][holes], top[top >= keep])                    # the others fill the gaps in order
    assert torch.equal(i[keep:], torch.arange(n, length, device=i.device))
    for old, new in zip(before, after):
        assert torch.equal(new[b, h, :left], old[b, h][i])
    assert torch.equal(score[b, h, :left], score0[b, h][i])
    assert not score[b, h, left:length].any() and torch.equal(score[b, h, length:], score0[b, h, length:])


@pytest.mark.parametrize("cap,G", [(3, 1), (300, 2)])
def test_the_largest_batch(dev, cap, G):
    import kv_cache_compression_gb300 as kv
    B, H, d = 65535, 1, 64
    g = torch.Generator(device=dev).manual_seed(cap)
    k, v = (torch.randn(B, H, cap, d, generator=g, device=dev, dtype=torch.float32).bfloat16() for _ in range(2))
    q = torch.randn(B, G, d, generator=g, device=dev).bfloat16()
    n = torch.randint(0, cap + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    n[0], n[-1] = cap, cap
    score0 = torch.rand(B, H, cap, generator=g, device=dev)
    some = [0, 1, 255, 32768, 65279, 65534]

    def part(t):
        return t[some].cpu()

    s = score0.clone()
    out = kv.decode_attend_scored(q, k, v, n, s)
    torch.cuda.synchronize()
    check_attend(part(q), to64(part(k)), to64(part(v)), part(n).tolist(), part(out), score0=part(score0), score=part(s))

    cache = kv.Q4Cache.empty(B, H, cap, d, dev)
    zero = torch.zeros(B, dtype=torch.int32, device=dev)
    held = kv.q4_append(cache, k, v, zero, n_new=n)
    assert torch.equal(held, n)
    k4, v4 = kv.q4_read(cache, cap, dtype=torch.float32)
    s = score0.clone()
    out = kv.q4_decode_attend(q, cache, n, s)
    torch.cuda.synchronize()
    lens = part(n).tolist()
    k64, v64 = to64(part(k4)), to64(part(v4))
    for b, m in enumerate(lens):
        k64[b, :, m:] = v64[b, :, m:] = 0                                    # (rows that were not written)
    size = {"k_size": 3 * abs(k64).max(-1, keepdims=True) + 0 * k64, "v_size": 3 * abs(v64).max(-1, keepdims=True) + 0 * v64}
    check_attend(part(q), k64, v64, lens, part(out), score0=part(score0), score=part(s), **size)

    keep, recent = cap // 2, 1
    s, k2, v2 = score0.clone(), k.clone(), v.clone()
    after, idx = kv.evict(k2, v2, s, n, keep=keep, recent=recent)
    torch.cuda.synchronize()
    assert torch.equal(after, n.clamp(max=keep + recent))
    for b in some:
        if n[b] > keep + recent:
            check_evicted((b, 0), (k, v), (k2, v2), score0, s, idx, n[b].item(), keep, recent)


def test_evictions_past_32_bits(dev):
    import kv_cache_compression_gb300 as kv
    B, H, cap, d, keep, recent = 1, 24, 800_000, 128, 699_990, 300
    g = torch.Generator(device=dev).manual_seed(3)
    k = torch.empty(B, H, cap, d, dtype=torch.bfloat16, device=dev)
    for h in range(H):
        k[0, h].normal_(generator=g)
    v = k.flip(2)
    assert (H - 1) * cap * d * 2 > 1 << 32
    score0 = torch.rand(B, H, cap, generator=g, device=dev, dtype=torch.float64).argsort(-1).float()   # no ties
    length = cap - 5
    n = torch.tensor([length], dtype=torch.int32, device=dev)
    k2, v2, s = k.clone(), v.clone(), score0.clone()
    after, idx = kv.evict(k2, v2, s, n, keep=keep, recent=recent)
    torch.cuda.synchronize()
    assert after.tolist() == [keep + recent]
    for h in (0, H - 1):
        check_evicted((0, h), (k, v), (k2, v2), score0, s, idx, length, keep, recent)
    assert torch.equal(k2[0, H - 1, keep + recent:], k[0, H - 1, keep + recent:])


@pytest.mark.parametrize("B,H,G", [(32, 5, 1), (16, 4, 20)])
def test_caches_much_longer_than_their_sequences(dev, B, H, G):
    """The joining kernel's blocks take turns over a head's rows (with twenty queries, in several passes)."""
    import kv_cache_compression_gb300 as kv
    d, cap = 64, 20011
    g = torch.Generator(device=dev).manual_seed(B)
    k, v = (torch.randn(B, H, cap, d, generator=g, device=dev).bfloat16() for _ in range(2))
    q = torch.randn(B, H * G, d, generator=g, device=dev).bfloat16()
    score0 = torch.rand(B, H, cap, generator=g, device=dev)
    lens = [(0, cap, 1000, 2049, cap - 1, 1)[b % 6] for b in range(B)]
    s = score0.clone()
    out = kv.decode_attend_scored(q, k, v, torch.tensor(lens, dtype=torch.int32, device=dev), s, decay=0.5)
    torch.cuda.synchronize()
    some = [0, 1, 2, 3, B - 4, B - 1]
    check_attend(q[some].cpu(), to64(k[some].cpu()), to64(v[some].cpu()), [lens[b] for b in some], out[some].cpu(),
                 score0=score0[some].cpu(), score=s[some].cpu(), decay=0.5, heads=[0, H - 1])


@pytest.mark.parametrize("B,H,cap", [(16, 32, 30011), (32, 32, 25013)])
def test_evictions_of_long_caches_of_many_heads(dev, B, H, cap):
    """More keys than one CTA's shared memory holds: clusters that do not all run at once, or keys read again."""
    import kv_cache_compression_gb300 as kv
    d, keep, recent = 64, cap - 900, 32
    g = torch.Generator(device=dev).manual_seed(cap)
    k, v = (torch.randn(B, H, cap, d, generator=g, device=dev).bfloat16() for _ in range(2))
    score0 = torch.rand(B, H, cap, generator=g, device=dev).argsort(-1).float()      # no ties
    lens = [cap - 7 * b for b in range(B)]
    k2, v2, s = k.clone(), v.clone(), score0.clone()
    after, idx = kv.evict(k2, v2, s, torch.tensor(lens, dtype=torch.int32, device=dev), keep=keep, recent=recent)
    torch.cuda.synchronize()
    assert after.tolist() == [min(n, keep + recent) for n in lens]
    for b in (0, 1, B - 1):
        for h in (0, H - 1):
            if lens[b] > keep + recent:
                check_evicted((b, h), (k, v), (k2, v2), score0, s, idx, lens[b], keep, recent)
