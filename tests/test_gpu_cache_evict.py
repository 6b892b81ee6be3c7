"""GPU parity of snapkv_evict and snapkv_q4_evict against the oracle, bit for bit, and the operators'
run together: compress, hold in 4 bits, decode with scores, evict."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests.cache_cases import check_attend, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(gpu_device):
    import __graft_entry__
    __graft_entry__.build()
    return gpu_device


def scores(g, shape, kind):
    s = torch.rand(shape, generator=g) ** 4
    if kind == "ties":
        s = (s * 4).floor() / 4
    elif kind == "equal":
        s.fill_(0.5)
    elif kind == "odd":                                  # NaN, infinities, negatives, both zeros
        r = torch.rand(shape, generator=g)
        s = torch.where(r < 0.1, torch.tensor(float("nan")), s - 0.3)
        s = torch.where(r > 0.95, torch.tensor(float("inf")), s)
        s = torch.where((r > 0.9) & (r < 0.95), torch.tensor(float("-inf")), s)
        s = torch.where((r > 0.5) & (r < 0.6), torch.tensor(-0.0), s)
        s = torch.where((r > 0.6) & (r < 0.7), torch.tensor(0.0), s)
    return s


def same(a, b):
    """Equal bit for bit."""
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def check(kv, dev, tensors, call, score, lens, keep, recent):
    """Runs an eviction on copies of `tensors` [B,H,cap,...] and compares every byte with the oracle."""
    B, H, cap = score.shape
    left = keep + recent
    got = [t.to(dev) for t in tensors]
    s = score.to(dev)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    len_out, idx = call(got, s, n, status)
    torch.cuda.synchronize()
    assert n.tolist() == lens
    clipped = [min(max(x, 0), cap) for x in lens]
    assert status.item() == (kv.snapkv.ERR_CAPACITY if any(x > cap for x in lens) else 0)
    assert len_out.tolist() == [min(x, left) for x in clipped]
    want = [t.clone() for t in tensors]
    want_s = score.clone()
    want_i = torch.arange(left, dtype=torch.int32).expand(B, H, left).clone()
    for b in range(B):
        if clipped[b] <= left:
            continue
        for h in range(H):
            src = torch.from_numpy(co.evict_slots(to64(score[b, h]), clipped[b], keep, recent).copy())
            for t, w in zip(tensors, want):
                w[b, h, :left] = t[b, h, src]
            want_s[b, h, :left] = score[b, h, src]
            want_i[b, h] = src.int()
            want_s[b, h, left:clipped[b]] = 0.0
    assert torch.equal(idx.cpu(), want_i)
    assert same(s, want_s)
    for i, (x, w) in enumerate(zip(got, want)):
        assert same(x, w), f"tensor {i}"


def dense_call(kv, keep, recent):
    return lambda t, s, n, st: kv.evict(t[0], t[1], s, n, keep=keep, recent=recent, dev_status=st)


def q4_call(kv, keep, recent):
    return lambda t, s, n, st: kv.q4_evict(kv.Q4Cache(*t), s, n, keep=keep, recent=recent, dev_status=st)


def rows_of(g, B, H, cap, d, dtype):
    if dtype == "q4":
        codes = [torch.randint(0, 256, (B, H, cap, d // 2), generator=g, dtype=torch.uint8) for _ in "kv"]
        meta = [torch.randn(B, H, cap, d // 64, 2, generator=g).bfloat16() for _ in "kv"]
        return [codes[0], meta[0], codes[1], meta[1]]
    return [torch.randn(B, H, cap, d, generator=g).to(dtype) for _ in "kv"]


KEEP = [(40, 20), (0, 30), (60, 0), (1, 1), (99, 0), (63, 36), (16, 70)]


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 64),
                                     (torch.float32, 128), ("q4", 64), ("q4", 128)])
@pytest.mark.parametrize("keep,recent", KEEP)
def test_small_caches(dev, dtype, d, keep, recent):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(keep + 7 * recent + d)
    lens = [100, 101, 60, 0, keep + recent, min(101, keep + recent + 1)]
    B, H, cap = len(lens), 2, 101                        # odd: rows of pairs start off 16-byte boundaries
    t = rows_of(g, B, H, cap, d, dtype)
    call = (q4_call if dtype == "q4" else dense_call)(kv, keep, recent)
    check(kv, dev, t, call, scores(g, (B, H, cap), "random"), lens, keep, recent)


@pytest.mark.parametrize("kind", ["ties", "equal", "odd"])
@pytest.mark.parametrize("keep,recent", [(50, 10), (700, 100), (1500, 1), (0, 600)])
def test_ties_and_unusual_scores(dev, kind, keep, recent):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(keep)
    B, H, cap = 3, 2, 2600
    t = rows_of(g, B, H, cap, 64, "q4")
    check(kv, dev, t, q4_call(kv, keep, recent), scores(g, (B, H, cap), kind), [2600, 1700, 30], keep, recent)


@pytest.mark.parametrize("B,H,cap,keep,recent,dtype", [
    (1, 1, 50000, 30000, 64, torch.bfloat16),      # one head over a whole cluster
    (1, 2, 30011, 30000, 0, "q4"),                 # a handful leaves
    (1, 2, 30011, 100, 5, torch.bfloat16),         # a handful stays
    (160, 2, 18000, 17900, 80, "q4"),              # one CTA a head, keys beyond its shared memory
    (2, 1, 5000, 1000, 3900, torch.float32),       # the newest rows come down over their old place
    (2, 1, 5000, 1099, 3900, "q4"),                # by one slot
])
def test_large_caches(dev, B, H, cap, keep, recent, dtype):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(cap)
    d = 64 if dtype == "q4" else 128
    t = rows_of(g, B, H, cap, d, dtype)
    call = (q4_call if dtype == "q4" else dense_call)(kv, keep, recent)
    lens = [cap - (b % 5) for b in range(B)]
    check(kv, dev, t, call, scores(g, (B, H, cap), "random"), lens, keep, recent)


def test_lengths_past_the_cache_are_clamped(dev):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(1)
    t = rows_of(g, 3, 2, 40, 64, torch.bfloat16)
    check(kv, dev, t, dense_call(kv, 20, 5), scores(g, (3, 2, 40), "random"), [45, 40, -2], 20, 5)


def test_without_indices_and_with_the_callers_buffers(dev):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(2)
    k, v = (x.to(dev) for x in rows_of(g, 2, 2, 300, 128, torch.bfloat16))
    s = scores(g, (2, 2, 300), "random").to(dev)
    n = torch.tensor([300, 280], dtype=torch.int32, device=dev)
    k1, v1, s1, k2, v2, s2 = k.clone(), v.clone(), s.clone(), k.clone(), v.clone(), s.clone()
    a, idx = kv.evict(k1, v1, s1, n, keep=200, recent=10)
    ws = kv.snapkv.new_workspace(kv.evict_workspace_size(2, 2, 300), dev)
    out = torch.empty_like(n)
    b, none = kv.evict(k2, v2, s2, n, out, keep=200, recent=10, want_idx=False, workspace=ws)
    torch.cuda.synchronize()
    assert none is None and b is out and torch.equal(a, b) and idx.shape == (2, 2, 210)
    assert same(k1, k2) and same(v1, v2) and same(s1, s2)


def test_from_a_graph_on_a_side_stream(dev):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(3)
    k, v = (x.to(dev) for x in rows_of(g, 2, 3, 6000, 64, torch.bfloat16))
    s = scores(g, (2, 3, 6000), "ties").to(dev)
    n = torch.tensor([6000, 5999], dtype=torch.int32, device=dev)
    k1, v1, s1 = k.clone(), v.clone(), s.clone()
    want, want_i = kv.evict(k1, v1, s1, n, keep=4000, recent=500)
    ws = kv.snapkv.new_workspace(kv.evict_workspace_size(2, 3, 6000), dev)
    k2, v2, s2, out, idx = k.clone(), v.clone(), s.clone(), torch.empty_like(n), torch.empty_like(want_i)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream(dev)):
        kv.evict(k2, v2, s2, n, out, keep=4000, recent=500, idx_out=idx, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(idx, want_i) and same(k2, k1) and same(v2, v1) and same(s2, s1)


@pytest.mark.parametrize("q4", [False, True])
def test_a_decode_loop_over_a_compressed_cache(dev, q4):
    """As a user runs them: a prompt is compressed, its cache held in 4 bits (or dense), every step appends a
    token and attends with the running score, and whenever the cache is full it is evicted down to its budget.
    The oracle keeps its own rows and scores and is fed only the tokens; its rows are followed to the end
    through the slots that the evictions report."""
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(21)
    B, H, G, d, l_obs, budget, slack = 2, 2, 4, 128, 8, 48, 6
    L = 300
    prompt_k = torch.randn(B, H, L, d, generator=g).bfloat16().to(dev)
    prompt_v = torch.randn(B, H, L, d, generator=g).bfloat16().to(dev)
    q_obs = torch.randn(B, G * H, l_obs, d, generator=g).bfloat16().to(dev)
    held, cap = budget + l_obs, budget + l_obs + slack
    res = kv.compress(q_obs, prompt_k, prompt_v, pool_kernel=5, budget=budget, cap=cap)
    score = torch.zeros(B, H, cap, device=dev)
    lens = [res["len"], torch.empty_like(res["len"])]
    if q4:
        cache = kv.Q4Cache.empty(B, H, cap, d, dev)
        zero = torch.zeros(B, dtype=torch.int32, device=dev)
        lens[0] = kv.q4_append(cache, res["k_out"][:, :, :held].contiguous(), res["v_out"][:, :, :held].contiguous(),
                               zero)
    else:
        k_cache, v_cache = res["k_out"], res["v_out"]
    torch.cuda.synchronize()

    def stored(x):
        return co.values(*co.quantise(to64(x))) if q4 else to64(x)
    rows_k, rows_v = stored(res["k_out"][:, :, :held]), stored(res["v_out"][:, :, :held])
    tally = np.zeros((B, H, held))
    evictions = 0
    for step in range(20):
        q = torch.randn(B, G * H, d, generator=g).bfloat16()
        kn, vn = (torch.randn(B, H, d, generator=g).bfloat16() for _ in range(2))
        if q4:
            lens[1] = kv.q4_append(cache, kn.to(dev), vn.to(dev), lens[0], lens[1])
            lens.reverse()
            before = score.clone()
            out = kv.q4_decode_attend(q.to(dev), cache, lens[0], score)
        else:
            kv.append(kn.to(dev), vn.to(dev), k_cache, v_cache, lens[0])
            before = score.clone()
            out = kv.decode_attend_scored(q.to(dev), k_cache, v_cache, lens[0], score)
        rows_k = np.concatenate([rows_k, stored(kn)[:, :, None]], 2)
        rows_v = np.concatenate([rows_v, stored(vn)[:, :, None]], 2)
        n = rows_k.shape[2]
        tally = np.concatenate([tally, np.zeros((B, H, 1))], 2)
        torch.cuda.synchronize()
        assert lens[0].tolist() == [n] * B
        sizes = dict(k_size=3 * np.broadcast_to(np.abs(rows_k).max(-1, keepdims=True), rows_k.shape),
                     v_size=3 * np.broadcast_to(np.abs(rows_v).max(-1, keepdims=True), rows_v.shape)) if q4 else {}
        check_attend(q, rows_k, rows_v, [n] * B, out, score0=before.cpu()[..., :n], score=score.cpu()[..., :n],
                     where=f"step {step}", **sizes)
        for b in range(B):
            for h in range(H):
                for i in range(G):
                    tally[b, h] += co.attend(to64(q)[b, h * G + i], rows_k[b, h], rows_v[b, h])[1]
        # running sums of at most 20 x 4 weights, each within 2^-12 of itself (far above the tolerance above)
        assert np.allclose(to64(score[..., :n]), tally, rtol=2.0 ** -12, atol=0)
        if n == cap:
            if q4:
                lens[1], idx = kv.q4_evict(cache, score, lens[0], lens[1], keep=held - 4, recent=4)
            else:
                lens[1], idx = kv.evict(k_cache, v_cache, score, lens[0], lens[1], keep=held - 4, recent=4)
            lens.reverse()
            torch.cuda.synchronize()
            evictions += 1
            src = idx.cpu().long().numpy()
            # nothing that left weighs more than what stayed; the newest four stay, in order
            for b in range(B):
                for h in range(H):
                    stays = set(src[b, h].tolist())
                    gone = [r for r in range(cap) if r not in stays]
                    assert len(stays) == held and src[b, h, -4:].tolist() == list(range(cap - 4, cap))
                    assert max(tally[b, h, gone]) <= min(tally[b, h, src[b, h, :-4]]) * (1 + 2.0 ** -11)
            take = np.take_along_axis
            rows_k, rows_v = (take(x, src[..., None], 2) for x in (rows_k, rows_v))
            tally = take(tally, src, 2)
            assert lens[0].tolist() == [held] * B and torch.all(score[..., held:] == 0)
    assert evictions == 3
