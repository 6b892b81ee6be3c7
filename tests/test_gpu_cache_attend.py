"""GPU parity of snapkv_decode_attend_scored and snapkv_q4_decode_attend against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests.cache_cases import check_attend, q4_inputs, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(gpu_device):
    import __graft_entry__
    __graft_entry__.build()
    return gpu_device


def dense(g, B, Hq, H, cap, d, dtype, lens, poison=True):
    """q, k, v, len and a score array, on the CPU; rows past a sequence's end hold NaN and infinities."""
    q = (torch.randn(B, Hq, d, generator=g) * 1.5).to(dtype)
    k = torch.randn(B, H, cap, d, generator=g).to(dtype)
    v = torch.randn(B, H, cap, d, generator=g).to(dtype)
    score = torch.rand(B, H, cap, generator=g)
    if poison:
        for b, n in enumerate(lens):
            n = max(0, n)
            k[b, :, n::2], k[b, :, n + 1::2] = float("nan"), float("inf")
            v[b, :, n::2], v[b, :, n + 1::2] = float("-inf"), float("nan")
            score[b, :, n:] = float("nan")
    return q, k, v, torch.tensor(lens, dtype=torch.int32), score


def four_bits(g, B, H, cap, d, lens):
    """A 4-bit cache of normal rows (CPU tensors), its fp64 values and magnitudes; rows past the end hold NaN
    pairs and arbitrary codes."""
    out = {}
    for name in ("k", "v"):
        x = torch.randn(B, H, cap, d, generator=g).bfloat16()
        u, h, z = co.quantise(to64(x))
        codes, meta = q4_inputs(u, h, z)
        for b, n in enumerate(lens):
            codes[b, :, max(0, n):] = 0xA5
            meta[b, :, max(0, n):] = float("nan")
        out[name] = (codes, meta, co.values(u, h, z), co.magnitudes(u, h, z))
    return out


LENS = [0, 1, 15, 16, 17, 33, 64, 65, 127, 200]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 8, 9, 16])
def test_dense_ragged_lengths(dev, dtype, d, G):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(100 * G + d)
    B, H, cap = len(LENS), 2, 200
    q, k, v, n, score = dense(g, B, G * H, H, cap, d, dtype, LENS)
    s = score.to(dev)
    out = kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n.to(dev), s, decay=0.75)
    plain = kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n.to(dev))
    torch.cuda.synchronize()
    assert torch.equal(out, plain)                     # the score does not touch the output
    check_attend(q, to64(k), to64(v), LENS, out, score0=score, score=s.cpu(), decay=0.75, where=f"{dtype} d{d} G{G}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 5, 8, 11])
def test_q4_ragged_lengths(dev, dtype, d, G):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(7 * G + d)
    B, H, cap = len(LENS), 2, 201                       # odd: heads start off 16-byte boundaries of the pairs
    c = four_bits(g, B, H, cap, d, LENS)
    cache = kv.Q4Cache(*(t.to(dev) for t in (*c["k"][:2], *c["v"][:2])))
    q = (torch.randn(B, G * H, d, generator=g) * 1.5).to(dtype)
    score = torch.rand(B, H, cap, generator=g)
    s = score.to(dev)
    n = torch.tensor(LENS, dtype=torch.int32, device=dev)
    out = kv.q4_decode_attend(q.to(dev), cache, n, s)
    plain = kv.q4_decode_attend(q.to(dev), cache, n)
    torch.cuda.synchronize()
    assert torch.equal(out, plain)
    check_attend(q, c["k"][2], c["v"][2], LENS, out, k_size=c["k"][3], v_size=c["v"][3], score0=score, score=s.cpu(),
                 where=f"q4 {dtype} d{d} G{G}")


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("B,H,G,cap,dtype", [
    (1, 1, 1, 40000, torch.bfloat16),        # one head over all CTAs
    (1, 2, 8, 12011, torch.float32),
    (40, 8, 8, 2311, torch.bfloat16),        # many heads in every CTA's share
    (1, 3, 16, 30011, torch.bfloat16),       # sixteen queries a pass
    (300, 1, 1, 70, torch.float32),
])
def test_long_and_wide(dev, q4, B, H, G, cap, dtype):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(cap + G)
    d = 128
    lens = [cap - (7 * b) % 64 for b in range(B)]
    pick = [0] if B > 8 else None
    n = torch.tensor(lens, dtype=torch.int32)
    q = (torch.randn(B, G * H, d, generator=g) * 1.5).to(dtype)
    score = torch.rand(B, H, cap, generator=g)
    s = score.to(dev)
    kx = torch.randn(B, H, cap, d, generator=g).to(dtype)
    vx = torch.randn(B, H, cap, d, generator=g).to(dtype)
    sizes = {}
    if q4:
        cache = kv.Q4Cache.empty(B, H, cap, d, dev)
        kv.q4_append(cache, kx.to(dev), vx.to(dev), torch.zeros(B, dtype=torch.int32, device=dev))
        out = kv.q4_decode_attend(q.to(dev), cache, n.to(dev), s, decay=0.0)
        k64, v64 = (to64(t) for t in kv.q4_read(cache, cap, dtype=torch.float32))
        # |z| + |h t| of a row is at most three times its largest value
        sizes = {name: 3 * np.broadcast_to(np.abs(t).max(-1, keepdims=True), t.shape)
                 for name, t in (("k_size", k64), ("v_size", v64))}
    else:
        out = kv.decode_attend_scored(q.to(dev), kx.to(dev), vx.to(dev), n.to(dev), s, decay=0.0)
        k64, v64 = to64(kx), to64(vx)
    torch.cuda.synchronize()
    rows = range(0, B, max(1, B // 4))
    sel = list(rows)
    check_attend(q[sel], k64[sel], v64[sel], [lens[b] for b in sel], out[sel], score0=score[sel], score=s.cpu()[sel],
                 decay=0.0, heads=pick, where=f"B{B} H{H} G{G} cap{cap}",
                 **{name: t[sel] for name, t in sizes.items()})


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("lens,cap", [
    ([0, 0, 700, 0, 1, 0, 64, 129, 0, 700] * 4 + [0, 0, 0], 700),       # 43 sequences, empty ones at both ends
    ([0] * 5, 400), ([0, 0, 3, 0], 3000), ([300] * 70, 300), ([5, 4000, 17, 0, 3999, 1], 4000)])
def test_schedules_with_empty_and_uneven_sequences(dev, q4, lens, cap):
    """Shares that start and end inside sequences, empty sequences anywhere, fewer tiles than CTAs."""
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(len(lens) + cap)
    B, H, G, d = len(lens), 2, 3, 64
    dtype = torch.bfloat16
    score = torch.rand(B, H, cap, generator=g)
    s = score.to(dev)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    if q4:
        c = four_bits(g, B, H, cap, d, lens)
        q = (torch.randn(B, G * H, d, generator=g) * 1.5).to(dtype)
        out = kv.q4_decode_attend(q.to(dev), kv.Q4Cache(*(t.to(dev) for t in (*c["k"][:2], *c["v"][:2]))), n, s)
        k64, v64, sizes = c["k"][2], c["v"][2], dict(k_size=c["k"][3], v_size=c["v"][3])
    else:
        q, k, v, _, _ = dense(g, B, G * H, H, cap, d, dtype, lens)
        out = kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n, s)
        k64, v64, sizes = to64(k), to64(v), {}
    torch.cuda.synchronize()
    check_attend(q, k64, v64, lens, out, score0=score, score=s.cpu(), where=f"{len(lens)} of {cap}", **sizes)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(dev, seed):
    import random
    import kv_cache_compression_gb300 as kv
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    B, H, G, d = rng.choice([1, 2, 3, 7, 40]), rng.choice([1, 2, 5]), rng.choice([1, 2, 4, 6, 8, 10, 17]), rng.choice([64, 128])
    cap = rng.choice([17, 100, 255, 256, 257, 513, 1000, 2049]) if B < 40 else rng.choice([65, 300])
    dtype, q4, decay = rng.choice([torch.bfloat16, torch.float32]), rng.random() < 0.5, rng.choice([0.0, 0.5, 1.0])
    lens = [rng.choice([0, 1, cap, cap, rng.randrange(cap + 1)]) for _ in range(B)]
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    score = torch.rand(B, H, cap, generator=g)
    s = score.to(dev)
    if q4:
        c = four_bits(g, B, H, cap, d, lens)
        q = (torch.randn(B, G * H, d, generator=g) * 1.5).to(dtype)
        cache = kv.Q4Cache(*(t.to(dev) for t in (*c["k"][:2], *c["v"][:2])))
        out = kv.q4_decode_attend(q.to(dev), cache, n, s, decay=decay)
        k64, v64, sizes = c["k"][2], c["v"][2], dict(k_size=c["k"][3], v_size=c["v"][3])
    else:
        q, k, v, _, _ = dense(g, B, G * H, H, cap, d, dtype, lens)
        out = kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n, s, decay=decay)
        k64, v64, sizes = to64(k), to64(v), {}
    torch.cuda.synchronize()
    check_attend(q, k64, v64, lens, out, score0=score, score=s.cpu(), decay=decay,
                 where=f"seed {seed}: {dtype} q4 {q4} B{B} H{H} G{G} d{d} cap{cap}", **sizes)


def test_one_query_per_head_matches_the_existing_decode(dev):
    """Without a score and with G = 1 the call computes what snapkv_decode_attend computes."""
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(5)
    for dtype in (torch.bfloat16, torch.float32):
        q, k, v, n, _ = dense(g, 3, 4, 4, 500, 128, dtype, [500, 3, 256], poison=False)
        a = kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n.to(dev))
        b = kv.decode_attend(q.to(dev), k.to(dev), v.to(dev), n.to(dev))
        torch.cuda.synchronize()
        for out in (a, b):
            check_attend(q, to64(k), to64(v), n.tolist(), out)


def test_peaked_and_equal_logits(dev):
    """One row takes all weight (the others' weights underflow), or all rows share it."""
    import kv_cache_compression_gb300 as kv
    B, H, cap, d = 1, 1, 300, 64
    q = torch.zeros(B, H, d)
    q[..., 0] = 200.0
    k = torch.zeros(B, H, cap, d)
    k[0, 0, 137, 0] = 50.0
    v = torch.randn(B, H, cap, d, generator=torch.Generator().manual_seed(1))
    s = torch.zeros(B, H, cap, device=dev)
    n = torch.tensor([cap], dtype=torch.int32, device=dev)
    out = kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n, s)
    torch.cuda.synchronize()
    assert torch.equal(out[0, 0].cpu(), v[0, 0, 137])
    assert s[0, 0, 137].item() == 1.0 and s.sum().item() == 1.0
    flat = torch.zeros(B, H, cap, device=dev)
    out = kv.decode_attend_scored(torch.zeros_like(q).to(dev), k.to(dev), v.to(dev), n, flat, decay=0.0)
    torch.cuda.synchronize()
    assert torch.all((flat - 1.0 / cap).abs() <= 2.0 ** -22 / cap)
    check_attend(torch.zeros_like(q), to64(k), to64(v), [cap], out)


def test_nan_in_a_visible_row_reaches_its_head_alone(dev):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(3)
    q, k, v, n, score = dense(g, 2, 4, 2, 100, 64, torch.bfloat16, [100, 60], poison=False)
    k[0, 1, 50, 3] = float("nan")
    out = kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n.to(dev)).cpu()
    assert torch.all(torch.isnan(out[0, 2:])) and torch.all(torch.isfinite(out[0, :2])) and torch.all(torch.isfinite(out[1]))


def test_decay_zero_does_not_read_the_old_score(dev):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(4)
    q, k, v, n, _ = dense(g, 1, 2, 2, 90, 64, torch.float32, [77])
    s = torch.full((1, 2, 90), float("nan"), device=dev)
    kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n.to(dev), s, decay=0.0)
    assert torch.all(torch.isfinite(s[..., :77])) and torch.all(torch.isnan(s[..., 77:]))
    assert torch.allclose(s[..., :77].sum(-1), torch.ones(1, 2, device=dev), atol=1e-5)


def test_lengths_outside_the_cache(dev):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(6)
    q, k, v, _, score = dense(g, 2, 2, 2, 50, 128, torch.bfloat16, [50, 50], poison=False)
    s = score.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    n = torch.tensor([57, -3], dtype=torch.int32, device=dev)
    out = kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n, s, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == kv.snapkv.ERR_CAPACITY
    check_attend(q, to64(k), to64(v), [50, 0], out, score0=score, score=s.cpu())
    assert torch.all(out[1] == 0)


def test_repeats_give_the_same_bits_on_any_stream_and_from_a_graph(dev):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(8)
    q, k, v, n, score = (t.to(dev) for t in dense(g, 2, 8, 2, 3001, 128, torch.bfloat16, [3001, 1700], poison=False))
    want_s = score.clone()
    want = kv.decode_attend_scored(q, k, v, n, want_s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(dev)
    s = score.clone()
    torch.cuda.synchronize()
    out = kv.decode_attend_scored(q, k, v, n, s, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(s, want_s)
    ws = kv.snapkv.new_workspace(kv.scored_workspace_size(2, 8, 2, 128, 3001), dev)
    o = torch.empty_like(q)
    s.copy_(score)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.decode_attend_scored(q, k, v, n, s, out=o, workspace=ws)
    s.copy_(score)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(s, want_s)
    n.fill_(5)                                          # lengths are read on the device at each replay
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, kv.decode_attend_scored(q, k, v, n))


def test_offsets_past_32_bits(dev):
    """A cache whose last heads lie beyond 2^32 bytes."""
    import kv_cache_compression_gb300 as kv
    B, H, cap, d = 1, 24, 800_000, 128
    g = torch.Generator(device=dev).manual_seed(9)
    k = torch.empty(B, H, cap, d, dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    for h in range(H):
        k[0, h].normal_(generator=g)
        v[0, h].normal_(generator=g)
    assert (H - 1) * cap * d * 2 > 1 << 32
    q = torch.randn(B, H, d, generator=g, device=dev).bfloat16()
    lens = [cap - 13]
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    s = torch.zeros(B, H, cap, device=dev)
    out = kv.decode_attend_scored(q, k, v, n, s)
    cache = kv.Q4Cache.empty(B, H, cap, d, dev)
    kv.q4_append(cache, k, v, torch.zeros(1, dtype=torch.int32, device=dev))
    out4 = kv.q4_decode_attend(q, cache, n)
    torch.cuda.synchronize()
    for h in (0, H - 1):
        kk, vv = k[0, h, :lens[0]].double(), v[0, h, :lens[0]].double()
        p = torch.softmax(kk @ q[0, h].double() / d ** 0.5, 0)
        size = (kk.abs() @ q[0, h].double().abs()).max().item() / d ** 0.5
        from tests.cache_cases import out_tolerance, weight_error
        tol = out_tolerance(to64(p @ vv), to64(p @ vv.abs()), d, lens[0], size, torch.bfloat16)
        assert np.all(np.abs(to64(out[0, h]) - to64(p @ vv)) <= tol)
        assert torch.all((s[0, h, :lens[0]].double() - p).abs() <= p * weight_error(d, lens[0], size) + 1e-30)
    k4, v4 = kv.q4_read(cache, 1000, start=torch.tensor([cap - 1000], dtype=torch.int32, device=dev),
                        dtype=torch.float32)
    u, hh, z = co.quantise(to64(k[0, H - 1, cap - 1000:]))
    assert np.array_equal(to64(k4[0, H - 1]), co.values(u, hh, z).astype(np.float32))
    # 4 bits keep a flat average of 800000 normal rows near the dense one: each value moves by at most a step
    # 2h < 0.5, independently, so the average by far less than 0.02
    assert (out4.float() - out.float()).abs().max().item() < 0.02


def test_two_calls_at_once(dev):
    """Two calls on two streams with their own workspaces."""
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(11)
    sets = [tuple(t.to(dev) for t in dense(g, 4, 8, 8, 2000, 128, torch.bfloat16, [2000, 1, 900, 1999], poison=False))
            for _ in range(2)]
    want = []
    for q, k, v, n, score in sets:
        s = score.clone()
        want.append((kv.decode_attend_scored(q, k, v, n, s), s))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in sets]
    for _ in range(5):
        got = []
        scores = [x[4].clone() for x in sets]
        torch.cuda.synchronize()
        for (q, k, v, n, _), s, st in zip(sets, scores, streams):
            with torch.cuda.stream(st):
                got.append((kv.decode_attend_scored(q, k, v, n, s), s))
        torch.cuda.synchronize()
        for (o, s), (wo, ws) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(s, ws)


@pytest.mark.parametrize("q4", [False, True])
def test_buffers_of_a_call_on_another_stream_are_not_reused_early(dev, q4):
    """The workspace that a call on a side stream allocates is free for that stream alone: memory taken and
    overwritten on the current stream right after the call must not be it."""
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(12)
    q, k, v, n, score = (t.to(dev) for t in dense(g, 2, 8, 4, 3000, 64, torch.bfloat16, [3000, 2990], poison=False))
    cache = kv.Q4Cache.empty(2, 4, 3000, 64, dev)
    kv.q4_append(cache, k, v, torch.zeros(2, dtype=torch.int32, device=dev))

    def attend(s, **kw):
        if q4:
            return kv.q4_decode_attend(q, cache, n, s, **kw)
        return kv.decode_attend_scored(q, k, v, n, s, **kw)
    want_s = score.clone()
    want = attend(want_s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(dev)
    need = kv.scored_workspace_size(2, 8, 4, 64, 3000)
    s = score.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                   # some 10 ms: the call's kernels start after what follows
    out = attend(s, stream=side)
    for _ in range(4):
        torch.empty(need, dtype=torch.uint8, device=dev).fill_(0xFF)
        torch.empty_like(q).fill_(7.0)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(s, want_s)


@pytest.mark.parametrize("B,H,G,cap", [
    (12, 5, 6, 9001),     # four rows a thread in the joining kernel
    (2, 1, 40, 3001),     # three passes, two rows a thread
    (1, 1, 70, 300),      # five passes over few tiles
])
def test_joins_of_every_size(dev, B, H, G, cap):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(B + G)
    d, dtype = 64, torch.bfloat16
    lens = [cap - 97 * b for b in range(B)]
    q, k, v, n, score = dense(g, B, G * H, H, cap, d, dtype, lens)
    s = score.to(dev)
    out = kv.decode_attend_scored(q.to(dev), k.to(dev), v.to(dev), n.to(dev), s, decay=0.5)
    torch.cuda.synchronize()
    sel = [0, B - 1]
    check_attend(q[sel], to64(k[sel]), to64(v[sel]), [lens[b] for b in sel], out[sel], score0=score[sel],
                 score=s.cpu()[sel], decay=0.5, heads=[0, H - 1], where=f"B{B} H{H} G{G}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("power", [-40, 0, 44, 55])
def test_large_and_small_queries_over_four_bits(dev, dtype, power):
    """Queries are scaled on their way to the tensor cores; 2^55 is as large as they may be."""
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(power + 50)
    B, H, G, d, cap = 1, 2, 2, 128, 300
    made = {}
    for name, scale in (("k", 2.0 ** -power), ("v", 1.0)):
        x = (torch.randn(B, H, cap, d, generator=g) * scale).bfloat16()
        u, h, z = co.quantise(to64(x))
        made[name] = (*(t.to(dev) for t in q4_inputs(u, h, z)), co.values(u, h, z), co.magnitudes(u, h, z))
    q = (torch.randn(B, G * H, d, generator=g).clamp(-1.9, 1.9) * 2.0 ** power).to(dtype)
    score = torch.zeros(B, H, cap)
    s = score.to(dev)
    n = torch.tensor([cap], dtype=torch.int32, device=dev)
    out = kv.q4_decode_attend(q.to(dev), kv.Q4Cache(*made["k"][:2], *made["v"][:2]), n, s)
    torch.cuda.synchronize()
    check_attend(q, made["k"][2], made["v"][2], [cap], out, k_size=made["k"][3], v_size=made["v"][3], score0=score,
                 score=s.cpu(), where=f"{dtype} 2^{power}")


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("G", [9, 16])
def test_short_bf16_calls_allocate_no_workspace(dev, q4, G):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(G)
    B, H, cap, d, lens = 2, 2, 256, 128, [256, 77]
    q, k, v, n, score = dense(g, B, G * H, H, cap, d, torch.bfloat16, lens, poison=False)
    cache = kv.Q4Cache.empty(B, H, cap, d, dev)
    kv.q4_append(cache, k.to(dev), v.to(dev), torch.zeros(B, dtype=torch.int32, device=dev))
    qd, kd, vd, nd, s = (t.to(dev) for t in (q, k, v, n, score))
    out = torch.empty_like(qd)
    before = torch.cuda.memory_stats(dev)["allocation.all.allocated"]
    if q4:
        kv.q4_decode_attend(qd, cache, nd, s, out=out)
    else:
        kv.decode_attend_scored(qd, kd, vd, nd, s, out=out)
    assert torch.cuda.memory_stats(dev)["allocation.all.allocated"] == before
    torch.cuda.synchronize()
    sizes = {}
    k64, v64 = to64(k), to64(v)
    if q4:
        k64, v64 = (to64(t) for t in kv.q4_read(cache, cap, dtype=torch.float32))
        sizes = {name: 3 * np.broadcast_to(np.abs(t).max(-1, keepdims=True), t.shape) for name, t in (("k_size", k64), ("v_size", v64))}
    check_attend(q, k64, v64, lens, out, score0=score, score=s.cpu(), where=f"q4 {q4} G{G}", **sizes)
