"""GPU parity of snapkv_q4_append and snapkv_q4_read against the oracle's format, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests.cache_cases import q4_inputs, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(gpu_device):
    import __graft_entry__
    __graft_entry__.build()
    return gpu_device


def filled(kv, B, H, cap, d, dev):
    """A cache of recognisable bytes, to see what a call leaves alone."""
    c = kv.Q4Cache.empty(B, H, cap, d, dev)
    for i, t in enumerate((c.k_codes, c.v_codes)):
        t.fill_(0x11 * (i + 1))
    for i, t in enumerate((c.k_meta, c.v_meta)):
        t.fill_(1.0 + i)
    return c


def check_rows(cache, before, k, v, starts, counts):
    """Rows starts[b] .. + counts[b] - 1 hold the quantised first rows of k, v; all others what they held."""
    B = k.shape[0]
    for x, codes, meta, codes0, meta0 in ((k, cache.k_codes, cache.k_meta, before[0], before[1]),
                                          (v, cache.v_codes, cache.v_meta, before[2], before[3])):
        want_codes, want_meta = codes0.cpu().clone(), meta0.cpu().clone()
        for b in range(B):
            if counts[b]:
                u, h, z = co.quantise(to64(x[b, :, :counts[b]]))
                c, m = q4_inputs(u, h, z)
                want_codes[b, :, starts[b]:starts[b] + counts[b]] = c
                want_meta[b, :, starts[b]:starts[b] + counts[b]] = m
        got, want = meta.cpu().float(), want_meta.float()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got, 7.0), torch.nan_to_num(want, 7.0))
        assert torch.equal(codes.cpu(), want_codes)


def snapshot(c):
    return [t.clone() for t in (c.k_codes, c.k_meta, c.v_codes, c.v_meta)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 5, 16, 33])
def test_rows_are_written_where_they_belong(dev, dtype, d, rows):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(rows + d)
    B, H, cap = 5, 3, 50
    starts = [0, 1, 7, cap - rows, cap - rows + 1]       # the last does not fit
    k = (torch.randn(B, H, rows, d, generator=g) * 3).to(dtype)
    v = (torch.randn(B, H, rows, d, generator=g) + 1).to(dtype)
    cache = filled(kv, B, H, cap, d, dev)
    before = snapshot(cache)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    lens = torch.tensor(starts, dtype=torch.int32, device=dev)
    out = kv.q4_append(cache, k.to(dev), v.to(dev), lens, dev_status=status)
    torch.cuda.synchronize()
    assert out.tolist() == [s + rows for s in starts[:-1]] + [starts[-1]]
    assert lens.tolist() == starts and status.item() == kv.snapkv.ERR_CAPACITY
    check_rows(cache, before, k, v, starts, [rows] * 4 + [0])
    if rows == 1:                                        # [B, H, d] is one row
        again = filled(kv, B, H, cap, d, dev)
        kv.q4_append(again, k[:, :, 0].contiguous().to(dev), v[:, :, 0].contiguous().to(dev), lens)
        torch.cuda.synchronize()
        assert torch.equal(again.k_codes, cache.k_codes) and torch.equal(again.v_meta, cache.v_meta)


def test_ragged_counts(dev):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(1)
    B, H, cap, d, rows = 6, 2, 40, 128, 20
    starts, counts = [0, 3, 30, 39, -1, 5], [20, 0, 10, 2, 4, 21]
    k, v = (torch.randn(B, H, rows, d, generator=g).bfloat16() for _ in range(2))
    cache = filled(kv, B, H, cap, d, dev)
    before = snapshot(cache)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = kv.q4_append(cache, k.to(dev), v.to(dev), torch.tensor(starts, dtype=torch.int32, device=dev),
                       n_new=torch.tensor(counts, dtype=torch.int32, device=dev), dev_status=status)
    torch.cuda.synchronize()
    # sequence 3 does not fit, 4 has a negative length, 5 asks for more rows than there are
    assert out.tolist() == [20, 3, 40, 39, -1, 5]
    assert status.item() == kv.snapkv.ERR_CAPACITY | kv.snapkv.ERR_INVALID_ARG
    check_rows(cache, before, k, v, starts, [20, 0, 10, 0, 0, 0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_groups_where_rounding_is_hard(dev, dtype):
    """Constant groups, ties, tiny and large steps, offsets much larger than the spread, and non-finite ones."""
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(2)
    rows = []
    for i in range(64):
        base = torch.randn(128, generator=g)
        # small whole multiples of one step: (x - z) / (2h) is often exactly half-way
        rows.append(torch.randint(-15, 16, (128,), generator=g) * 0.25)
        rows.append(torch.randint(-30, 31, (128,), generator=g) * 2.0 ** -7)
        rows.append(base * 2.0 ** (i - 32))
        rows.append(100.0 + base * 2.0 ** -(i % 8))
        rows.append(torch.full((128,), float(base[0])))
        # magnitudes far apart: the difference to the centre is rounded, a border may lie at zero
        rows.append(base * 10.0 ** torch.randint(-6, 2, (128,), generator=g))
        rows.append(torch.where(base > 0, base, base * 2.0 ** -30))
        rows.append(torch.where(torch.arange(128) == i, base[0] * 1e-30, torch.zeros(128)))
        rows.append(torch.where(torch.arange(128) == 2 * i, torch.tensor(float("nan")), base))
        rows.append(torch.where(torch.arange(128) == i, torch.tensor(float("-inf")), base))
    k = torch.stack(rows).to(dtype)[None, None]
    v = (k * -1.0).to(dtype)
    n = k.shape[2]
    cache = filled(kv, 1, 1, n + 3, 128, dev)
    before = snapshot(cache)
    kv.q4_append(cache, k.to(dev), v.to(dev), torch.tensor([2], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    check_rows(cache, before, k, v, [2], [n])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_random_rows_match_bit_for_bit(dev, dtype):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(3)
    B, H, rows, d = 2, 4, 5003, 128
    k = torch.randn(B, H, rows, d, generator=g).to(dtype)
    v = (torch.randn(B, H, rows, d, generator=g) * torch.rand(B, H, rows, 1, generator=g) * 8).to(dtype)
    cache = filled(kv, B, H, rows, d, dev)
    before = snapshot(cache)
    kv.q4_append(cache, k.to(dev), v.to(dev), torch.zeros(B, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    check_rows(cache, before, k, v, [0, 0], [rows, rows])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_read_returns_the_values_and_zeros_outside(dev, dtype, d):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(4)
    B, H, cap = 3, 2, 37
    k, v = (torch.randn(B, H, cap, d, generator=g).bfloat16() for _ in range(2))
    cache = kv.Q4Cache.empty(B, H, cap, d, dev)
    kv.q4_append(cache, k.to(dev), v.to(dev), torch.zeros(B, dtype=torch.int32, device=dev))
    starts, rows = [0, -4, 30], 20
    got = kv.q4_read(cache, rows, start=torch.tensor(starts, dtype=torch.int32, device=dev), dtype=dtype)
    whole = kv.q4_read(cache, cap, dtype=dtype)
    torch.cuda.synchronize()
    for x, part, full in ((k, got[0], whole[0]), (v, got[1], whole[1])):
        val = torch.from_numpy(co.values(*co.quantise(to64(x))).astype(np.float32)).to(dtype)
        assert torch.equal(full.cpu(), val)
        for b, s in enumerate(starts):
            for r in range(rows):
                want = val[b, :, s + r] if 0 <= s + r < cap else torch.zeros(H, d, dtype=dtype)
                assert torch.equal(part[b, :, r].cpu(), want), (b, r)


def test_append_and_read_from_a_graph_on_a_side_stream(dev):
    import kv_cache_compression_gb300 as kv
    g = torch.Generator().manual_seed(5)
    B, H, cap, d = 2, 2, 12, 64
    cache = kv.Q4Cache.empty(B, H, cap, d, dev)
    new = torch.zeros(B, H, d, device=dev)
    lens = [torch.zeros(B, dtype=torch.int32, device=dev) for _ in range(2)]
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):           # two steps: the length arrays alternate
        kv.q4_append(cache, new, new, lens[0], lens[1])
        kv.q4_append(cache, new, new, lens[1], lens[0])
    rows = torch.randn(cap // 2, B, H, d, generator=g)
    for r in rows:
        new.copy_(r)
        graph.replay()
    k, v = kv.q4_read(cache, cap, dtype=torch.float32)
    torch.cuda.synchronize()
    assert lens[0].tolist() == [cap, cap]
    want = torch.from_numpy(co.values(*co.quantise(rows.double().numpy()))).float()
    for i in range(cap):
        assert torch.equal(k[:, :, i].cpu(), want[i // 2]) and torch.equal(v[:, :, i].cpu(), want[i // 2])
