"""Rows appended to dense and 8-bit caches and read out of 8 bits, against the fp64 oracle (include/snapkv_draft.h)."""
import numpy as np
import pytest
import torch

import kv_cache_compression_gb300 as kv
from oracle import draft_oracle as do
from tests.cache_cases import to64

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
SIZES = [(1, 1, 64, 1, 1), (2, 3, 128, 4, 9), (3, 2, 64, 31, 50), (2, 2, 128, 32, 40), (1, 5, 128, 333, 400), (4, 1, 64, 70, 100)]


def rows(seed, B, H, n, d, dtype):
    """Rows of sizes from 2^-30 to 2^30, some zero, some whose largest value makes ties common."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, n, d, generator=g)
    x *= torch.exp2(torch.randint(-30, 31, (B, H, n, 1), generator=g).float())
    kind = torch.randint(0, 6, (B, H, n, 1), generator=g)
    x = torch.where(kind == 0, torch.zeros_like(x), x)
    whole = torch.randint(-254, 255, (B, H, n, d), generator=g).float()
    whole[..., 0] = 254
    x = torch.where(kind == 1, whole * 0.5, x)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_quantised_rows(gpu_device, size, dtype):
    B, H, d, n, cap = size
    k, v = rows(1, B, H, n, d, dtype), rows(2, B, H, n, d, dtype)
    cache = kv.Q8Cache.empty(B, H, cap, d, gpu_device)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0x55)
    for t in (cache.k_step, cache.v_step):
        t.fill_(7.0)
    start = [(cap - n) * b // max(1, B - 1) if B > 1 else cap - n for b in range(B)]
    len_in = torch.tensor(start, dtype=torch.int32, device=gpu_device)
    len_out = kv.q8_append(cache, k.to(gpu_device), v.to(gpu_device), len_in)
    assert len_out.tolist() == [s + n for s in start]
    for x, codes, step in ((k, cache.k_codes, cache.k_step), (v, cache.v_codes, cache.v_step)):
        sign, u, h = do.quantise(to64(x))
        want, want_h = np.full((B, H, cap, d), 0x55, dtype=np.uint8), np.full((B, H, cap), 7.0)
        for b in range(B):
            want[b, :, start[b]:start[b] + n] = do.codes(sign, u)[b]
            want_h[b, :, start[b]:start[b] + n] = h[b]
        got, got_h = codes.cpu().numpy(), to64(step)
        assert np.array_equal(got_h, want_h)
        zero = (want & 127) == 0     # zeros may have either sign
        assert np.array_equal(np.where(zero, got & 127, got), np.where(zero, 0, want))
    for out in (BF16, FP32):
        k_out, v_out = kv.q8_read(cache, n, start=len_in, dtype=out)
        for x, y in ((k, k_out), (v, v_out)):
            sign, u, h = do.quantise(to64(x))
            exact = torch.from_numpy(do.values(do.codes(sign, u), h))
            assert torch.equal(y.cpu(), rounded(exact, out))


def rounded(x, dtype):
    """x fp64 rounded once, to nearest even (not through fp32, which would round twice)."""
    if dtype == FP32:
        return x.float()
    bits = x.view(torch.int64)
    low = bits & ((1 << 45) - 1)
    up = (low > (1 << 44)) | ((low == (1 << 44)) & (((bits >> 45) & 1) == 1))
    bits = (bits - low) + up.to(torch.int64) * (1 << 45)
    return bits.view(torch.float64).to(BF16)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("T,most", [(1, 1), (16, 6), (64, 33), (40, 40), (7, 31)])
def test_picked_rows(gpu_device, T, most, dtype, q8):
    B, H, d, cap = 5, 3, 128, 90
    rng = np.random.default_rng(T)
    k, v = (rows(s, B, H, T, d, dtype).to(gpu_device) for s in (3, 4))
    pick = rng.integers(0, T, size=(B, most)).astype(np.int32)     # repeats among them
    n = np.array([most, 0, most // 2, 1, most], dtype=np.int32)
    start = np.array([0, 5, cap - most // 2, cap - 1, cap - most], dtype=np.int32)
    pick[1], pick[2, most // 2:] = -1, T       # not looked at
    args = dict(pick=torch.from_numpy(pick).to(gpu_device), n_new=torch.from_numpy(n).to(gpu_device))
    len_in = torch.from_numpy(start).to(gpu_device)
    status = torch.zeros(1, dtype=torch.int32, device=gpu_device)
    if q8:
        cache = kv.Q8Cache.empty(B, H, cap, d, gpu_device)
        cache.k_step.fill_(0)
        cache.v_step.fill_(0)
        before = [t.clone() for t in (cache.k_codes, cache.v_codes)]
        len_out = kv.q8_append(cache, k, v, len_in, dev_status=status, **args)
        after = [cache.k_codes, cache.v_codes]
        new = [torch.from_numpy(do.codes(*do.quantise(to64(x))[:2])) for x in (k, v)]
    else:
        held = [rows(s, B, H, cap, d, dtype).to(gpu_device) for s in (5, 6)]
        before = [t.clone() for t in held]
        len_out = kv.append_rows(*held, k, v, len_in, dev_status=status, **args)
        after, new = held, [k.cpu(), v.cpu()]
    assert status.item() == 0 and len_out.tolist() == (start + n).tolist()
    for old, now, x in zip(before, after, new):
        for b in range(B):
            for h in range(H):
                want = do.append(old[b, h].float().cpu().numpy(), x[b, h].float().numpy(), pick[b], int(n[b]), int(start[b]))
                got = now[b, h].float().cpu().numpy()
                if q8:
                    want, got = (np.where(t % 128 == 0, 0, t) for t in (want, got))
                assert np.array_equal(got, want), f"b{b} h{h}"


@pytest.mark.parametrize("rows_n", [4, 40])
def test_sequences_that_cannot_take_their_rows_are_left_alone(gpu_device, rows_n):
    B, H, d, cap = 6, 2, 64, 50
    k, v = (rows(s, B, H, rows_n, d, BF16).to(gpu_device) for s in (3, 4))
    held = [rows(s, B, H, cap, d, BF16).to(gpu_device) for s in (5, 6)]
    before = [t.clone() for t in held]
    len_in = torch.tensor([cap - rows_n + 1, -1, 0, 0, 0, 0], dtype=torch.int32, device=gpu_device)
    n = torch.tensor([rows_n, 1, rows_n + 1, -1, rows_n, 2], dtype=torch.int32, device=gpu_device)
    pick = torch.zeros(B, rows_n, dtype=torch.int32, device=gpu_device)
    pick[4, rows_n - 1] = rows_n
    pick[5, 1] = -1
    for b, code in ((0, kv.snapkv.ERR_CAPACITY), (1, kv.snapkv.ERR_CAPACITY), (2, kv.snapkv.ERR_INVALID_ARG),
                    (3, kv.snapkv.ERR_INVALID_ARG), (4, kv.snapkv.ERR_INVALID_ARG), (5, kv.snapkv.ERR_INVALID_ARG)):
        status = torch.zeros(1, dtype=torch.int32, device=gpu_device)
        only = [t[b:b + 1].contiguous() for t in (*held, k, v, len_in)]
        out = kv.append_rows(*only, n_new=n[b:b + 1].contiguous(), pick=pick[b:b + 1].contiguous(), dev_status=status)
        assert status.item() == code and out.tolist() == [len_in[b].item()], b
        assert all(torch.equal(x, y[b:b + 1]) for x, y in zip(only, before)), b
    status = torch.zeros(1, dtype=torch.int32, device=gpu_device)
    assert torch.equal(kv.append_rows(*held, k, v, len_in, n_new=n, pick=pick, dev_status=status), len_in)
    assert status.item() == kv.snapkv.ERR_CAPACITY | kv.snapkv.ERR_INVALID_ARG
    assert all(torch.equal(x, y) for x, y in zip(held, before))


def test_rows_that_are_not_finite_read_back_as_nan(gpu_device):
    x = torch.full((1, 1, 4, 64), 127.0)   # (a step of one)
    x[0, 0, 1, 5], x[0, 0, 2, 63], x[0, 0, 3, 0] = float("inf"), float("nan"), 3e38
    for dtype in (FP32, BF16):
        cache = kv.Q8Cache.empty(1, 1, 6, 64, gpu_device)
        zero = torch.zeros(1, dtype=torch.int32, device=gpu_device)
        kv.q8_append(cache, x.to(dtype).to(gpu_device), x.to(dtype).to(gpu_device), zero)
        k, _ = kv.q8_read(cache, 4, dtype=FP32)
        assert torch.equal(k[0, 0, 0].cpu(), x[0, 0, 0]) and torch.isnan(k[0, 0, 1:3]).all()
        assert torch.isfinite(k[0, 0, 3]).all()
        k, v = kv.q8_read(cache, 4, start=zero + 5)
        assert not k[0, 0, 1:].any() and not v[0, 0, 1:].any()
        k, _ = kv.q8_read(cache, 2, start=zero - 1, dtype=FP32)
        assert not k[0, 0, 0].any() and torch.equal(k[0, 0, 1].cpu(), x[0, 0, 0])
