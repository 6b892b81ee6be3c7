"""The operators for drafted tokens at the largest batches that a call may have, beyond 2^32 bytes, and with many tokens."""
import numpy as np
import pytest
import torch

import kv_cache_compression_gb300 as kv
from tests.cache_cases import to64
from tests.draft_cases import check_tree
from tests.test_gpu_tree import BF16, FP32, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("cap,G,T", [(5, 1, 1), (270, 1, 2), (140, 3, 6)])
def test_the_largest_batch(gpu_device, cap, G, T, q8):
    B, H, d = 65535, 1, 64
    if B * G * T > 1 << 22:
        pytest.skip("more rows than a call takes")
    g = torch.Generator(device=gpu_device).manual_seed(cap)
    k, v = (torch.randn(B, H, cap, d, generator=g, device=gpu_device).bfloat16() for _ in "kv")
    kn, vn = (torch.randn(B, H, T, d, generator=g, device=gpu_device).bfloat16() for _ in "kv")
    q = torch.randn(B, G, T, d, generator=g, device=gpu_device).bfloat16()
    n = torch.randint(0, cap + 1, (B,), generator=g, device=gpu_device, dtype=torch.int32)
    n[0], n[-1] = cap, cap
    some = [0, 1, 255, 256, 32768, 65279, 65533, 65534]
    if q8:
        cache = kv.Q8Cache.empty(B, H, cap, d, gpu_device)
        assert torch.equal(kv.q8_append(cache, k, v, torch.zeros_like(n)), torch.full_like(n, cap))
        out = kv.q8_tree_attend(q, cache, n, kn, vn)
        k, v = kv.q8_read(cache, cap, dtype=FP32)
    else:
        out = kv.tree_attend(q, k, v, n, kn, vn)
    check_tree(q[some].cpu(), to64(k[some]), to64(v[some]), n[some].tolist(), out[some].cpu(), k_new=kn[some].cpu(), v_new=vn[some].cpu())
    held = kv.append_rows(k, v, kn.to(k.dtype), vn.to(k.dtype), (n - T).clamp_min(0))
    assert torch.equal(held, (n - T).clamp_min(0) + T) or cap < T
    b = 65534
    assert torch.equal(k[b, 0, cap - T:cap], kn[b, 0].to(k.dtype))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T", [3, 40])
def test_beyond_four_gigabytes(gpu_device, T, q8):
    B, H, d, cap = 3, 1, 128, (1 << 24) + 3
    lens = [5, 0, cap - 60]
    g = torch.Generator(device=gpu_device).manual_seed(T)
    kn, vn = (torch.randn(B, H, T, d, generator=g, device=gpu_device).bfloat16() for _ in "kv")
    q = torch.randn(B, H, T, d, generator=g, device=gpu_device).bfloat16()
    start = torch.tensor(lens, dtype=torch.int32, device=gpu_device)
    if q8:
        cache = kv.Q8Cache.empty(B, H, cap, d, gpu_device)
        for t in (cache.k_codes, cache.v_codes, cache.k_step, cache.v_step):
            t.zero_()
        n = kv.q8_append(cache, kn, vn, start)
        k, v = kv.q8_read(cache, T, start=start, dtype=FP32)   # (what the rows stand for, not rounded to bf16)
        out = kv.q8_tree_attend(q, cache, torch.tensor([40, T, 7], dtype=torch.int32, device=gpu_device), kn, vn)
        far = kv.q8_tree_attend(q, cache, n)
    else:
        keys, values = (torch.zeros(B, H, cap, d, device=gpu_device, dtype=BF16) for _ in "kv")
        n = kv.append_rows(keys, values, kn, vn, start)
        k, v = (torch.stack([t[b, :, s:s + T] for b, s in enumerate(lens)]) for t in (keys, values))
        assert torch.equal(k, kn) and torch.equal(v, vn)
        out = kv.tree_attend(q, keys, values, torch.tensor([40, T, 7], dtype=torch.int32, device=gpu_device), kn, vn)
        far = kv.tree_attend(q, keys, values, n)
    assert n.tolist() == [s + T for s in lens]
    near = np.zeros((2, B, H, 40, d))     # the caches' first 40 rows, as far as they are asked for
    for i, t in enumerate((k, v)):
        near[i, 0, :, 5:5 + min(T, 35)] = to64(t[0])[:, :35]
        near[i, 1, :, :T] = to64(t[1])
    check_tree(q.cpu(), near[0], near[1], [40, T, 7], out.cpu(), k_new=kn.cpu(), v_new=vn.cpu())
    # all rows of the third cache: zeros, whose logits are 0, and the appended ones
    kk, vv, qq = to64(k[2, 0]), to64(v[2, 0]), to64(q[2, 0])
    s = qq @ kk.T / d ** 0.5
    w = np.exp(s)
    ref = w @ vv / (w.sum(1) + lens[2])[:, None]
    err = np.abs(to64(far[2, 0]) - ref)
    # the zeros' 2^24 weights of one are summed up exactly; the others' errors are those of the weights, and a sum of tiles
    # cut by tensor cores loses 2^-23 of itself at each of its additions at most
    size = (w @ np.abs(vv)) / (w.sum(1) + lens[2])[:, None]
    assert np.all(err <= 2.0 ** -8 * (np.abs(ref) + 2 * size) + 2.0 ** -14 * size + 1e-37)


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_many_tokens(gpu_device, dtype):
    """Several passes side by side, and more than one tile of drafted rows."""
    for B, H, G, d, T, cap, lens, n_new in ((1, 1, 2, 64, 700, 500, [333], None), (2, 1, 1, 128, 600, 130, [130, 0], [600, 513]),
                                            (1, 2, 1, 64, 1100, 60, [60], None)):
        x = make(gpu_device, T, B, H, G, d, T, cap, dtype)
        out, lse = run(x, lens, n_new=n_new)
        some = [0, 1, T // 2, (n_new or [T])[0] - 1]
        k64, v64 = x["k64"], x["v64"]
        kn, vn, q = to64(x["k_new"]), to64(x["v_new"]), to64(x["q"])
        for b in range(B):
            for i in range(H * G):
                for t in some:
                    if n_new and t >= n_new[b]:
                        assert not out[b, i, t].any()
                        continue
                    kk = np.concatenate([k64[b, i // G, :lens[b]], kn[b, i // G, :t + 1]])
                    vv = np.concatenate([v64[b, i // G, :lens[b]], vn[b, i // G, :t + 1]])
                    s = kk @ q[b, i, t] / d ** 0.5
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    tol = 2.0 ** -7 * (np.abs(p @ vv) + p @ np.abs(vv)) if dtype == BF16 else 1e-5 * (p @ np.abs(vv)) + 1e-30
                    assert np.all(np.abs(to64(out[b, i, t]) - p @ vv) <= tol), (b, i, t)
                    assert abs(lse[b, i, t].item() - (s.max() + np.log(np.exp(s - s.max()).sum()))) < 1e-4
