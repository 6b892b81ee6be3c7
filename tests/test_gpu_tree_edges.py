"""Tree attention where it can go wrong: masks that leave rows empty, values that are not finite in places that nobody sees, maxima that
grow, lengths and counts out of range, streams and graphs (include/snapkv_draft.h)."""
import numpy as np
import pytest
import torch

import kv_cache_compression_gb300 as kv
from kv_cache_compression_gb300 import snapkv as sk
from tests.cache_cases import to64
from tests.draft_cases import check_tree, random_tree
from tests.test_gpu_tree import BF16, FP32, check, make, run

pytestmark = pytest.mark.gpu

# one of every kernel: (dtype, 8-bit, G, T)
KINDS = [(FP32, False, 2, 3), (FP32, True, 4, 9), (BF16, False, 1, 5), (BF16, False, 3, 5), (BF16, True, 2, 4), (BF16, True, 2, 12),
         (BF16, False, 2, 20), (BF16, True, 4, 20), (BF16, False, 4, 50), (BF16, True, 3, 70)]
kinds = pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{str(k[0])[6:]}-{'q8' if k[1] else 'dense'}-{k[2]}x{k[3]}")


def same(a, b):
    return torch.equal(a.view(torch.int32 if a.dtype == FP32 else torch.int16), b.view(torch.int32 if b.dtype == FP32 else torch.int16))


@kinds
@pytest.mark.parametrize("d", [64, 128])
def test_masks_that_leave_rows_empty(gpu_device, kind, d):
    dtype, q8, G, T = kind
    B, H, cap = 3, 2, 300
    x = make(gpu_device, 21, B, H, G, d, T, cap, dtype, q8=q8)
    rng = np.random.default_rng(5)
    mask = rng.random((B, T, T)) < 0.4            # any pattern, not only trees: rows may see later tokens, or none
    mask[0, 0] = False
    mask[1] = False
    mask[2, T // 2] = False
    for lens, n_new in (([0, 0, 0], None), ([0, 130, 300], None), ([0, 1, 0], [T, 0, max(1, T // 2)])):
        out, lse = run(x, lens, mask=mask, n_new=n_new)
        check(x, lens, out, lse, mask=mask, n_new=n_new)
    assert not run(x, [0, 0, 0], mask=mask)[0][1].any()


@kinds
def test_one_mask_for_all_and_masks_of_bytes(gpu_device, kind):
    dtype, q8, G, T = kind
    B, H, d, cap = 2, 2, 64, 200
    x = make(gpu_device, 22, B, H, G, d, T, cap, dtype, q8=q8)
    one = random_tree(np.random.default_rng(1), 1, T)[0]
    out, lse = run(x, [200, 77], mask=one)
    check(x, [200, 77], out, lse, mask=np.stack([one, one]))
    many = (one.astype(np.uint8) * np.random.default_rng(2).integers(1, 256, size=(B, T, T))).astype(np.uint8)
    again, lse2 = run(x, [200, 77], mask=many)
    assert same(out, again) and same(lse, lse2)
    causal, lse3 = run(x, [200, 77], mask=np.tril(np.ones((T, T), dtype=bool)))
    none, lse4 = run(x, [200, 77])
    assert same(causal, none) and same(lse3, lse4)


@kinds
@pytest.mark.parametrize("d", [64, 128])
def test_what_lies_behind_the_rows_is_not_used(gpu_device, kind, d):
    """NaN and infinities behind the cached rows, behind the drafted ones and in their steps."""
    dtype, q8, G, T = kind
    B, H, cap = 2, 2, 420
    x = make(gpu_device, 23, B, H, G, d, T, cap, dtype, q8=q8)
    lens, n_new = [131, 300], [T, max(1, T - 2)]
    mask = random_tree(np.random.default_rng(3), B, T)
    want, lse = run(x, lens, mask=mask, n_new=n_new)
    check(x, lens, want, lse, mask=mask, n_new=n_new)
    dirty = dict(x)
    for name in ("k", "v"):
        for b in range(B):
            if q8:
                dirty[name + "_step"] = dirty[name + "_step"].clone()
                dirty[name + "_codes"] = dirty[name + "_codes"].clone()
                dirty[name + "_step"][b, :, lens[b]:] = torch.tensor([float("nan"), float("inf"), -float("inf")], device=gpu_device).repeat(200)[:cap - lens[b]]
                dirty[name + "_codes"][b, :, lens[b]:] = 255
            else:
                dirty[name] = dirty[name].clone()
                dirty[name][b, :, lens[b]:] = float("nan")
                dirty[name][b, :, lens[b]::2] = float("inf")
            dirty[name + "_new"] = dirty[name + "_new"].clone()
            dirty[name + "_new"][b, :, n_new[b]:] = float("nan")
    dirty["q"] = x["q"].clone()
    for b in range(B):
        dirty["q"][b, :, n_new[b]:] = float("nan")
    got, lse2 = run(dirty, lens, mask=mask, n_new=n_new)
    assert same(want, got) and same(lse, lse2)


@kinds
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_drafted_row_that_is_not_finite_reaches_those_alone_that_see_it(gpu_device, kind, bad, where):
    dtype, q8, G, T = kind
    if T < 3:
        pytest.skip("needs branches")
    B, H, d, cap = 1, 2, 128, 150
    x = make(gpu_device, 24, B, H, G, d, T, cap, dtype, q8=q8)
    mask = random_tree(np.random.default_rng(4), B, T)
    row = T // 2
    want, lse = run(x, [150], mask=mask)
    dirty = dict(x)
    dirty[where + "_new"] = x[where + "_new"].clone()
    dirty[where + "_new"][0, 1, row, 5] = bad
    got, lse2 = run(dirty, [150], mask=mask)
    sees = torch.from_numpy(mask[0, :, row]).to(gpu_device)
    o, w = got.view(H, G, T, d), want.view(H, G, T, d)
    assert same(o[0].contiguous(), w[0].contiguous())                         # another head
    assert same(o[1][:, ~sees].contiguous(), w[1][:, ~sees].contiguous())     # tokens that do not see it
    assert same(lse2.view(H, G, T)[1][:, ~sees].contiguous(), lse.view(H, G, T)[1][:, ~sees].contiguous())
    hit = o[1][:, sees]
    if where == "v" and dtype == FP32:
        assert not torch.isfinite(hit[..., 5]).any()
    elif where == "v":
        assert torch.isnan(hit).all()
    elif bad != bad:
        assert torch.isnan(hit).all()


@kinds
@pytest.mark.parametrize("scale", [0.0, 60.0])
def test_flat_and_steep_weights(gpu_device, kind, scale):
    dtype, q8, G, T = kind
    x = make(gpu_device, 25, 2, 1, G, 64, T, 900, dtype, q8=q8, scale=scale)
    out, lse = run(x, [900, 333])
    check(x, [900, 333], out, lse)


@kinds
@pytest.mark.parametrize("grow", [0.02, 0.2, -0.2])
def test_maxima_that_grow_and_fall(gpu_device, kind, grow):
    """Keys whose logits rise (or fall) from row to row: every tile raises the maximum, by little or by much."""
    dtype, q8, G, T = kind
    B, H, d, cap = 1, 2, 128, 1700
    x = make(gpu_device, 26, B, H, G, d, T, cap, dtype, q8=q8)
    g = torch.Generator().manual_seed(2)
    way = torch.randn(H, 1, d, generator=g).to(dtype)
    q = (way.double()[:, None] + 0.1 * torch.randn(H, G, T, d, generator=g).double()).reshape(1, H * G, T, d).to(dtype)
    x["q"] = q.to(gpu_device)
    ramp = (torch.arange(cap) * grow / d ** 0.5).view(1, 1, cap, 1)
    k = (way.double()[None] * ramp + 0.3 * torch.randn(B, H, cap, d, generator=g)).to(dtype)
    if q8:
        from tests.draft_cases import q8_rows
        code, step, x["k64"] = q8_rows(k.double().numpy())
        x["k_codes"], x["k_step"] = code.to(gpu_device), step.to(gpu_device)
    else:
        x["k"], x["k64"] = k.to(gpu_device), k.double().numpy()
    out, lse = run(x, [cap])
    check(x, [cap], out, lse)


@kinds
def test_lengths_and_counts_out_of_range_are_clamped_and_reported(gpu_device, kind):
    dtype, q8, G, T = kind
    B, H, d, cap = 4, 1, 64, 290
    x = make(gpu_device, 27, B, H, G, d, T, cap, dtype, q8=q8)
    status = torch.zeros(1, dtype=torch.int32, device=gpu_device)
    out, lse = run(x, [cap + 5, -3, 40, 12], n_new=[T, T, -1, 1], dev_status=status)
    check(x, [cap, 0, 40, 12], out, lse, n_new=[T, T, 0, 1])
    assert status.item() == sk.ERR_CAPACITY | sk.ERR_INVALID_ARG
    status.zero_()
    run(x, [cap, 0, 40, 12], n_new=[T, 1, 0, T + 1], dev_status=status)
    assert status.item() == sk.ERR_INVALID_ARG
    status.zero_()
    run(x, [1 << 30, 0, 40, 12], dev_status=status)
    assert status.item() == sk.ERR_CAPACITY


@kinds
@pytest.mark.parametrize("cap", [100, 600])
def test_streams_and_graphs(gpu_device, kind, cap):
    dtype, q8, G, T = kind
    B, H, d = 2, 2, 128
    x = make(gpu_device, 28, B, H, G, d, T, cap, dtype, q8=q8)
    lens = torch.tensor([cap, cap // 3], dtype=torch.int32, device=gpu_device)
    cache = kv.Q8Cache(x["k_codes"], x["k_step"], x["v_codes"], x["v_step"]) if q8 else None

    def call(**kw):
        if q8:
            return kv.q8_tree_attend(x["q"], cache, lens, x["k_new"], x["v_new"], **kw)
        return kv.tree_attend(x["q"], x["k"], x["v"], lens, x["k_new"], x["v_new"], **kw)

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert same(want, got)
    # two graphs, a workspace each, replayed on two streams at once, and again after the inputs have changed
    graphs = []
    for _ in range(2):
        ws = torch.empty(max(1, kv.tree_workspace_size(B, H * G, H, d, T, cap)), dtype=torch.uint8, device=gpu_device)
        out, lse = torch.empty_like(x["q"]), torch.empty(x["q"].shape[:3], device=gpu_device)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out=out, lse=lse, workspace=ws)
        graphs.append((graph, out, torch.cuda.Stream(), ws))
    for change in (False, True):
        if change:
            lens.copy_(torch.tensor([cap // 2, 0], dtype=torch.int32))
            x["q"].mul_(0.5)
            want = call()
        torch.cuda.synchronize()
        for graph, out, stream, _ in graphs:
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for _, out, _, _ in graphs:
            assert same(want, out)


def test_a_workspace_that_is_too_small_is_refused(gpu_device):
    x = make(gpu_device, 29, 1, 2, 1, 64, 4, 400, BF16)
    ws = torch.empty(kv.tree_workspace_size(1, 2, 2, 64, 4, 400) - 1, dtype=torch.uint8, device=gpu_device)
    with pytest.raises(sk.SnapKVError):
        run(x, [400], workspace=ws)


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes(gpu_device, seed):
    rng = np.random.default_rng(1000 + seed)
    dtype, q8 = (BF16, BF16, FP32)[rng.integers(3)], bool(rng.integers(2))
    B, H, G, d = int(rng.integers(1, 6)), int(rng.integers(1, 5)), int(rng.choice([1, 2, 3, 4, 7])), int(rng.choice([64, 128]))
    T = int(np.exp(rng.uniform(0, np.log(90))))
    cap = int(np.exp(rng.uniform(0, np.log(2500))))
    drafts = rng.random() < 0.8
    x = make(gpu_device, seed, B, H, G, d, T, cap, dtype, q8=q8)
    lens = [int(rng.integers(0, cap + 1)) if rng.random() < 0.8 else cap for _ in range(B)]
    n_new = [int(rng.integers(0, T + 1)) for _ in range(B)] if rng.random() < 0.5 else None
    mask = random_tree(rng, B, T) if drafts and rng.random() < 0.7 else None
    out, lse = run(x, lens, drafts=drafts, mask=mask, n_new=n_new)
    check(x, lens, out, lse, drafts=drafts, mask=mask, n_new=n_new, heads=[int(rng.integers(H))], where=f"seed {seed}")


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("T", [4, 24])
def test_a_run_of_speculative_decoding(gpu_device, T, q8):
    """A compressed prompt, and steps that draft a tree, attend, and append an accepted path: every step's attention is that of
    the rows that were accepted so far."""
    B, H, G, d = 2, 2, 2, 128
    g = torch.Generator().manual_seed(11)
    k, v = (torch.randn(B, H, 700, d, generator=g).bfloat16().to(gpu_device) for _ in "kv")
    q_obs = torch.randn(B, H, 16, d, generator=g).bfloat16().to(gpu_device)
    cap = 260
    res = kv.compress(q_obs, k, v, pool_kernel=5, budget=150, cap=cap)
    held = 150 + 16
    if q8:
        cache = kv.Q8Cache.empty(B, H, cap, d, gpu_device)
        n = kv.q8_append(cache, res["k_out"][:, :, :held].contiguous(), res["v_out"][:, :, :held].contiguous(),
                         torch.zeros(B, dtype=torch.int32, device=gpu_device))
    else:
        keys, values = res["k_out"], res["v_out"]
        n = res["len"].clone()
    assert n.tolist() == [held] * B
    rng = np.random.default_rng(12)
    length = [held] * B
    for step in range(8):
        q = torch.randn(B, H * G, T, d, generator=g).bfloat16().to(gpu_device)
        new = [torch.randn(B, H, T, d, generator=g).bfloat16().to(gpu_device) for _ in "kv"]
        mask = random_tree(rng, B, T)
        m = torch.from_numpy(mask).to(gpu_device)
        if q8:
            out = kv.q8_tree_attend(q, cache, n, *new, m)
            now = kv.q8_read(cache, cap, dtype=torch.float32)
        else:
            out = kv.tree_attend(q, keys, values, n, *new, m)
            now = keys, values
        check_tree(q, to64(now[0]), to64(now[1]), length, out, k_new=new[0], v_new=new[1], mask=mask, where=f"step {step}")
        paths = [np.flatnonzero(mask[b, rng.integers(T)]) for b in range(B)]        # a token and its ancestors
        most = max(map(len, paths))
        pick = np.zeros((B, most), dtype=np.int32)
        for b, p in enumerate(paths):
            pick[b, :len(p)] = p
        args = dict(pick=torch.from_numpy(pick).to(gpu_device),
                    n_new=torch.tensor([len(p) for p in paths], dtype=torch.int32, device=gpu_device))
        if q8:
            n = kv.q8_append(cache, *new, n, **args)
        else:
            n = kv.append_rows(keys, values, *new, n, **args)
            for b, p in enumerate(paths):
                for h in range(H):
                    assert torch.equal(keys[b, h, length[b]:length[b] + len(p)], new[0][b, h, p])
                    assert torch.equal(values[b, h, length[b]:length[b] + len(p)], new[1][b, h, p])
        length = [x + len(p) for x, p in zip(length, paths)]
        assert n.tolist() == length
