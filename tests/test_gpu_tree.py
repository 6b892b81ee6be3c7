"""Tree attention over dense and 8-bit caches against the fp64 oracle (include/snapkv_draft.h)."""
import numpy as np
import pytest
import torch

import kv_cache_compression_gb300 as kv
from tests.cache_cases import to64
from tests.draft_cases import Q8_FLOOR, check_tree, q8_rows, random_tree

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def make(dev, seed, B, H, G, d, T, cap, dtype, *, q8=False, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = {"q": (torch.randn(B, H * G, T, d, generator=g) * 1.5 * scale).to(dtype)}
    for n in ("k", "v"):
        rows = torch.randn(B, H, cap, d, generator=g).to(dtype)
        if q8:
            code, step, x[n + "64"] = q8_rows(rows.double().numpy())
            x[n + "_codes"], x[n + "_step"] = code.to(dev), step.to(dev)
        else:
            x[n], x[n + "64"] = rows.to(dev), rows.double().numpy()
        x[n + "_new"] = torch.randn(B, H, T, d, generator=g).to(dtype).to(dev)
    x["q"] = x["q"].to(dev)
    return x


def run(x, lens, *, drafts=True, mask=None, n_new=None, lse=True, **kw):
    dev = x["q"].device
    B, Hq, T, d = x["q"].shape
    lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    n = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device=dev)
    m = None if mask is None else torch.from_numpy(mask).to(dev)
    ls = torch.full((B, Hq, T), float("nan"), device=dev) if lse else None
    new = (x["k_new"], x["v_new"], m) if drafts else ()
    out = torch.full_like(x["q"], float("nan"))
    if "k" in x:
        kv.tree_attend(x["q"], x["k"], x["v"], lens, *new, n_new=n, lse=ls, out=out, **kw)
    else:
        cache = kv.Q8Cache(x["k_codes"], x["k_step"], x["v_codes"], x["v_step"])
        kv.q8_tree_attend(x["q"], cache, lens, *new, n_new=n, lse=ls, out=out, **kw)
    return out, ls


def check(x, lens, out, lse, *, drafts=True, mask=None, n_new=None, **kw):
    new = dict(k_new=x["k_new"], v_new=x["v_new"], mask=mask) if drafts else {}
    floor = Q8_FLOOR if "k_codes" in x and out.dtype == BF16 else 0.0
    check_tree(x["q"], x["k64"], x["v64"], lens, out, lse, n_new=n_new, floor=floor, **new, **kw)


SHAPES = [  # B, H, G, d, T, cap, lengths
    (1, 1, 1, 64, 1, 1, [1]), (1, 2, 1, 128, 1, 17, [0]), (2, 1, 1, 64, 3, 63, [63, 0]), (1, 4, 1, 64, 5, 83, [83]),
    (2, 3, 2, 128, 4, 65, [64, 65]), (3, 2, 4, 64, 16, 129, [128, 1, 129]), (2, 2, 7, 128, 9, 200, [200, 127]),
    (1, 2, 4, 128, 33, 300, [257]), (1, 1, 8, 128, 64, 500, [499]), (2, 1, 4, 64, 65, 130, [130, 5]), (1, 1, 3, 64, 130, 70, [70]),
    (5, 2, 1, 128, 2, 1500, [1500, 3, 0, 700, 1024]), (1, 2, 1, 64, 8, 4000, [3999]),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:6])))
def test_trees(gpu_device, shape, dtype, q8):
    B, H, G, d, T, cap, lens = shape
    x = make(gpu_device, 7, B, H, G, d, T, cap, dtype, q8=q8)
    mask = random_tree(np.random.default_rng(T), B, T)
    out, lse = run(x, lens, mask=mask)
    check(x, lens, out, lse, mask=mask)
    again, lse2 = run(x, lens, mask=mask)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("shape", SHAPES[1:11:2], ids=lambda s: "x".join(map(str, s[:6])))
def test_causal_ragged_and_without_drafts(gpu_device, shape, dtype, q8):
    B, H, G, d, T, cap, lens = shape
    x = make(gpu_device, 8, B, H, G, d, T, cap, dtype, q8=q8)
    n_new = [(T * (b + 1) // B) if b else T // 2 for b in range(B)]
    for drafts in (True, False):
        out, lse = run(x, lens, drafts=drafts, n_new=n_new)
        check(x, lens, out, lse, drafts=drafts, n_new=n_new)
        out, lse = run(x, lens, drafts=drafts)
        check(x, lens, out, lse, drafts=drafts)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", [(1, 1), (2, 3), (1, 8), (3, 3), (1, 16), (16, 1), (1, 17), (4, 8), (1, 33), (5, 13), (1, 100), (8, 16), (3, 43), (4, 64), (1, 257)])
def test_every_number_of_rows(gpu_device, G, T, d, q8):
    """bf16 calls of one query row a KV head up to three times 128, whose kernels differ."""
    B, H, cap = 2, 2, 700
    x = make(gpu_device, 9, B, H, G, d, T, cap, BF16, q8=q8)
    mask = random_tree(np.random.default_rng(T), B, T)
    for lens, n_new in (([700, 129], None), ([1, 640], [T, max(1, T - 5)]), ([0, 16], [max(1, T // 2), 0])):
        out, lse = run(x, lens, mask=mask, n_new=n_new)
        check(x, lens, out, lse, mask=mask, n_new=n_new)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("shape", [  # B, H, G, d, T, cap, tokens of each sequence
    (1, 2, 4, 128, 70, 300, None), (2, 1, 3, 64, 128, 150, None), (1, 1, 4, 128, 150, 400, None), (1, 2, 4, 64, 97, 260, None),
    (1, 1, 2, 128, 448, 140, None), (1, 1, 1, 64, 1025, 130, None), (1, 1, 1, 64, 1153, 129, None),
    (4, 2, 4, 128, 64, 700, [64, 33, 0, 1]), (3, 1, 4, 64, 110, 900, [110, 32, 97]), (3, 2, 1, 64, 440, 500, [129, 440, 300]),
    (2, 1, 4, 128, 70, 1300, [69, 33]), (2, 1, 1, 128, 1030, 140, [1030, 900])])
def test_passes_of_many_rows(gpu_device, shape, q8):
    """Whole and half passes, side by side or one after the other."""
    B, H, G, d, T, cap, n_new = shape
    x = make(gpu_device, T + cap, B, H, G, d, T, cap, BF16, q8=q8)
    lens = [cap, cap // 2, cap - 1, 3][:B]
    rng = np.random.default_rng(T)
    mask = random_tree(rng, B, T)
    for drafts in (True, False):
        out, lse = run(x, lens, drafts=drafts, mask=mask if drafts else None, n_new=n_new)
        check(x, lens, out, lse, drafts=drafts, mask=mask if drafts else None, n_new=n_new, heads=[H - 1], where=f"{drafts}")
