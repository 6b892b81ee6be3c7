"""One workspace for calls of every kernel of the tree attention, one after the other, whatever an earlier call left in it
(include/snapkv_draft.h)."""
import numpy as np
import pytest
import torch

import kv_cache_compression_gb300 as kv
from tests.test_gpu_tree import BF16, FP32, make
from tests.test_gpu_tree_edges import same

pytestmark = pytest.mark.gpu

# dtype, 8 bits, B, H, G, d, T, cap: every kernel, few and many sequences, short caches and long ones, lists of few tiles and of many
CALLS = [(BF16, False, 2, 8, 4, 128, 64, 3000), (BF16, False, 1, 1, 1, 64, 3, 270), (FP32, False, 3, 2, 2, 128, 3, 900),
         (BF16, True, 2, 4, 3, 128, 70, 700), (BF16, True, 40, 2, 2, 64, 4, 500), (BF16, False, 3, 1, 3, 64, 128, 150),
         (FP32, True, 4, 4, 4, 64, 9, 2000), (BF16, False, 2, 8, 1, 128, 20, 5000), (BF16, True, 1, 2, 2, 128, 12, 300),
         (BF16, False, 1, 3, 1, 64, 300, 400), (BF16, True, 8, 8, 1, 128, 1, 4000), (BF16, False, 70, 1, 2, 64, 20, 300)]


def prepared(dev, i, call):
    dtype, q8, B, H, G, d, T, cap = call
    x = make(dev, 50 + i, B, H, G, d, T, cap, dtype, q8=q8)
    rng = np.random.default_rng(i)
    lens = torch.tensor([cap] + [int(rng.integers(0, cap + 1)) for _ in range(B - 1)], dtype=torch.int32, device=dev)
    n_new = torch.tensor([int(rng.integers(0, T + 1)) for _ in range(B)], dtype=torch.int32, device=dev) if i % 2 else None
    out, lse = torch.empty_like(x["q"]), torch.empty(B, H * G, T, device=dev)
    cache = kv.Q8Cache(x["k_codes"], x["k_step"], x["v_codes"], x["v_step"]) if q8 else None

    def attend(workspace=None):
        kw = dict(n_new=n_new, lse=lse, out=out, workspace=workspace)
        if q8:
            kv.q8_tree_attend(x["q"], cache, lens, x["k_new"], x["v_new"], **kw)
        else:
            kv.tree_attend(x["q"], x["k"], x["v"], lens, x["k_new"], x["v_new"], **kw)
        return out, lse
    attend.size = kv.tree_workspace_size(B, H * G, H, d, T, cap)
    attend.lens = lens
    return attend


@pytest.mark.parametrize("fill", [0xFF, 0x7F, 0x00])
def test_one_workspace_for_all(gpu_device, fill):
    calls = [prepared(gpu_device, i, c) for i, c in enumerate(CALLS)]
    want = [[t.clone() for t in c()] for c in calls]
    ws = torch.full((max(c.size for c in calls),), fill, dtype=torch.uint8, device=gpu_device)
    for order in (range(len(calls)), reversed(range(len(calls)))):   # what a call leaves is larger than the next one's, and smaller
        for i in order:
            got = calls[i](ws)
            assert all(same(a, b) for a, b in zip(got, want[i])), CALLS[i]


def test_graphs_that_share_a_workspace_one_after_the_other(gpu_device):
    calls = [prepared(gpu_device, i, c) for i, c in enumerate(CALLS)]
    ws = torch.full((max(c.size for c in calls),), 0xFF, dtype=torch.uint8, device=gpu_device)
    graphs = []
    for c in calls:
        c(ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            result = c(ws)
        graphs.append((graph, result))
    for shorter in (False, True):
        if shorter:
            for c in calls:
                c.lens.copy_(c.lens // 3)
        want = [[t.clone() for t in c()] for c in calls]
        for order in (range(len(calls)), reversed(range(len(calls)))):
            for i in order:
                for t in graphs[i][1]:
                    t.fill_(float("nan"))
                graphs[i][0].replay()
            torch.cuda.synchronize()
            for i, c in enumerate(calls):
                assert all(same(a, b) for a, b in zip(graphs[i][1], want[i])), CALLS[i]
