"""Tree attention at the edges of the values that include/snapkv_draft.h allows, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from tests.cache_cases import to64
from tests.draft_cases import q8_rows
from tests.test_gpu_tree import BF16, check, make, run

pytestmark = pytest.mark.gpu

# bf16 over 8 bits, (G, T): up to eight, sixteen and 32 query rows a KV head, passes of 128 and of 256
Q8_KINDS = [(2, 4), (2, 8), (2, 12), (4, 20), (3, 70)]


def put(x, name, rows, q8, dev):
    """Cached rows fp64 [B,H,cap,d] (which the call's type holds exactly) in place of those of make()."""
    if q8:
        codes, step, x[name + "64"] = q8_rows(rows)
        x[name + "_codes"], x[name + "_step"] = codes.to(dev), step.to(dev)
    else:
        x[name], x[name + "64"] = torch.from_numpy(rows).to(x["q"].dtype).to(dev), rows


def steps_of_logits(x, q8, dev, rise=7.5, period=4):
    """Logits 0 in every row, but `rise` (log2) in the second half of every `period` tiles of 128 rows."""
    B, H, cap, d = x["k64"].shape
    x["q"] = torch.zeros_like(x["q"])
    x["q"][..., 0] = 1.0
    high = np.arange(cap) // 128 % period >= period // 2
    k = np.zeros((B, H, cap, d))
    k[..., 0] = np.where(high, rise * np.log(2.0) * np.sqrt(d), 0.0)
    put(x, "k", to64(torch.from_numpy(k).to(x["q"].dtype)), q8, dev)
    x["k_new"] = torch.zeros_like(x["k_new"])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", Q8_KINDS)
@pytest.mark.parametrize("rise", [7.5, 5.5])
def test_the_largest_values_of_8_bits(gpu_device, G, T, d, rise):
    """Values of V just below 2^48, under weights that may exceed one, as a maximum that grows by little is left as it is."""
    B, H, cap = 1, 64, 5000
    x = make(gpu_device, 31, B, H, G, d, T, cap, BF16, q8=True)
    steps_of_logits(x, True, gpu_device, rise)
    rng = np.random.default_rng(32)
    v = rng.uniform(-1, 1, size=(B, H, cap, d)) * 2.0 ** 47
    v[..., 3] = 2.0 ** 48 * (1 - 2.0 ** -9)
    v[..., 5] = 0.0                                  # (a code of zero)
    put(x, "v", v, True, gpu_device)
    x["v_new"] = (x["v_new"].float().clamp(-1, 1) * 2.0 ** 47).to(BF16)
    out, lse = run(x, [cap])
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    check(x, [cap], out, lse, heads=[0, 17, H - 1])
