"""Tree attention at the edges of the values that include/snapkv_draft.h allows, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from tests.cache_cases import to64
from tests.draft_cases import Q8_FLOOR, check_tree, q8_rows
from tests.test_gpu_tree import BF16, FP32, check, make, run

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


# one of every kernel: (dtype, 8-bit, G, T)
KINDS = [(FP32, False, 2, 3), (FP32, False, 4, 9), (FP32, True, 4, 9), (BF16, False, 1, 5), (BF16, False, 3, 5), (BF16, False, 2, 20), (BF16, False, 4, 50),
         *((BF16, True, *k) for k in Q8_KINDS)]
kinds = pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{str(k[0])[6:]}-{'q8' if k[1] else 'dense'}-{k[2]}x{k[3]}")


@kinds
@pytest.mark.parametrize("size", [(2, 700), (64, 2600)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("log2", [24, 28, 30, 31, 32, 33, 37, 50, 90])
def test_large_logits(gpu_device, kind, size, log2):
    """One key's logit is about twice the others' (or half of them, where they are negative), by far more than a logit's error:
    its weight is one and the others' are zero."""
    dtype, q8, G, T = kind
    (H, cap), d = size, 64
    x = make(gpu_device, 33, 1, H, G, d, T, cap, dtype, q8=q8)
    rng = np.random.default_rng(log2)
    half = log2 // 2
    for sign in (1.0, -1.0):
        # every row of queries another mantissa, so that logits are rounded up and down
        size_q = rng.integers(129, 256, size=(H * G, T)) / 128.0 * 2.0 ** half
        x["q"] = torch.zeros_like(x["q"])
        x["q"][0, ..., 0] = torch.from_numpy(size_q).to(x["q"])
        best = rng.integers(0, cap, size=H)
        best[:2] = 0, cap - 1
        k = np.zeros((1, H, cap, d))
        k[..., 0] = sign * (1.0 if sign > 0 else 1.9921875) * 2.0 ** (log2 - half)
        k[0, np.arange(H), best, 0] = sign * (1.9921875 if sign > 0 else 1.0) * 2.0 ** (log2 - half)
        put(x, "k", k, q8, gpu_device)
        out, lse = run(x, [cap], drafts=False)
        head = np.arange(H * G) // G
        want = x["v64"][0, head, best[head]][:, None]
        logit = to64(x["q"])[0, ..., 0] * x["k64"][0, head, best[head], 0][:, None] / np.sqrt(d)
        # half a step of the output; the weight, one but for the rounding of the maximum that it is taken under (and over 8 bits times
        # a step), is off by 2^-8 where it is held as one bf16 value and by 2^-16 as two; its own error (2^-22 for exp2) and fp32's in
        # what follows
        part = 0.0 if dtype == FP32 else 2.0 ** -8 if G * T > (32 if q8 else 16) else 2.0 ** -16
        tol = (torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -7) + part + 2.0 ** -20) * np.abs(want) + 2.0 ** -96
        assert np.all(np.abs(to64(out)[0] - want) <= tol), f"sign {sign}"
        assert np.all(np.abs(to64(lse)[0] - logit) <= 2.0 ** -20 * np.abs(logit)), f"sign {sign}"


@pytest.mark.parametrize("kind", KINDS[5:7] + KINDS[-2:], ids=lambda k: f"{'q8' if k[1] else 'dense'}-{k[2]}x{k[3]}")
def test_rows_of_large_logits_leave_their_neighbours_alone(gpu_device, kind):
    dtype, q8, G, T = kind
    H, cap, d = 2, 700, 64
    x = make(gpu_device, 34, 1, H, G, d, T, cap, dtype, q8=q8)
    want, lse = run(x, [cap])
    x["q"] = x["q"].clone()
    x["q"][:, :, ::3] *= 2.0 ** 30
    got, lse2 = run(x, [cap])
    rest = [t for t in range(T) if t % 3]
    assert torch.equal(got[:, :, rest].view(torch.int16), want[:, :, rest].view(torch.int16)) and torch.equal(lse2[:, :, rest], lse[:, :, rest])
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("kind", [k for k in KINDS if not k[1]], ids=lambda k: f"{str(k[0])[6:]}-{k[2]}x{k[3]}")
@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_values_of_dense_rows(gpu_device, kind, d):
    """2^8 times the sum of |V| just below 2^128, under weights that may exceed one by 2^7.5."""
    dtype, q8, G, T = kind
    B, H, cap = 1, 64, 5000
    x = make(gpu_device, 35, B, H, G, d, T, cap, dtype)
    steps_of_logits(x, False, gpu_device)
    rng = np.random.default_rng(36)
    v = torch.from_numpy(rng.uniform(1, 2, size=(B, H, cap, d)) * 2.0 ** 106).to(dtype)   # 2^8 x 5000 x 2^107 < 2^127.3
    put(x, "v", to64(v), False, gpu_device)
    x["v_new"] = (x["v_new"].float().clamp(-1, 1) * 2.0 ** 107).to(dtype)
    out, lse = run(x, [cap])
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    check(x, [cap], out, lse, heads=[0, 17, H - 1])


q8_kinds = pytest.mark.parametrize("G,T", Q8_KINDS)


@q8_kinds
@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_queries_over_8_bits(gpu_device, G, T, d):
    x = make(gpu_device, 37, 1, 2, G, d, T, 700, BF16, q8=True)
    x["q"] = (x["q"].float().clamp(-1.99, 1.99) * 2.0 ** 47).to(BF16)
    put(x, "k", to64(torch.randn(1, 2, 700, d, generator=torch.Generator().manual_seed(38))) * 2.0 ** -48, True, gpu_device)
    x["k_new"] = (x["k_new"].float() * 2.0 ** -48).to(BF16)
    out, lse = run(x, [700])
    check(x, [700], out, lse)


@q8_kinds
def test_the_largest_products_with_drafted_rows_over_8_bits(gpu_device, G, T):
    """One drafted row's logit (of 2^61 sqrt(d), or of its half where they are negative) is far above all others."""
    d = 128
    for sign in (1.0, -1.0):
        x = make(gpu_device, 39, 1, 2, G, d, T, 300, BF16, q8=True)
        x["q"] = torch.zeros_like(x["q"])
        x["q"][..., 0] = 1.5 * 2.0 ** 40
        x["k_new"] = torch.zeros_like(x["k_new"])
        x["k_new"][..., 0] = sign * 2.0 ** 20 * (1.0 if sign > 0 else 1.3125)
        x["k_new"][:, :, 0, 0] = sign * 2.0 ** 20 * (1.3125 if sign > 0 else 1.0)       # (1.5 x 1.3125 x 2^60 < 2^61)
        out, lse = run(x, [300 if sign > 0 else 0])
        want = x["v_new"][:, :, :1].repeat_interleave(G, 1).double()
        logit = 1.5 * 2.0 ** 60 * sign * (1.3125 if sign > 0 else 1.0) / d ** 0.5
        assert torch.all((out.double() - want).abs() <= 2.0 ** -6.9 * want.abs())   # an output's and a weight's half step
        assert torch.all((lse.double() - logit).abs() <= 2.0 ** -20 * abs(logit))


@q8_kinds
@pytest.mark.parametrize("log2", [-40, -60, -70, -80])
def test_small_weights_of_large_drafted_rows_over_8_bits(gpu_device, G, T, log2):
    """Cached zeros under weights of one, and drafted rows whose weights of about 2^log2 are all that outputs hang on."""
    d = 64
    x = make(gpu_device, 40, 1, 2, G, d, T, 300, BF16, q8=True)
    x["q"] = torch.zeros_like(x["q"])
    x["q"][..., 0] = 1.0
    for name in ("k", "v"):
        put(x, name, np.zeros((1, 2, 300, d)), True, gpu_device)
    x["k_new"] = torch.zeros_like(x["k_new"])
    x["k_new"][..., 0] = log2 * np.log(2.0) * d ** 0.5
    x["v_new"] = (x["v_new"].float().clamp(-1, 1) * 2.0 ** 47).to(BF16)
    out, lse = run(x, [300])
    lost = 2.0 ** -81 * 2.0 ** 47      # of each drafted row's share, rounded to a multiple of 2^-80
    check_tree(x["q"], x["k64"], x["v64"], [300], out, lse, k_new=x["k_new"], v_new=x["v_new"], floor=lost * T / (300 + T) / 300)
    assert out.abs().max() > 0


@q8_kinds
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("log2", [-60, -72])
def test_the_smallest_values_of_8_bits(gpu_device, G, T, d, log2):
    """Steps of V down to about 2^-79: outputs are right but for 2^-96 of each row."""
    x = make(gpu_device, 41, 2, 2, G, d, T, 300, BF16, q8=True)
    v = to64(torch.randn(2, 2, 300, d, generator=torch.Generator().manual_seed(42))) * 2.0 ** log2
    put(x, "v", v, True, gpu_device)
    x["v_new"] = (x["v_new"].float() * 2.0 ** log2).to(BF16)
    out, lse = run(x, [300, 131])
    check(x, [300, 131], out, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", [(1, 17), (2, 12), (4, 8), (1, 32)])
def test_weights_of_two_parts_up_to_32_rows_over_8_bits(gpu_device, G, T, d):
    """Calls of 17 to 32 query rows a KV head over 8 bits hold weights to 16 bits, as those of fewer: every token is held to the
    tolerance of a call of its own, with the drafted rows that it sees behind the cached ones."""
    cap = 300
    x = make(gpu_device, 43, 1, 2, G, d, T, cap, BF16, q8=True)
    out, lse = run(x, [cap])
    for t in range(T):
        k, v = (np.concatenate([x[n + "64"], to64(x[n + "_new"])[:, :, :t + 1]], 2) for n in "kv")
        check_tree(x["q"][:, :, t:t + 1], k, v, [cap + t + 1], out[:, :, t:t + 1], lse[:, :, t:t + 1], floor=Q8_FLOOR, where=f"token {t}")
