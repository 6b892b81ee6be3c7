"""fp32 attention holds what 24-bit operands give: norms of the errors on random inputs, and inputs whose results hang
on bits that two bf16 parts would lose. tests/test_cache_precision_host.py shows that arithmetic with two parts of any
operand fails these bounds."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests import precision_cases as pc
from tests.cache_cases import check_attend, q4_inputs, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(gpu_device):
    import __graft_entry__
    __graft_entry__.build()
    return gpu_device


def run(dev, q, k, v):
    """q [Hq, d] over dense rows k, v [H, n, d], or over k, v = (levels, h, z): outputs and, added up over a KV
    head's queries, weights."""
    import kv_cache_compression_gb300 as kv
    q4 = isinstance(k, tuple)
    H, n = (k[0] if q4 else k).shape[:2]
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    score = torch.zeros(1, H, n, device=dev)
    if q4:
        cache = kv.Q4Cache(*(t[None].to(dev) for t in (*q4_inputs(*k), *q4_inputs(*v))))
        out = kv.q4_decode_attend(q[None].to(dev), cache, lens, score, decay=0.0)
    else:
        out = kv.decode_attend_scored(q[None].to(dev), k[None].to(dev), v[None].to(dev), lens, score, decay=0.0)
    torch.cuda.synchronize()
    return out[0].cpu(), score[0].cpu()


@pytest.mark.parametrize("q_scale", [0.5, 1.5])
@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("d,n", pc.SHAPES)
def test_norms_of_the_errors(dev, d, n, q4, q_scale):
    q, k, v = pc.random_heads(d, n, q_scale)
    if q4:
        # Sums over the parts |z| + |h t| of a value, on average 1.2 times the value's own size: half as much again
        # as the dense bound.
        made = [co.quantise(to64(x)) for x in (k, v)]
        out, weight = run(dev, q, *made)
        k, v = (torch.from_numpy(co.values(*x)) for x in made)
        exact = pc.exact_heads(q, k, v)
        bound = pc.bounds(q, k.float(), v.float(), 3)
    else:
        out, weight = run(dev, q, k, v)
        exact, bound = pc.exact_heads(q, k, v), pc.bounds(q, k, v, 2)
    error = pc.norm_error(out, exact[0]), pc.norm_error(weight, exact[1])
    assert error[0] <= bound[0] and error[1] <= bound[1], f"errors {error} of {bound}"


def tensors(case, d):
    return [torch.from_numpy(np.asarray(x, dtype=np.float32)) for x in case(d)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", [pc.case_q, pc.case_k])
def test_logits_of_low_bits(dev, case, d):
    """The leading parts of the logits' products cancel exactly: what is left is as large as the tolerance says."""
    q, k, v = tensors(case, d)
    out, weight = run(dev, q[None], k[None], v[None])
    size = np.zeros((1, 1, *k.shape))
    size[0, 0, :, 0] = np.abs(to64(k) @ to64(q)) / abs(to64(q[0]))
    check_attend(q[None, None], to64(k)[None, None], to64(v)[None, None], [k.shape[0]], out[None], k_size=size,
                 score0=torch.zeros(1, 1, k.shape[0]), score=weight[None], decay=0.0, where=case.__name__)


@pytest.mark.parametrize("d", [64, 128])
def test_logits_of_low_bits_over_four_bits(dev, d):
    """As above, of a query (x, y, 0, ...) and keys 15 h (1, -1, ...) with h = 2^16 times -8 .. 8."""
    rng = np.random.default_rng(d)
    n = 300
    x, y = pc.low_bits(1, d + 5)
    q = np.zeros((1, d))
    q[0, 0], q[0, 1] = x[0], y[0]
    j = rng.integers(-8, 9, n)
    u = np.full((1, n, d), 8)
    u[0, :, 0], u[0, :, 1] = np.where(j >= 0, 15, 0), np.where(j >= 0, 0, 15)
    h = np.broadcast_to(np.abs(j)[None, :, None] * 2.0 ** 16, (1, n, d // 64)).copy()
    made_k, made_v = (u, h, np.zeros_like(h)), co.quantise(rng.standard_normal((1, n, d)))
    q = torch.from_numpy(q.astype(np.float32))
    out, weight = run(dev, q, made_k, made_v)
    k64, v64 = co.values(*made_k), co.values(*made_v)
    size = np.zeros((1, *k64.shape))
    size[0, 0, :, 0] = np.abs(k64[0] @ to64(q[0])) / x[0]
    check_attend(q[None], k64[None], v64[None], [n], out[None], k_size=size, v_size=co.magnitudes(*made_v)[None],
                 score0=torch.zeros(1, 1, n), score=weight[None], decay=0.0, where="q4")


@pytest.mark.parametrize("d", [64, 128])
def test_values_of_low_bits(dev, d):
    """Sixteen rows' products (at most 2 in size, cut to 2^-22 when 17 terms are added) are off by 17 * 2^-22 at most, their
    average by 2^-22, and little is added by the smaller parts: 2^-21 of a result of 2^-19."""
    q, k, v = tensors(pc.case_v, d)
    out, _ = run(dev, q[None], k[None], v[None])
    ref = co.attend(to64(q), to64(k), to64(v))[0]
    assert np.abs(ref - 2.0 ** -19).max() < 2.0 ** -30
    assert np.abs(to64(out[0]) - ref).max() <= 2.0 ** -21


def check_weights(out, ref, pairs, total, size):
    """Pairs of weights 2^-19 apart. Each weight is off by the exponential's 2^-22 of itself and some 2^-24 of roundings
    (2^-21 a pair), and a pair's products by an eighth of 17 * 2^-23: 2^-20 a pair, half of what there is."""
    per_pair = size * pairs / total
    assert np.abs(ref - per_pair * 2.0 ** -19).max() < per_pair * 2.0 ** -23
    assert np.abs(to64(out) - ref).max() <= per_pair * 2.0 ** -20


@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_low_bits(dev, d):
    q, k, v = tensors(pc.case_p, d)
    out, _ = run(dev, q[None], k[None], v[None])
    ref, p, _, _ = co.attend(to64(q), to64(k), to64(v))
    check_weights(out[0], ref, (k.shape[0] - 1) // 2, 1 / p[0], 1.0)


@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_low_bits_over_four_bits(dev, d):
    """The same weights, from two groups' centres (d = 128) or two channels' levels (d = 64), of values 15/16 and -15/16."""
    n, ng = 301, d // 64
    low = np.arange(n - 1) % 2 == 1
    a, b = np.log(pc.HIGH_WEIGHT) * np.sqrt(d), np.log(pc.LOW_WEIGHT) * np.sqrt(d)
    q, u, h, z = np.zeros((1, d)), np.full((1, n, d), 8), np.zeros((1, n, ng)), np.zeros((1, n, ng))
    if d == 128:
        q[0, 0], q[0, 64] = a, b
        z[0, 1:, 0], z[0, 1:, 1] = ~low, low
    else:
        q[0, 0], q[0, 1] = (a + b) / 2, (a - b) / 2
        h[0, 1:] = 1.0
        u[0, 1:, 1] = np.where(low, 7, 8)
    hv = np.full((1, n, ng), 2.0 ** -4)
    hv[0, 0] = 0.0
    uv = np.zeros((1, n, d), dtype=np.int64)
    uv[0, 1:] = np.where(low, 0, 15)[:, None]
    made_k, made_v = (u, h, z), (uv, hv, np.zeros_like(hv))
    q = torch.from_numpy(q.astype(np.float32))
    out, _ = run(dev, q, made_k, made_v)
    ref, p, _, _ = co.attend(to64(q[0]), co.values(*made_k)[0], co.values(*made_v)[0])
    check_weights(out[0], ref, (n - 1) // 2, 1 / p[0], 15 / 16)
