"""The bounds of tests/test_gpu_cache_precision.py on the CPU: the arithmetic with three parts an operand is within
them, and with two parts of any operand it is not."""
import numpy as np
import pytest

from tests import precision_cases as pc


def emulated(q, k, v, **kw):
    got = [pc.emulated_head(q[h].numpy(), k[h].numpy(), v[h].numpy(), **kw) for h in range(q.shape[0])]
    return np.stack([o for o, _ in got]), np.stack([p for _, p in got])


@pytest.mark.parametrize("factor", [2, 3])
@pytest.mark.parametrize("d,n", pc.SHAPES)
def test_the_norm_bounds_tell_two_parts_from_three(d, n, factor):
    for q_scale in (0.5, 1.5):
        q, k, v = pc.random_heads(d, n, q_scale)
        out_bound, weight_bound = pc.bounds(q, k, v, factor)
        exact = pc.exact_heads(q, k, v)
        errors = {name: [pc.norm_error(x, e) for x, e in zip(emulated(q, k, v, **kw), exact)]
                  for name, kw in (("all", {}), ("q", dict(nq=2)), ("k", dict(nk=2)), ("v", dict(nv=2)), ("p", dict(np_=2)))}
        assert errors["all"][0] < 0.7 * out_bound and errors["all"][1] < 0.7 * weight_bound
        assert errors["q"][1] > weight_bound and errors["k"][1] > weight_bound
        assert errors["v"][0] > out_bound
        if factor == 2 and q_scale == 0.5:
            assert errors["p"][0] > out_bound


def f32(*arrays):
    return [np.asarray(a, dtype=np.float32).astype(np.float64) for a in arrays]


@pytest.mark.parametrize("d", [64, 128])
def test_the_constructed_cases_lose_their_results_with_two_parts(d):
    from oracle import cache_oracle as co
    for case, kw in ((pc.case_q, dict(nq=2)), (pc.case_k, dict(nk=2))):
        q, k, v = f32(*case(d))
        o, p, _, _ = co.attend(q, k, v)
        for n_parts, off in ((3, False), (2, True)):
            _, w = pc.emulated_head(q, k, v, **{name: n_parts for name in kw})
            assert (pc.norm_error(w, p) > 0.1) == off
            assert off or pc.norm_error(w, p) < 1e-6
    for case, kw, step in ((pc.case_v, dict(nv=2), 2.0 ** -19), (pc.case_p, dict(np_=2), 0.0)):
        q, k, v = f32(*case(d))
        o, p, _, _ = co.attend(q, k, v)
        size = np.abs(o).max()
        assert size > 2.0 ** -22 and (not step or abs(size - step) < 2.0 ** -40)
        assert np.abs(pc.emulated_head(q, k, v)[0] - o).max() < size / 8
        assert np.abs(pc.emulated_head(q, k, v, **kw)[0] - o).max() > 0.9 * size
