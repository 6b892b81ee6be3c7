"""Inputs whose results depend on the low bits of fp32 operands, and an emulation of the tensor-core arithmetic with
fewer of them: shared by the precision tests of fp32 attention (on the GPU, and of the bounds themselves on the CPU).

fp32 operands reach the tensor cores as three bf16 parts (24 bits). An operand of two parts keeps 16: what lies below
2^-17 of its size is lost."""
import numpy as np
import torch

from oracle import cache_oracle as co

SHAPES = [(64, 83), (64, 300), (64, 2049), (128, 83), (128, 2049)]   # d, rows
HEADS = 16


def random_heads(d, n, q_scale):
    """q [H, d], k, v [H, n, d] of fixed values, fp32."""
    g = torch.Generator().manual_seed(1000 * d + n + int(16 * q_scale))
    return (torch.randn(HEADS, d, generator=g) * q_scale, torch.randn(HEADS, n, d, generator=g),
            torch.randn(HEADS, n, d, generator=g))


def norm_error(x, ref):
    x, ref = np.asarray(x, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    return np.linalg.norm(x - ref) / np.linalg.norm(ref)


def exact_heads(q, k, v):
    """Outputs and weights in 64 bits, head by head."""
    got = [co.attend(q[h].numpy(), k[h].numpy(), v[h].numpy())[:2] for h in range(q.shape[0])]
    return np.stack([o for o, _ in got]), np.stack([p for _, p in got])


def plain_heads(q, k, v):
    """The same in elementary fp32 operations."""
    s = torch.einsum("hd,hnd->hn", q, k) / q.shape[-1] ** 0.5
    p = (s - s.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    return torch.einsum("hn,hnd->hd", p, v).numpy(), p.numpy()


def bounds(q, k, v, factor):
    """Bounds on the relative (2-norm) errors of the outputs and of the weights: `factor` times the plain form's and
    2^-22, the error of the exponential instruction."""
    return [factor * norm_error(x, e) + 2.0 ** -22 for x, e in zip(plain_heads(q, k, v), exact_heads(q, k, v))]


def parts(x, n):
    """x as the sum of n bf16 parts, in 64 bits."""
    rest, out = np.asarray(x, dtype=np.float64), 0.0
    for _ in range(n):
        part = co.bf16(rest.astype(np.float32))
        out, rest = out + part, rest - part
    return out


def truncated(x):
    """x cut to 24 bits, as a tensor-core sum is."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(m * 2.0 ** 24) * 2.0 ** -24, e)


def emulated_head(q, k, v, nq=3, nk=3, nv=3, np_=3):
    """One head with operands in so many parts, logits summed sixteen channels at a time."""
    q, k, v = parts(q, nq), parts(k, nk), parts(v, nv)
    s = np.zeros(k.shape[0])
    for c in range(0, q.size, 16):
        s = truncated(s + k[:, c:c + 16] @ q[c:c + 16])
    s = (s / np.sqrt(q.size)).astype(np.float32).astype(np.float64)
    p = np.exp(s - s.max())
    return parts(p, np_) @ v / p.sum(), p / p.sum()


def low_bits(n, seed):
    """n pairs of numbers in [1, 2) that differ by 20 .. 60 units of 2^-23, either way: little or nothing of the
    differences is left in 16 bits (steps of 2^-16 or 2^-15)."""
    rng = np.random.default_rng(seed)
    x = np.floor(rng.uniform(1.1, 1.9, n) * 2.0 ** 23) * 2.0 ** -23
    return x, x + rng.integers(20, 61, n) * rng.choice([-1, 1], n) * 2.0 ** -23


def case_q(d, n=300):
    """Logits are c (x - y), of a query (x, y, 0, ...) and keys (c, -c, 0, ...)."""
    x, y = low_bits(1, d)
    q, k = np.zeros(d), np.zeros((n, d))
    q[0], q[1] = x[0], y[0]
    c = np.random.default_rng(d).integers(-8, 9, n) * 2.0 ** 20
    k[:, 0], k[:, 1] = c, -c
    return q, k, np.random.default_rng(d + 1).standard_normal((n, d))


def case_k(d, n=300):
    """Logits are A (x_r - y_r), of a query (A, -A, 0, ...) and keys (x_r, y_r, 0, ...)."""
    q, k = np.zeros(d), np.zeros((n, d))
    q[0], q[1] = 2.0 ** 20, -2.0 ** 20
    k[:, 0], k[:, 1] = low_bits(n, d + 2)
    return q, k, np.random.default_rng(d + 3).standard_normal((n, d))


def case_v(d, n=300):
    """Equal weights over values +(y + 2^-18) and -y, where 2^-18 is below half a step of y's second part: the sum of
    the parts that are lost is the result, 2^-19."""
    y = 1.0 + np.random.default_rng(d + 4).integers(128, 256, (n // 2, d)) * 2.0 ** -16   # 2^-9 .. 2^-8 over bf16's 1
    v = np.stack([y + 2.0 ** -18, -y], 1).reshape(n, d)
    return np.zeros(d), np.zeros((n, d)), v


# A weight of two parts (184 * 2^-8 + 160 * 2^-17), and one 2^-19 above it, below half a step of its second part.
LOW_WEIGHT = 184 * 2.0 ** -8 + 160 * 2.0 ** -17
HIGH_WEIGHT = LOW_WEIGHT + 2.0 ** -19


def case_p(d, n=300):
    """A row of weight 1 and value 0, and pairs of rows with weights 2^-19 apart and values 1 and -1."""
    q, k, v = np.zeros(d), np.zeros((n, d)), np.zeros((n, d))
    q[0] = np.sqrt(d)
    k[1:, 0] = np.where(np.arange(n - 1) % 2, np.log(LOW_WEIGHT), np.log(HIGH_WEIGHT))
    v[1:] = np.where(np.arange(n - 1) % 2, -1.0, 1.0)[:, None]
    k[-1:], v[-1:] = -60.0 * (1 - n % 2), v[-1:] * (n % 2)      # (an even n leaves a row over: no weight)
    return q, k, v
