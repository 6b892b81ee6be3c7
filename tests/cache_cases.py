"""Shared by the tests of the cache operators: inputs, and the oracle's tolerances."""
import numpy as np
import torch

from oracle import cache_oracle as co


def to64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def logit_error(d, size):
    """Bound on a logit's error: d products summed in fp32 (a tensor-core sum may drop up to one unit of
    the last place, 2^-23 of the running magnitude, per addition), a few roundings around them."""
    return (d + 8) * 2.0 ** -23 * size


def weight_error(d, n, size):
    """Bound on a weight's relative error: its own and the sum's logit errors, exp2 (2^-22) and its argument
    (|s| + |m| below 2 size, rounded: 2^-24 each), n terms summed in fp32."""
    return 2 * logit_error(d, size) + 4 * size * 2.0 ** -23 + 2.0 ** -21 + (n / 16 + 32) * 2.0 ** -23


def out_tolerance(ref, pv, d, n, size, dtype):
    """Half a step of the output's type, and the internal error times sum p |v|. bf16 calls round weights
    to two bf16 parts (2^-17), fp32 calls split values and weights into three (2^-24 each)."""
    half = torch.finfo(dtype).eps / 2
    inner = (weight_error(d, n, size) + (n / 16 + 32) * 2.0 ** -23 +
             (2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -22)) * pv
    return half * (np.abs(ref) + inner) + inner + 1e-37


def check_attend(q, k, v, lens, out, *, k_size=None, v_size=None, score0=None, score=None, decay=1.0, heads=None,
                 where=""):
    """out [B,Hq,d] (and score [B,H,cap]) against the oracle; k, v (and sizes) fp64 [B,H,cap,d]."""
    B, Hq, d = q.shape
    H = k.shape[1]
    G = Hq // H
    qh, o = to64(q), to64(out)
    for b in range(B):
        n = max(0, min(int(lens[b]), k.shape[2]))
        for h in range(H) if heads is None else heads:
            total, total_err = np.zeros(n), np.zeros(n)
            for g in range(G):
                ks = None if k_size is None else k_size[b, h, :n]
                vs = None if v_size is None else v_size[b, h, :n]
                ref, p, size, pv = co.attend(qh[b, h * G + g], k[b, h, :n], v[b, h, :n], ks, vs)
                tol = out_tolerance(ref, pv, d, n, size, out.dtype)
                err = np.abs(o[b, h * G + g] - ref)
                assert np.all(err <= tol), f"{where} b{b} h{h} g{g} n{n}: {err.max():.3g} of {tol[err.argmax()]:.3g}"
                total += p
                total_err += p * (weight_error(d, n, size) + G * 2.0 ** -23)
            if score is not None:
                s0, s1 = to64(score0[b, h]), to64(score[b, h])
                want = total + (decay * s0[:n] if decay else 0.0)
                tol = total_err + np.abs(want) * 2.0 ** -22 + 2.0 ** -120
                err = np.abs(s1[:n] - want)
                assert np.all(err <= tol), f"{where} score b{b} h{h} n{n}: {(err / tol).max():.3g} of the tolerance"
                assert np.array_equal(s1[n:], s0[n:], equal_nan=True), f"{where} score past the end b{b} h{h}"


def q4_inputs(u, h, z):
    """The cache tensors (codes, meta) of level numbers and (h, z), on the CPU."""
    meta = np.stack([h, z], -1).astype(np.float32)
    return torch.from_numpy(co.pack(u)), torch.from_numpy(meta).to(torch.bfloat16)
