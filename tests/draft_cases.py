"""Shared by the tests of the operators for drafted tokens: inputs, and the oracle's tolerances."""
import numpy as np
import torch

from oracle import draft_oracle as do
from tests.cache_cases import out_tolerance, to64, weight_error


def random_tree(rng, B, T, spread=4):
    """Masks [B, T, T] of random trees: token i hangs on one of the `spread` before it, or on the cached text."""
    mask = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for i in range(T):
            p = i - 1 - int(rng.integers(0, spread))
            if p >= 0:
                mask[b, i] = mask[b, p]
            mask[b, i, i] = True
    return mask


def check_tree(q, k, v, lens, out, lse=None, *, k_new=None, v_new=None, mask=None, n_new=None, heads=None, seqs=None,
               floor=0.0, where=""):
    """out [B,Hq,T,d] (and lse) against the oracle; k, v fp64 [B,H,cap,d]; mask [B,T,T] (None: causal). floor: what each row's
    share of an output may lose."""
    B, Hq, T, d = q.shape
    H, cap = k.shape[1:3]
    G = Hq // H
    qh, o = to64(q), to64(out)
    ls = None if lse is None else to64(lse)
    kn = vn = None
    if k_new is not None:
        kn, vn = to64(k_new), to64(v_new)
    for b in range(B) if seqs is None else seqs:
        n = max(0, min(int(lens[b]), cap))
        m = T if n_new is None else max(0, min(int(n_new[b]), T))
        sees = None
        if kn is not None:
            sees = np.tril(np.ones((T, T), dtype=bool)) if mask is None else np.asarray(mask[b], dtype=bool)
            sees = sees[:m, :m]
        assert not o[b, :, m:].any(), f"{where} b{b}: tokens that are not there"
        if ls is not None:
            assert np.all(ls[b, :, m:] == -np.inf), f"{where} b{b}: lse of tokens that are not there"
        for h in range(H) if heads is None else heads:
            for i in range(h * G, (h + 1) * G):
                new = (None, None) if kn is None else (kn[b, h, :m], vn[b, h, :m])
                ref, want, size, pv = do.attend(qh[b, i, :m], k[b, h, :n], v[b, h, :n], *new, sees)
                # bf16 calls of more than sixteen rows a KV head round every weight to bf16, by half a step (a value
                # 1.f x 2^e has steps of 2^(e - 7): at most 2^-8 of it), and sum the weights up as they were: the output moves by
                # 2^-8 sum p |v| at most
                coarse = 2.0 ** -8 if out.dtype == torch.bfloat16 and G * T > 16 else 0.0
                for t in range(m):
                    at = f"{where} b{b} h{h} i{i} t{t} n{n}"
                    tol = out_tolerance(ref[t], pv[t], d, n + m, size[t], out.dtype) + coarse * pv[t] * (1 + 2.0 ** -8) + (n + m) * floor
                    err = np.abs(o[b, i, t] - ref[t])
                    assert np.all(err <= tol), f"{at}: {err.max():.3g} of {tol[err.argmax()]:.3g}"
                    if ls is None:
                        continue
                    if want[t] == -np.inf:
                        assert ls[b, i, t] == -np.inf, at
                    else:   # the sum's relative error, the maximum's, and what is rounded at the end
                        tol = weight_error(d, n + m, size[t]) + (np.abs(want[t]) + size[t] + 8) * 2.0 ** -22
                        assert abs(ls[b, i, t] - want[t]) <= tol, f"{at}: lse {ls[b, i, t]} not {want[t]} +- {tol:.3g}"


# bf16 calls over 8-bit caches sum outputs up at 2^-53 of their size, in fp32, whose smallest step is 2^-149
Q8_FLOOR = 2.0 ** -96


def q8_rows(x):
    """The cache tensors (codes, steps) of rows x fp64 [B,H,cap,d], on the CPU, and the values they stand for."""
    sign, u, h = do.quantise(x)
    code = do.codes(sign, u)
    return torch.from_numpy(code), torch.from_numpy(h.astype(np.float32)), do.values(code, h)
