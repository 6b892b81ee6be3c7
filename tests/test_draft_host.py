"""Host checks of include/snapkv_draft.h: exported symbols, refusals before any CUDA call, the binding's argument
checks, and the oracle of the 8-bit format. No GPU needed."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from kv_cache_compression_gb300 import build as kbuild
from kv_cache_compression_gb300 import draft as kd
from kv_cache_compression_gb300 import snapkv as sk
from oracle import draft_oracle as do

P = ctypes.c_void_p
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kd.lib()


def test_every_declared_function_is_exported(lib):
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "snapkv_draft.h")
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    names = set(re.findall(r"\b(snapkv_\w+)\s*\(", text))
    assert names == {"snapkv_tree_workspace_size", "snapkv_tree_attend", "snapkv_q8_tree_attend", "snapkv_append_rows",
                     "snapkv_q8_append", "snapkv_q8_read"}
    for n in names:
        assert hasattr(lib, n), n
    assert ctypes.sizeof(kd._Q8Struct) == 56 and kd._Q8Struct.batch.offset == 40


def test_workspace_sizes(lib):
    size = kd.tree_workspace_size
    assert size(2, 8, 4, 128, 8, 256) == 0 and size(2, 8, 4, 128, 9, 256) > 0 and size(2, 8, 4, 128, 8, 257) > 0   # short: none
    assert size(2, 8, 4, 128, 5, 1000) > 0 and size(2, 8, 4, 128, 5, 1000) % 256 == 0
    assert size(64, 32, 32, 128, 64, 1 << 30) < 64 << 20          # bounded, whatever the cache's length
    for bad in ((0, 8, 4, 128, 5, 9), (2, 9, 4, 128, 5, 9), (2, 8, 4, 96, 5, 9), (2, 8, 4, 128, 0, 9), (2, 8, 4, 128, 5, 0),
                (2, 2, 4, 128, 5, 9), (1, 1 << 12, 1, 64, 1 << 11, 9), (65536, 1, 1, 64, 1, 9), (1, 2, 2, 64, -1, 9)):
        assert size(*bad) == 0, bad


def _tree(lib, **kw):
    a = dict(q=MB, k=2 * MB, v=4 * MB, cap=300, len_=6 * MB, kn=7 * MB, vn=8 * MB, n=9 * MB, mask=10 * MB, stride=25, out=11 * MB,
             lse=12 * MB, B=2, Hq=4, H=2, d=64, T=5, dt=1, ws=16 * MB, wsb=64 * MB, dev=None)
    a.update(kw)
    return lib.snapkv_tree_attend(P(a["q"]), P(a["k"]), P(a["v"]), a["cap"], P(a["len_"]), P(a["kn"]), P(a["vn"]), P(a["n"]),
                                  P(a["mask"]), a["stride"], P(a["out"]), P(a["lse"]), a["B"], a["Hq"], a["H"], a["d"],
                                  a["T"], a["dt"], P(a["ws"]), a["wsb"], P(a["dev"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), sk.ERR_INVALID_ARG), (dict(k=0), sk.ERR_INVALID_ARG), (dict(v=0), sk.ERR_INVALID_ARG),
    (dict(len_=0), sk.ERR_INVALID_ARG), (dict(out=0), sk.ERR_INVALID_ARG), (dict(kn=0), sk.ERR_INVALID_ARG),
    (dict(vn=0), sk.ERR_INVALID_ARG), (dict(kn=0, vn=0), sk.ERR_INVALID_ARG),        # a mask without drafted rows
    (dict(stride=24), sk.ERR_INVALID_ARG), (dict(stride=-25), sk.ERR_INVALID_ARG), (dict(T=0), sk.ERR_INVALID_ARG),
    (dict(T=1 << 20), sk.ERR_INVALID_ARG), (dict(Hq=3), sk.ERR_INVALID_ARG), (dict(Hq=1), sk.ERR_INVALID_ARG),
    (dict(Hq=0), sk.ERR_INVALID_ARG), (dict(d=96), sk.ERR_UNSUPPORTED), (dict(d=0), sk.ERR_INVALID_ARG),
    (dict(dt=2), sk.ERR_INVALID_ARG), (dict(cap=0), sk.ERR_INVALID_ARG), (dict(cap=(1 << 30) + 1), sk.ERR_INVALID_ARG),
    (dict(B=0), sk.ERR_INVALID_ARG), (dict(B=32768, Hq=2), sk.ERR_INVALID_ARG), (dict(k=2 * MB + 8), sk.ERR_INVALID_ARG),
    (dict(vn=8 * MB + 8), sk.ERR_INVALID_ARG), (dict(lse=12 * MB + 2), sk.ERR_INVALID_ARG),
    (dict(n=9 * MB + 1), sk.ERR_INVALID_ARG), (dict(out=MB), sk.ERR_INVALID_ARG), (dict(out=2 * MB), sk.ERR_INVALID_ARG),
    (dict(out=7 * MB), sk.ERR_INVALID_ARG), (dict(out=10 * MB - 2048), sk.ERR_INVALID_ARG),
    (dict(lse=11 * MB), sk.ERR_INVALID_ARG), (dict(lse=9 * MB), sk.ERR_INVALID_ARG), (dict(dev=6 * MB), sk.ERR_INVALID_ARG),
    (dict(ws=0), sk.ERR_WORKSPACE), (dict(ws=16 * MB + 128), sk.ERR_WORKSPACE), (dict(wsb=100), sk.ERR_WORKSPACE),
    (dict(ws=8 * MB), sk.ERR_INVALID_ARG), (dict(ws=2 * MB), sk.ERR_INVALID_ARG),
])
def test_tree_refusals(lib, kw, status):
    assert _tree(lib, **kw) == status


def _cache(**kw):
    a = dict(kc=32 * MB, ks=33 * MB, vc=34 * MB, vs=35 * MB, cap=300, B=2, H=2, d=64)
    a.update(kw)
    return kd._Q8Struct(a["kc"], a["ks"], a["vc"], a["vs"], a["cap"], a["B"], a["H"], a["d"])


@pytest.mark.parametrize("kw,status", [
    (dict(kc=0), sk.ERR_INVALID_ARG), (dict(vs=0), sk.ERR_INVALID_ARG), (dict(vc=34 * MB + 8), sk.ERR_INVALID_ARG),
    (dict(ks=33 * MB + 2), sk.ERR_INVALID_ARG), (dict(cap=0), sk.ERR_INVALID_ARG), (dict(d=32), sk.ERR_UNSUPPORTED),
    (dict(H=0), sk.ERR_INVALID_ARG), (dict(B=65536), sk.ERR_INVALID_ARG),
])
def test_bad_caches_are_refused_by_every_call(lib, kw, status):
    for c, want in ((ctypes.byref(_cache(**kw)), status), (None, sk.ERR_INVALID_ARG)):
        assert lib.snapkv_q8_append(c, P(MB), P(2 * MB), 1, None, 0, None, P(3 * MB), P(4 * MB), 1, None, None) == want
        assert lib.snapkv_q8_read(c, None, 1, P(MB), P(2 * MB), 1, None) == want
        assert lib.snapkv_q8_tree_attend(P(MB), c, P(3 * MB), None, None, None, None, 0, P(4 * MB), None, 4, 1, 1,
                                         P(5 * MB), MB, None, None) == want


def test_q8_tree_refusals(lib):
    c = ctypes.byref(_cache())

    def call(q=MB, kn=None, vn=None, mask=None, stride=0, out=2 * MB, lse=None, hq=4, T=3, dt=1, ws=40 * MB, wsb=64 * MB):
        return lib.snapkv_q8_tree_attend(P(q), c, P(3 * MB), P(kn), P(vn), None, P(mask), stride, P(out), P(lse), hq, T, dt,
                                         P(ws), wsb, None, None)
    assert call(q=0) == call(out=0) == call(hq=5) == call(T=0) == call(dt=7) == call(kn=4 * MB) == sk.ERR_INVALID_ARG
    assert call(mask=4 * MB) == call(kn=4 * MB, vn=5 * MB, mask=6 * MB, stride=3) == sk.ERR_INVALID_ARG
    assert call(out=32 * MB) == call(lse=33 * MB) == call(out=35 * MB) == call(ws=34 * MB) == sk.ERR_INVALID_ARG
    assert call(ws=0) == call(wsb=16) == call(ws=40 * MB + 64) == sk.ERR_WORKSPACE


@pytest.mark.parametrize("q8", [False, True])
def test_append_refusals(lib, q8):
    c = ctypes.byref(_cache())

    def call(kc=20 * MB, vc=24 * MB, kn=MB, vn=2 * MB, rows=4, pick=5 * MB, picks=3, n=None, lin=3 * MB, lout=4 * MB, dt=1):
        rest = (P(kn), P(vn), rows, P(pick), picks, P(n), P(lin), P(lout))
        if q8:
            return lib.snapkv_q8_append(c, *rest, dt, None, None)
        return lib.snapkv_append_rows(P(kc), P(vc), 300, *rest, 2, 2, 64, dt, None, None)
    assert call(kn=0) == call(vn=0) == call(lin=0) == call(lout=0) == sk.ERR_INVALID_ARG
    assert call(rows=0) == call(rows=-1) == call(rows=(1 << 30) + 1) == call(dt=4) == sk.ERR_INVALID_ARG
    assert call(picks=0) == call(picks=-2) == call(picks=1 << 31) == sk.ERR_INVALID_ARG
    assert call(kn=MB + 8) == call(pick=5 * MB + 2) == call(lout=4 * MB + 1) == sk.ERR_INVALID_ARG
    assert call(lout=3 * MB) == call(lout=5 * MB + 8) == call(n=4 * MB) == sk.ERR_INVALID_ARG
    assert call(lout=MB) == call(kn=32 * MB if q8 else 20 * MB) == sk.ERR_INVALID_ARG
    if not q8:
        assert call(kc=0) == call(vc=20 * MB) == call(vc=24 * MB + 4) == sk.ERR_INVALID_ARG
        assert lib.snapkv_append_rows(P(MB), P(2 * MB), 300, P(3 * MB), P(4 * MB), 1, None, 0, None, P(5 * MB), P(6 * MB), 2, 2,
                                      80, 1, None, None) == sk.ERR_UNSUPPORTED


def test_read_refusals(lib):
    c = ctypes.byref(_cache())

    def read(k=MB, v=2 * MB, rows=4, start=None, dt=1):
        return lib.snapkv_q8_read(c, P(start), rows, P(k), P(v), dt, None)
    assert read(k=0) == read(rows=0) == read(dt=2) == read(v=MB) == read(start=3 * MB + 1) == sk.ERR_INVALID_ARG
    assert read(v=33 * MB) == read(k=MB + 4) == read(start=MB) == sk.ERR_INVALID_ARG


def test_the_binding_checks_its_tensors(lib):
    B, H, cap, d, T = 2, 2, 8, 64, 3
    k, q, n = torch.zeros(B, H, cap, d), torch.zeros(B, 4, T, d), torch.zeros(B, dtype=torch.int32)
    new, mask = torch.zeros(B, H, T, d), torch.ones(B, T, T, dtype=torch.bool)
    call = kd.tree_attend
    with pytest.raises(ValueError, match="CUDA"):
        call(q, k, k.clone(), n, new, new.clone(), mask)
    with pytest.raises(ValueError, match="q must be"):
        call(q[:, :, 0], k, k.clone(), n)
    with pytest.raises(ValueError, match="v_cache has shape"):
        call(q, k, k[:, :, :4], n)
    with pytest.raises(TypeError, match="k_cache is"):
        call(q, k.bfloat16(), k, n)
    with pytest.raises(ValueError, match="go together"):
        call(q, k, k.clone(), n, new)
    with pytest.raises(ValueError, match="needs k_new"):
        call(q, k, k.clone(), n, mask=mask)
    with pytest.raises(TypeError, match="mask is"):
        call(q, k, k.clone(), n, new, new.clone(), mask.int())
    with pytest.raises(ValueError, match="mask has shape"):
        call(q, k, k.clone(), n, new, new.clone(), mask[:, :, :2])
    with pytest.raises(ValueError, match="mask must be contiguous"):
        call(q, k, k.clone(), n, new, new.clone(), mask.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="k_new has shape"):
        call(q, k, k.clone(), n, new[:, :, :2], new)
    with pytest.raises(ValueError, match="lse has shape"):
        call(q, k, k.clone(), n, lse=torch.zeros(B, H, T))
    with pytest.raises(TypeError, match="n_new is"):
        call(q, k, k.clone(), n, n_new=n.long())
    with pytest.raises(ValueError, match="out has shape"):
        call(q, k, k.clone(), n, out=torch.zeros(B, 4, T + 1, d))
    for bad in (torch.zeros(B, 3, T, d), torch.zeros(B, 4, 0, d)):
        with pytest.raises(sk.SnapKVError):
            call(bad, k, k.clone(), n)
    with pytest.raises(TypeError):
        call(q.half(), k.half(), k.half(), n)
    c = kd.Q8Cache.empty(B, H, cap, d, "cpu")
    assert c.shape == (B, H, cap, d) and c.k_step.shape == (B, H, cap)
    with pytest.raises(ValueError, match="k_codes"):
        kd.Q8Cache(c.k_codes[..., :32], c.k_step, c.v_codes, c.v_step)
    with pytest.raises(ValueError, match="v_step"):
        kd.Q8Cache(c.k_codes, c.k_step, c.v_codes, c.v_step[:, :, :4])
    with pytest.raises(ValueError, match="CUDA"):
        kd.q8_tree_attend(q, c, n, new, new.clone())
    with pytest.raises(ValueError, match="v_new has shape"):
        kd.q8_append(c, new, new[:, :1], n)
    with pytest.raises(ValueError, match="pick must be"):
        kd.append_rows(k, k.clone(), new, new, n, pick=n)
    with pytest.raises(ValueError, match="pick has shape"):
        kd.append_rows(k, k.clone(), new, new, n, pick=torch.zeros(B + 1, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="k_new is"):
        kd.append_rows(k, k.clone(), new.bfloat16(), new, n)
    with pytest.raises(ValueError, match="CUDA"):
        kd.q8_append(c, new, new.clone(), n)
    with pytest.raises(sk.SnapKVError):
        kd.q8_read(c, 0)
    with pytest.raises(ValueError, match="v_out has shape"):
        kd.q8_read(c, 2, v_out=torch.zeros(B, H, 3, d).bfloat16())

    class Elsewhere:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream is of cuda:1"):
        kd.q8_read(c, 1, stream=Elsewhere())
    with pytest.raises(ValueError, match="stream is of cuda:1"):
        call(q, k, k.clone(), n, stream=Elsewhere())


# ------------------------------------------------------------------------------- the oracle itself

def test_the_format_holds_its_own_values():
    """Every code with a step is found again from the value it stands for, if the row's largest is 127 steps."""
    code = np.arange(256, dtype=np.uint8).reshape(2, 128)
    for h in (1.0, 2.0 ** -60, 3.0 * 2.0 ** 20):
        x = do.values(code, np.array([h, h]))
        sign, u, step = do.quantise(x)
        assert np.all(step == h) and np.array_equal(do.codes(sign, u) & 127, code & 127)
        assert np.array_equal(do.values(do.codes(sign, u), step), x)


def test_quantisation_is_within_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((300, 128)) * np.exp2(rng.integers(-40, 40, size=(300, 1)))
    sign, u, h = do.quantise(x)
    assert u.max() <= 127
    err = np.abs(do.values(do.codes(sign, u), h) - x)
    assert np.all(err <= 0.5 * h[:, None] * (1 + 2.0 ** -20))
    zero = do.quantise(np.full((1, 64), 2.0 ** -74))
    assert zero[2][0] == 0 and not zero[1].any()                     # 2^-74 / 127 is below 2^-80
    assert do.quantise(np.full((1, 64), 2.0 ** -73))[2][0] > 0
    assert np.isnan(do.quantise(np.array([[1.0, np.inf]]))[2][0]) and np.isnan(do.quantise(np.array([[np.nan, 1.0]]))[2][0])


def test_ties_go_to_the_even_magnitude():
    x = np.zeros((1, 64))
    x[0, :8] = [127, 0.5, 1.5, 2.5, -0.5, -3.5, 126.5, 125.5]
    sign, u, h = do.quantise(x)
    assert h[0] == 1 and list(u[0, :8]) == [127, 0, 2, 2, 0, 4, 126, 126] and sign[0, 5] == -1


def test_attention_oracle_on_a_written_out_case():
    q = np.array([[8.0] + [0.0] * 63] * 3)
    k = np.zeros((1, 64))
    new = np.zeros((3, 64))
    new[:, 0] = np.log([2.0, 4.0, np.e])     # logits ln 2, ln 4, 1 (8 / sqrt(64) = 1)
    v, v_new = np.full((1, 64), 1.0), np.arange(3.0)[:, None] * np.ones(64)
    mask = np.array([[1, 0, 0], [1, 1, 0], [0, 0, 0]], dtype=bool)
    out, lse, _, _ = do.attend(q, k, v, new, v_new, mask)
    assert np.allclose(out[:, 0], [(1 + 0) / 3, (1 + 0 + 4) / 7, 1.0]) and np.allclose(lse, np.log([3, 7, 1]))
    out, lse, _, _ = do.attend(q, k[:0], v[:0], new, v_new, mask)
    assert not out[2].any() and lse[2] == -np.inf
