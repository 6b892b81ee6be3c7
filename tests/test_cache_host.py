"""Host checks of include/snapkv_cache.h: exported symbols, refusals before any CUDA call, the
binding's argument checks, and the oracle of the 4-bit format. No GPU needed."""
import ctypes
import re

import numpy as np
import pytest
import torch

from kv_cache_compression_gb300 import build as kbuild
from kv_cache_compression_gb300 import cache as kc
from kv_cache_compression_gb300 import snapkv as sk
from oracle import cache_oracle as co
from tests.cache_cases import q4_inputs

P = ctypes.c_void_p
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kc.lib()


def test_every_declared_function_is_exported(lib):
    import os
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "snapkv_cache.h")
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    names = set(re.findall(r"\b(snapkv_\w+)\s*\(", text))
    assert names == {"snapkv_scored_workspace_size", "snapkv_decode_attend_scored", "snapkv_q4_append", "snapkv_q4_read",
                     "snapkv_q4_decode_attend", "snapkv_evict_workspace_size", "snapkv_evict", "snapkv_q4_evict"}
    for n in names:
        assert hasattr(lib, n), n
    assert ctypes.sizeof(kc._Q4Struct) == 56 and kc._Q4Struct.batch.offset == 40


def test_workspace_sizes(lib):
    plain, scored = (kc.scored_workspace_size(2, 8, 4, 128, 1000, s) for s in (False, True))
    assert plain > 0 and scored - plain == 2 * 4 * 1000 * 2 * 4                        # a logit per query and row
    wide = [kc.scored_workspace_size(2, 64, 4, 128, 1000, s) for s in (False, True)]   # eight queries at a time
    assert wide[1] - wide[0] == 2 * 64 * 1000 * 4
    assert kc.scored_workspace_size(1, 3, 2, 128, 1000) == 0                          # not a multiple
    assert kc.scored_workspace_size(1, 2, 2, 96, 1000) == 0
    assert kc.scored_workspace_size(2, 8, 4, 128, 256) == 0                            # short: none
    assert kc.scored_workspace_size(2, 64, 4, 128, 256) > 0                            # unless in several passes
    assert kc.evict_workspace_size(2, 3, 2048) == 0                                    # short: none
    assert kc.evict_workspace_size(2, 3, 2049) == 49408                                # 49176, in 256s
    assert kc.evict_workspace_size(2, 3, 0) == 0
    assert kc.evict_workspace_size(65536, 1, 10) == 0


def _attend(lib, **kw):
    a = dict(q=MB, k=2 * MB, v=4 * MB, cap=300, len_=6 * MB, score=7 * MB, decay=1.0, out=8 * MB, B=2, Hq=4, H=2,
             d=64, dt=1, ws=9 * MB, wsb=1 << 19, dev=None)
    a.update(kw)
    return lib.snapkv_decode_attend_scored(P(a["q"]), P(a["k"]), P(a["v"]), a["cap"], P(a["len_"]), P(a["score"]),
                                           a["decay"], P(a["out"]), a["B"], a["Hq"], a["H"], a["d"], a["dt"],
                                           P(a["ws"]), a["wsb"], P(a["dev"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), sk.ERR_INVALID_ARG), (dict(k=0), sk.ERR_INVALID_ARG), (dict(v=0), sk.ERR_INVALID_ARG),
    (dict(len_=0), sk.ERR_INVALID_ARG), (dict(out=0), sk.ERR_INVALID_ARG), (dict(k=2 * MB + 8), sk.ERR_INVALID_ARG),
    (dict(score=7 * MB + 4), sk.ERR_INVALID_ARG), (dict(len_=6 * MB + 2), sk.ERR_INVALID_ARG),
    (dict(Hq=3), sk.ERR_INVALID_ARG), (dict(Hq=0), sk.ERR_INVALID_ARG), (dict(Hq=1), sk.ERR_INVALID_ARG),
    (dict(d=96), sk.ERR_UNSUPPORTED), (dict(d=0), sk.ERR_INVALID_ARG), (dict(dt=2), sk.ERR_INVALID_ARG),
    (dict(cap=0), sk.ERR_INVALID_ARG), (dict(cap=(1 << 30) + 1), sk.ERR_INVALID_ARG), (dict(B=0), sk.ERR_INVALID_ARG),
    (dict(B=32768, H=2, Hq=2), sk.ERR_INVALID_ARG), (dict(Hq=1 << 22), sk.ERR_INVALID_ARG), (dict(decay=-0.1), sk.ERR_INVALID_ARG),
    (dict(decay=1.5), sk.ERR_INVALID_ARG), (dict(decay=float("nan")), sk.ERR_INVALID_ARG),
    (dict(ws=0), sk.ERR_WORKSPACE), (dict(ws=9 * MB + 16), sk.ERR_WORKSPACE), (dict(wsb=100), sk.ERR_WORKSPACE),
    (dict(out=2 * MB), sk.ERR_INVALID_ARG),          # the output over the keys
    (dict(out=MB), sk.ERR_INVALID_ARG),              # over the queries
    (dict(score=4 * MB), sk.ERR_INVALID_ARG),        # the score over the values
    (dict(ws=7 * MB), sk.ERR_INVALID_ARG),           # the workspace over the score
    (dict(ws=2 * MB, score=0), sk.ERR_INVALID_ARG),  # over the keys
    (dict(dev=6 * MB), sk.ERR_INVALID_ARG),          # the status word over the lengths
])
def test_attend_refusals(lib, kw, status):
    assert _attend(lib, **kw) == status


def test_short_bf16_calls_of_up_to_sixteen_queries_need_no_workspace(lib):
    """The size serves either type; a call asks for what its own type needs. (These calls are refused after that, for an
    output that lies over the queries.)"""
    short = dict(ws=0, wsb=0, cap=256, out=MB, Hq=32, H=2)
    assert kc.scored_workspace_size(2, 32, 2, 64, 256) > 0
    assert _attend(lib, **short) == sk.ERR_INVALID_ARG
    assert _attend(lib, **short, dt=0) == sk.ERR_WORKSPACE                 # fp32: two passes
    assert _attend(lib, **dict(short, cap=257)) == sk.ERR_WORKSPACE
    assert _attend(lib, **dict(short, Hq=34)) == sk.ERR_WORKSPACE          # seventeen queries: two passes
    for q_heads, cap, dtype, none in ((32, 256, torch.bfloat16, True), (32, 256, torch.float32, False), (18, 1, torch.bfloat16, True),
                                      (34, 256, torch.bfloat16, False), (32, 257, torch.bfloat16, False)):
        assert (kc.scored_workspace_size(2, q_heads, 2, 64, cap, True, dtype) == 0) == none
    assert kc.scored_workspace_size(2, 8, 2, 64, 1000, True, torch.bfloat16) == kc.scored_workspace_size(2, 8, 2, 64, 1000)


def _cache(**kw):
    a = dict(kc=16 * MB, km=17 * MB, vc=18 * MB, vm=19 * MB, cap=300, B=2, H=2, d=64)
    a.update(kw)
    return kc._Q4Struct(a["kc"], a["km"], a["vc"], a["vm"], a["cap"], a["B"], a["H"], a["d"])


@pytest.mark.parametrize("kw,status", [
    (dict(kc=0), sk.ERR_INVALID_ARG), (dict(vm=0), sk.ERR_INVALID_ARG), (dict(km=17 * MB + 4), sk.ERR_INVALID_ARG),
    (dict(cap=0), sk.ERR_INVALID_ARG), (dict(d=32), sk.ERR_UNSUPPORTED), (dict(H=0), sk.ERR_INVALID_ARG),
])
def test_bad_caches_are_refused_by_every_call(lib, kw, status):
    c = ctypes.byref(_cache(**kw))
    assert lib.snapkv_q4_append(c, P(MB), P(2 * MB), 1, None, P(3 * MB), P(4 * MB), 1, None, None) == status
    assert lib.snapkv_q4_read(c, None, 1, P(MB), P(2 * MB), 1, None) == status
    assert lib.snapkv_q4_decode_attend(P(MB), c, P(3 * MB), None, 1.0, P(4 * MB), 4, 1, P(5 * MB), MB, None, None) == status
    assert lib.snapkv_q4_evict(c, P(MB), P(3 * MB), P(4 * MB), 10, 5, None, P(5 * MB), MB, None, None) == status
    assert lib.snapkv_q4_append(None, P(MB), P(2 * MB), 1, None, P(3 * MB), P(4 * MB), 1, None, None) \
        == sk.ERR_INVALID_ARG


def test_q4_refusals(lib):
    c = ctypes.byref(_cache())

    def append(k=MB, v=2 * MB, rows=4, n_new=None, lin=3 * MB, lout=4 * MB, dt=1):
        return lib.snapkv_q4_append(c, P(k), P(v), rows, P(n_new), P(lin), P(lout), dt, None, None)
    assert append(k=0) == append(lin=0) == append(lout=0) == sk.ERR_INVALID_ARG
    assert append(rows=0) == append(rows=-1) == append(dt=5) == append(v=2 * MB + 8) == sk.ERR_INVALID_ARG
    assert append(lout=3 * MB) == append(lout=3 * MB + 4) == sk.ERR_INVALID_ARG       # overlaps len_in
    assert append(n_new=4 * MB) == sk.ERR_INVALID_ARG                                  # overlaps len_out
    assert append(k=16 * MB) == sk.ERR_INVALID_ARG                                     # reads what it writes

    def read(k=MB, v=2 * MB, rows=4, start=None, dt=1):
        return lib.snapkv_q4_read(c, P(start), rows, P(k), P(v), dt, None)
    assert read(k=0) == read(rows=0) == read(dt=2) == read(k=2 * MB) == read(start=3 * MB + 1) == sk.ERR_INVALID_ARG
    assert read(v=19 * MB) == sk.ERR_INVALID_ARG                                       # over the cache

    def attend(q=MB, out=2 * MB, hq=4, score=None, ws=6 * MB, wsb=MB, decay=1.0):
        return lib.snapkv_q4_decode_attend(P(q), c, P(3 * MB), P(score), decay, P(out), hq, 1, P(ws), wsb, None, None)
    assert attend(q=0) == attend(out=0) == attend(hq=3) == attend(out=16 * MB) == attend(decay=2.0) == sk.ERR_INVALID_ARG
    assert attend(ws=0) == attend(score=5 * MB, ws=6 * MB + 8) == attend(wsb=1000) == sk.ERR_WORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), sk.ERR_INVALID_ARG), (dict(score=0), sk.ERR_INVALID_ARG), (dict(lin=0), sk.ERR_INVALID_ARG),
    (dict(keep=-1), sk.ERR_INVALID_ARG), (dict(recent=-1), sk.ERR_INVALID_ARG),
    (dict(keep=0, recent=0), sk.ERR_INVALID_ARG), (dict(keep=2996), sk.ERR_INVALID_ARG),
    (dict(keep=1 << 62, recent=1 << 62), sk.ERR_INVALID_ARG),
    (dict(lout=3 * MB), sk.ERR_INVALID_ARG), (dict(idx=4 * MB), sk.ERR_INVALID_ARG), (dict(v=10 * MB), sk.ERR_INVALID_ARG),
    (dict(ws=0), sk.ERR_WORKSPACE), (dict(wsb=47999), sk.ERR_WORKSPACE), (dict(ws=7 * MB + 128), sk.ERR_WORKSPACE),
    (dict(ws=5 * MB), sk.ERR_INVALID_ARG), (dict(d=80), sk.ERR_UNSUPPORTED), (dict(dt=9), sk.ERR_INVALID_ARG),
])
def test_evict_refusals(lib, kw, status):
    a = dict(k=10 * MB, v=20 * MB, cap=3000, score=5 * MB, lin=3 * MB, lout=4 * MB, keep=50, recent=5, idx=6 * MB, d=64,
             dt=1, ws=7 * MB, wsb=48000)
    a.update(kw)
    assert lib.snapkv_evict(P(a["k"]), P(a["v"]), a["cap"], P(a["score"]), P(a["lin"]), P(a["lout"]), a["keep"],
                            a["recent"], P(a["idx"]), 2, 2, a["d"], a["dt"], P(a["ws"]), a["wsb"], None, None) == status


def test_the_binding_checks_its_tensors(lib):
    B, H, cap, d = 2, 2, 8, 64
    k = torch.zeros(B, H, cap, d)
    q, n, score = torch.zeros(B, 4, d), torch.zeros(B, dtype=torch.int32), torch.zeros(B, H, cap)
    with pytest.raises(ValueError, match="CUDA"):
        kc.decode_attend_scored(q, k, k.clone(), n, score)
    with pytest.raises(ValueError, match="v_cache has shape"):
        kc.decode_attend_scored(q, k, k[:, :, :4], n)
    with pytest.raises(TypeError, match="k_cache is"):
        kc.decode_attend_scored(q, k.bfloat16(), k, n)
    with pytest.raises(ValueError, match="contiguous"):
        kc.decode_attend_scored(q, k.transpose(1, 2).contiguous().transpose(1, 2), k, n)
    with pytest.raises(TypeError, match="len_ is"):
        kc.decode_attend_scored(q, k, k.clone(), n.long())
    with pytest.raises(ValueError, match="score has shape"):
        kc.decode_attend_scored(q, k, k.clone(), n, torch.zeros(B, H, cap + 1))
    with pytest.raises(sk.SnapKVError):
        kc.decode_attend_scored(torch.zeros(B, 3, d), k, k.clone(), n)
    with pytest.raises(TypeError):
        kc.decode_attend_scored(q.half(), k.half(), k.half(), n)
    c = kc.Q4Cache.empty(B, H, cap, d, "cpu")
    assert c.shape == (B, H, cap, d) and c.k_meta.shape == (B, H, cap, 1, 2)
    with pytest.raises(ValueError, match="k_codes"):
        kc.Q4Cache(c.k_codes[..., :16], c.k_meta, c.v_codes, c.v_meta)
    with pytest.raises(ValueError, match="v_meta"):
        kc.Q4Cache(c.k_codes, c.k_meta, c.v_codes, c.v_meta[:, :, :4])
    with pytest.raises(ValueError, match="v_new has shape"):
        kc.q4_append(c, k, k[:, :1], n)
    with pytest.raises(ValueError, match="CUDA"):
        kc.q4_append(c, k, k, n)
    with pytest.raises(ValueError, match="idx_out has shape"):
        kc.evict(k, k.clone(), score, n, keep=3, recent=2, idx_out=torch.zeros(B, H, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="len_in"):
        kc.q4_evict(c, score, n[:1], keep=3, recent=2)


# ------------------------------------------------------------------------------- the oracle itself

def _unpack(codes):
    """Levels from codes, word by word (the other direction of the oracle's pack)."""
    d = codes.shape[-1] * 2
    ng = d // 64
    words = codes.copy().view(np.uint32)
    t = np.zeros((*codes.shape[:-1], d), dtype=np.int64)
    for w in range(d // 8):
        for e in range(8):
            half = (words[..., w] >> np.uint32(16 * (e & 1))) & 0xFFFF
            j = e >> 1
            m = 2 * ((half >> np.uint32(co.MAG_BIT[j])) & 7).astype(np.int64) + 1
            s = (half >> np.uint32(co.SIGN_BIT[j])) & 1
            t[..., 64 * (w % ng) + 8 * (w // ng) + e] = np.where(s == 1, -m, m)
    return t


def test_the_binding_refuses_what_it_cannot_serve(lib):
    q, none = torch.zeros(1, 4, 64), torch.zeros(1, 0, 8, 64)
    n = torch.ones(1, dtype=torch.int32)
    with pytest.raises(sk.SnapKVError):   # no heads
        kc.decode_attend_scored(q, none, none, n)
    k, score = torch.zeros(1, 4, 8, 64), torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):   # (and no index of 2^50 rows is allocated first)
        kc.evict(k, k.clone(), score, n, keep=1 << 50, recent=0)

    class Elsewhere:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream is of cuda:1"):
        kc.decode_attend_scored(q, k, k, n, stream=Elsewhere())
    with pytest.raises(ValueError, match="stream is of cuda:1"):
        kc.q4_read(kc.Q4Cache.empty(1, 4, 8, 64, "cpu"), 1, stream=Elsewhere())


@pytest.mark.parametrize("keep,recent", [((1 << 64) + 3, 2), (3, 1 << 64), (1 << 63, 1 << 63), (-1, 4), (4, -1)])
def test_the_binding_refuses_counts_that_its_integers_do_not_hold(lib, keep, recent):
    """2^64 + 3 must not evict down to 3 rows."""
    k, score, n = torch.zeros(1, 4, 8, 64), torch.zeros(1, 4, 8), torch.ones(1, dtype=torch.int32)
    for want_idx in (True, False):
        with pytest.raises(sk.SnapKVError, match="snapkv_evict"):
            kc.evict(k, k.clone(), score, n, keep=keep, recent=recent, want_idx=want_idx)
        with pytest.raises(sk.SnapKVError, match="snapkv_q4_evict"):
            kc.q4_evict(kc.Q4Cache.empty(1, 4, 8, 64, "cpu"), score, n, keep=keep, recent=recent, want_idx=want_idx)


@pytest.mark.parametrize("d", [64, 128])
def test_every_level_survives_the_format(d):
    rng = np.random.default_rng(d)
    u = rng.integers(0, 16, size=(50, d))
    assert np.array_equal(_unpack(co.pack(u)), 2 * u - 15)
    # eight channels use all 32 bits of a word, each bit once
    used = np.zeros(32, dtype=int)
    for j in range(4):
        for half in (0, 16):
            used[half + co.SIGN_BIT[j]] += 1
            used[half + co.MAG_BIT[j]:half + co.MAG_BIT[j] + 3] += 1
    assert np.all(used == 1)


def test_quantisation_is_within_a_step():
    rng = np.random.default_rng(7)
    for scale in (1.0, 1e-4, 1e4):
        x = co.bf16(rng.standard_normal((200, 128)) * scale)
        u, h, z = co.quantise(x)
        err = np.abs(co.values(u, h, z) - x).reshape(200, 2, 64)
        # half a step of 2h; h rounded by 2^-9 over 15 levels and z by 2^-9 of itself at the ends
        assert np.all(err <= (h + 15 * h * 2.0 ** -8 + np.abs(z) * 2.0 ** -8)[..., None])
        assert set(np.unique(u)) <= set(range(16))
    u, h, z = co.quantise(np.full((1, 64), 3.0))
    assert np.all(u == 8) and h[0, 0] == 0 and co.values(u, h, z)[0, 0] == 3.0
    x = np.ones((1, 128))
    x[0, 70] = np.inf
    u, h, z = co.quantise(x)
    v = co.values(u, h, z)
    assert np.all(v[0, :64] == 1.0) and np.all(np.isnan(v[0, 64:]))


def test_codes_and_pairs_are_the_cache_tensors():
    u, h, z = co.quantise(np.random.default_rng(1).standard_normal((2, 3, 5, 64)))
    codes, meta = q4_inputs(u, h, z)
    assert codes.shape == (2, 3, 5, 32) and codes.dtype == torch.uint8
    assert meta.shape == (2, 3, 5, 1, 2) and torch.equal(meta[..., 0].double(), torch.from_numpy(h))


def test_eviction_oracle_on_a_written_out_case():
    #            0    1    2    3    4    5   6   7   8
    score = np.array([0.5, 0.1, 0.9, 0.1, 0.7, 0.6, np.nan, 9.0, 0.0])
    # recent 2 (slots 7, 8 stay whatever they weigh), of 0 .. 6 the four largest: 2, 4, 5, 0
    assert list(co.evict_slots(score, 9, 4, 2)) == [0, 4, 2, 5, 7, 8]
    # recent 1, of 0 .. 7 the five largest: 7, 2, 4, 5, 0; slots 1 and 3 are freed and take 5 and 7
    assert list(co.evict_slots(score, 9, 5, 1)) == [0, 5, 2, 7, 4, 8]
    # the six largest: slots 1 and 3 tie for the last place, the lower one stays
    assert list(co.evict_slots(score, 9, 6, 1)) == [0, 1, 2, 7, 4, 5, 8]
    assert list(co.evict_slots(score, 5, 4, 2)) == [0, 1, 2, 3, 4]        # not full: untouched
    assert list(co.evict_slots(score, 9, 0, 3)) == [6, 7, 8]
