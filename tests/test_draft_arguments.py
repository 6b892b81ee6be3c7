"""Arguments of the binding of include/snapkv_draft.h that only look like others. No GPU needed."""
import contextlib

import pytest
import torch

from kv_cache_compression_gb300 import build as kbuild
from kv_cache_compression_gb300 import cache as kc
from kv_cache_compression_gb300 import draft as kd
from kv_cache_compression_gb300 import snapkv as sk


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kd.lib()


@pytest.mark.parametrize("counted", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_a_pick_of_no_rows_is_not_taken_for_no_pick(q8, counted):
    """A tensor without elements has address 0, which the library reads as "no pick: all rows"."""
    B, H, cap, d, T = 2, 2, 8, 64, 3
    new, n = torch.zeros(B, H, T, d), torch.zeros(B, dtype=torch.int32)
    pick = torch.zeros(B, T, dtype=torch.int32)[:, :0]
    held = (kd.Q8Cache.empty(B, H, cap, d, "cpu"),) if q8 else (torch.zeros(B, H, cap, d), torch.zeros(B, H, cap, d))
    call = kd.q8_append if q8 else kd.append_rows
    with pytest.raises(sk.SnapKVError) as refused:
        call(*held, new, new.clone(), n, pick=pick, n_new=n.clone() if counted else None)
    assert refused.value.status == sk.ERR_INVALID_ARG
    with pytest.raises(ValueError, match="pick has shape"):
        call(*held, new, new.clone(), n, pick=torch.zeros(B + 1, 0, dtype=torch.int32))


@pytest.mark.parametrize("name", ["evict", "q4_evict", "q8_read", "q4_read"])
def test_numbers_of_numpy_go_with_a_stream(monkeypatch, name):
    """NumPy's numbers have a device, too ("cpu"): it is not a tensor's."""
    np = pytest.importorskip("numpy")

    class Stream:
        device = torch.device("cpu")

    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    B, H, cap, d = 1, 2, 8, 64
    n = torch.zeros(B, dtype=torch.int32)
    dense = (torch.zeros(B, H, cap, d), torch.zeros(B, H, cap, d))
    score = torch.zeros(B, H, cap)
    q4, q8 = kc.Q4Cache.empty(B, H, cap, d, "cpu"), kd.Q8Cache.empty(B, H, cap, d, "cpu")
    call = {"evict": lambda k, **kw: kc.evict(*dense, score, n, keep=k, recent=k, want_idx=False, **kw),
            "q4_evict": lambda k, **kw: kc.q4_evict(q4, score, n, keep=k, recent=k, want_idx=False, **kw),
            "q8_read": lambda k, **kw: kd.q8_read(q8, k, **kw), "q4_read": lambda k, **kw: kc.q4_read(q4, k, **kw)}[name]
    with pytest.raises(ValueError, match="needs CUDA tensors"):   # (as far as a call comes without a GPU)
        call(np.int64(2), stream=Stream())
    Stream.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream is of cuda:1"):
        call(2, stream=Stream())
