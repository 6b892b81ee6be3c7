"""pytest plugin (-p tests.watch_draft_status): calls of the operators for drafted tokens that pass no status word get one, and a
test in which a kernel reports a violated bound or a wait that ran out fails, although most tests do not look at it."""
import pytest


@pytest.fixture(autouse=True)
def watched_draft_status(monkeypatch):
    import torch
    from kv_cache_compression_gb300 import draft, snapkv
    words = [torch.zeros(1, dtype=torch.int32, device=f"cuda:{i}") for i in range(torch.cuda.device_count())]
    torch.cuda.synchronize()
    given = draft._status
    monkeypatch.setattr(draft, "_status", lambda t, device: given(t, device) if t is not None or device.type != "cuda"
                        else words[device.index].data_ptr())
    yield
    for word in words:
        torch.cuda.synchronize(word.device)
        assert word.item() & (snapkv.ERR_INTERNAL | snapkv.ERR_TIMEOUT) == 0, f"status {word.item()}"
