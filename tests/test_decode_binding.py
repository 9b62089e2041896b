"""What the binding keeps and checks on the host, with stand-ins for the CUDA side (CPU only)."""
import contextlib
import threading

import pytest
import torch

import speculative_decoding_rejection_verify_gb300 as sv


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def host(monkeypatch):
    """torch.cuda as the workspaces see it, on the CPU."""
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return torch.device("cpu", 0)


def test_two_threads_never_share_a_workspace(host):
    """Each thread's scratch of one stream is its own, and is the same from call to call."""
    stream, got, both = FakeStream(11), {}, threading.Barrier(2)

    def work(name):
        first = sv.workspace(1000, host, stream)
        both.wait(20)
        again = sv.workspace(500, host, stream)
        got[name] = (first, again)
        both.wait(20)

    threads = [threading.Thread(target=work, args=(n,)) for n in "ab"]
    for t in threads:
        t.start()
    for t in threads:
        t.join(20)
    for first, again in got.values():
        assert first is again
    assert got["a"][0].data_ptr() != got["b"][0].data_ptr()
    assert sv.workspace(10, host, FakeStream(12)) is not sv.workspace(10, host, stream)
    assert sv.workspace(2000, host, stream).numel() == 2000
