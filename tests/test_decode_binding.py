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
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
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


def test_a_captured_call_gets_scratch_of_its_own(host, monkeypatch):
    """While a graph is being captured the scratch is fresh at every call and not kept: a replay may come at any time, also
    after a larger call has replaced the cached buffer, and beside another graph's."""
    stream = FakeStream(21)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    cached = sv.workspace(1000, host, stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    first, second = sv.workspace(1000, host, stream), sv.workspace(1000, host, stream)
    assert len({x.data_ptr() for x in (cached, first, second)}) == 3
    assert first.numel() == second.numel() == 1000 and first.dtype == torch.uint8
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    assert sv.workspace(1000, host, stream) is cached
    fresh = FakeStream(22)  # nothing is cached: what a capture takes is not kept either
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    one = sv.workspace(1000, host, fresh)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    assert sv.workspace(1000, host, fresh) is not one


def test_the_capture_that_counts_is_that_of_the_calls_own_stream(monkeypatch):
    """A call on another stream than the current one asks about its own."""
    now, capturing = [FakeStream(1)], {2}

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[-1].cuda_stream in capturing)
    device, plain, captured = torch.device("cpu", 0), FakeStream(1), FakeStream(2)
    assert sv.workspace(100, device, plain) is sv.workspace(100, device, plain)
    assert sv.workspace(100, device, captured) is not sv.workspace(100, device, captured)


def test_tensors_on_another_device_than_the_current_one_are_refused(monkeypatch):
    """The library launches on the current device, so tensors of another would be reached from the wrong GPU."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    sv._launches_on(1)
    for index in (0, 2):
        with pytest.raises(ValueError, match=f"cuda:{index}.*cuda:1"):
            sv._launches_on(index)


def test_sizes_that_have_no_workspace_are_left_to_the_call():
    """Zero bytes, not an error of the binding's own: the library tells sizes beyond a limit from impossible ones."""
    sv._build.build()
    for T, q_heads, heads, D in ((65, 4, 2, 64), (2, 4, 2, 96), (2, 129, 1, 64), (2, 3, 2, 64)):
        assert sv.decode._attention_bytes(T, q_heads, heads, D) == 0
    assert sv.decode._attention_bytes(2, 4, 2, 64) > 0


def test_a_callers_workspace_is_checked():
    """Bytes on the device of the call, without gaps: the library writes numel() of them behind the address."""
    device = torch.device("cpu", 0)
    good = torch.zeros(512, dtype=torch.uint8)
    assert sv._given_workspace(good, good.device) is good
    with pytest.raises(TypeError, match="uint8"):
        sv._given_workspace(good.view(torch.float32), good.device)
    with pytest.raises(ValueError, match="expected cuda:0"):
        sv._given_workspace(good, torch.device("cuda", 0))
    with pytest.raises(ValueError, match="contiguous"):
        sv._given_workspace(good[::2], good.device)


def test_two_threads_never_share_a_staging_buffer(host, monkeypatch):
    """verify_host blocks its own thread only: another one's call may copy its inputs in meanwhile."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    got, both = {}, threading.Barrier(2)

    def work(name):
        first = sv._staging(1000, host)
        both.wait(20)
        got[name] = (first, sv._staging(500, host))
        both.wait(20)

    threads = [threading.Thread(target=work, args=(n,)) for n in "ab"]
    for t in threads:
        t.start()
    for t in threads:
        t.join(20)
    assert all(first is again for first, again in got.values())
    assert got["a"][0].data_ptr() != got["b"][0].data_ptr()
