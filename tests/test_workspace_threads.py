"""The binding's cached workspaces, without a GPU: one per device, stream and host thread."""
import threading

import pytest
import torch

import w4a16_gemm_awq_b200 as w4


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def cache(monkeypatch):
    """CPU tensors in the place of device memory, and a cache of the test's own."""
    monkeypatch.setattr(w4, "_workspaces", {})
    real = torch.zeros
    monkeypatch.setattr(w4.torch, "zeros", lambda n, dtype, device: real(n, dtype=dtype))


def test_one_workspace_per_stream_and_thread(cache):
    dev = torch.device("cuda", 0)

    def get(nbytes, stream):
        return w4.workspace(dev, nbytes, FakeStream(stream))
    a = get(1000, 1)
    assert get(500, 1) is a and get(1000, 2) is not a
    bigger = get(5000, 1)
    assert bigger is not a and bigger.numel() >= 5000 and get(1000, 1) is bigger
    assert not get(1000, 1).any()
    others, hold = [], threading.Barrier(3)

    def work():
        others.append(get(1000, 1))
        hold.wait(30)  # both threads live at once, so their identities differ
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    hold.wait(30)
    for t in threads:
        t.join(30)
    assert len({id(t) for t in (bigger, *others)}) == 3
