"""Results that go back to the host are waited for on their own device, which need not be the current one (weights on
cuda:1 bring the call there).  Played with stand-ins, without a GPU."""
import torch

import kimi_delta_attention_gated_gb300 as kda


class Result:
    """A device tensor, as far as the copy back looks at it."""

    def __init__(self, device):
        self.device, self.is_cuda = torch.device(device), True

    def to(self, where):
        return ("copy", self.device)


class Pinned:
    def __init__(self):
        self.copied = None

    def is_pinned(self):
        return True

    def copy_(self, t, non_blocking):
        self.copied = (t, non_blocking)


def test_each_results_device_is_waited_for(monkeypatch):
    waited = []

    class Stream:
        def __init__(self, device):
            self.device = device

        def synchronize(self):
            waited.append(self.device)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(device))
    a, b, dest = Result("cuda:1"), Result("cuda:0"), Pinned()
    out = kda._to_host((a, None, b), True, (dest, None, None))
    assert out == (dest, None, ("copy", b.device)) and dest.copied == (a, True)
    assert sorted(waited, key=str) == [torch.device("cuda:0"), torch.device("cuda:1")]
    waited.clear()
    kda._to_host((a,), True, (dest,))
    assert waited == [torch.device("cuda:1")]
    assert kda._to_host((a, b), False) == (a, b) and len(waited) == 1
