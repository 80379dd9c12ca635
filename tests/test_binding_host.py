"""How the binding finds the current device and stream (no GPU needed)."""
import torch

import speculative_decoding_tree_attention_gb300 as tv


def test_a_torch_without_the_quick_ways_is_asked_the_public_way(monkeypatch):
    """The private accessors of torch._C are only a shorter way to the same numbers."""
    class Stream:
        cuda_stream = 17

    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    monkeypatch.setattr(tv, "_raw", None)
    monkeypatch.setattr(tv, "_current", None, raising=False)
    assert tv._run(3, None, lambda handle: handle) == 17
