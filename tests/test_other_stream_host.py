"""Who keeps the memory of a call on another stream than the current one (no GPU needed)."""
import torch

from delta_rule_sequence_b200 import prism as P


class _Tensor:
    def __init__(self):
        self.on = []

    def record_stream(self, stream):
        self.on.append(stream)


def test_inputs_wait_for_the_call_and_results_for_their_reader(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: "here")
    given, out, result = _Tensor(), _Tensor(), _Tensor()
    P._on_other_stream("there", None, (given, None, out), (result, out, None))
    assert given.on == ["there"] and result.on == ["here"] and out.on == ["there", "here"]
    for stream in (None, "here"):
        t = _Tensor()
        P._on_other_stream(stream, None, (t,), (t,))
        assert t.on == []
