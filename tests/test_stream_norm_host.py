"""The chunk stream's output norm on CPU: what it is given, and that it leaves the state alone."""
import pytest
import torch

from delta_rule_sequence_b200.stream import StreamingScan


def _stream(norm_fn):
    element = lambda q, k, v, a, b, u, w, chunk: (torch.ones(1), q.sum())  # noqa: E731
    scan = lambda q, k, v, a, b, u, w, S0, chunk: (q + (0 if S0 is None else S0), None)  # noqa: E731
    return StreamingScan(None, element_fn=element, compose_fn=lambda a, b: (a[0], a[1] + b[1]),
                         fold_fn=lambda S, E, f: f if S is None else S + f, scan_fn=scan, norm_fn=norm_fn)


def test_norm_sees_each_chunk_and_its_gate():
    seen = []

    def norm(o, gate):
        seen.append((o.clone(), gate))
        return -o

    s, plain = _stream(norm), _stream(None)
    for i in range(3):
        q = torch.full((1, 4, 1, 2), float(i + 1))
        gate = None if i == 1 else q * 10
        y, o = s.step(q, None, None, None, None, gate=gate), plain.step(q, None, None, None, None)
        assert torch.equal(y, -o) and torch.equal(seen[i][0], o) and seen[i][1] is gate
    assert torch.equal(s.state(), plain.state())


def test_a_gate_without_a_norm_is_refused():
    with pytest.raises(ValueError):
        _stream(None).step(torch.zeros(1, 4, 1, 2), None, None, None, None, gate=torch.zeros(1, 4, 1, 2))


def test_a_chunk_whose_norm_fails_is_not_in_the_stream():
    """The caller corrects the gate and gives the chunk again: it counts once."""
    def norm(o, gate):
        if gate.shape != o.shape:
            raise ValueError("gate")
        return o * gate

    s, plain = _stream(norm), _stream(None)
    q = torch.full((1, 4, 1, 2), 3.0)
    for i in range(3):
        with pytest.raises(ValueError):
            s.step(q, None, None, None, None, gate=q[:, :2])
        y, o = s.step(q, None, None, None, None, gate=2 * torch.ones_like(q)), plain.step(q, None, None, None, None)
        assert torch.equal(y, 2 * o) and s.counter.count == i + 1
    assert torch.equal(s.state(), plain.state())
