"""Calls of the decay scan and the group norm on another stream than the current one, given temporaries."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _decay():
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, dtype=BF: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    B, T, H, d = 2, 300, 4, 64
    q, k, v, dO = (r(B, T, H, d) for _ in range(4))
    S0, dS = (r(B, H, d, d, dtype=torch.float32) for _ in range(2))
    a = torch.tensor([0.5, 0.9, 0.99, 1.0], device="cuda")
    return q, k, v, a, S0, torch.tensor([300, 77], dtype=torch.int32, device="cuda"), dO, dS


def _norm():
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s, dtype=BF: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, gate, dy = (r(3, 200, 96) for _ in range(3))
    w, b = (r(96, dtype=torch.float32) for _ in range(2))
    return x, w, b, gate, dy, r(3, 8, dtype=torch.float32), r(3, 8, dtype=torch.float32).abs()


def _calls():
    from delta_rule_sequence_b200 import prism as P

    def step(t, s):
        S = t[4]
        return [P.prism_decay_step(t[0][:, :1], t[1][:, :1], t[2][:, :1], t[3], S, stream=s)]

    return {
        "scan": (_decay, lambda t, s: list(P.prism_decay_scan_fwd(*t[:6], stream=s))),
        "grad": (_decay, lambda t, s: list(P.prism_decay_scan_bwd(*t[:6], dO=t[6], dS_final=t[7], stream=s).values())),
        "step": (_decay, step),
        "norm": (_norm, lambda t, s: list(P.prism_group_norm_fwd(t[0], 8, *t[1:4], activation="silu", stream=s))),
        "norm grad": (_norm, lambda t, s: list(P.prism_group_norm_bwd(t[0], 8, t[5], t[6], *t[1:4], dy=t[4], activation="silu",
                                                                      stream=s).values())),
    }


@pytest.mark.parametrize("name", ["scan", "grad", "step", "norm", "norm grad"])
def test_temporaries_keep_their_memory_until_the_other_stream_is_through(name):
    make, call = _calls()[name]
    want = call(make(), None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    given = make()
    used = {"scan": 6, "grad": 8, "step": 5, "norm": 4, "norm grad": 7}[name]
    shapes = [(t.shape, t.dtype, t.data_ptr()) for t in given[:used]]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # a tenth of a second of work before the call's
    out = call(given, s)
    busy = not s.query()
    del given
    later = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype, _ in shapes]
    taken = {t.data_ptr() for t in later} & {p for _, _, p in shapes}
    assert busy, "the stream was through before the temporaries were gone"
    assert not taken
    for t in later:
        t.fill_(-1 if t.dtype == torch.int32 else float("nan"))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
