"""Host-only checks of the decay scan's and the group norm's entry points: bad calls are refused before
anything is launched (no GPU needed; the pointers are never followed)."""
import ctypes

import pytest
import torch

from delta_rule_sequence_b200 import prism as P

OK, INVALID, UNSUPPORTED = P.PRISM_OK, P.PRISM_ERR_INVALID_ARG, P.PRISM_ERR_UNSUPPORTED
MB = 1 << 20


def ptr(i, off=0):
    """The i-th buffer: 16 MB apart, so that no two overlap."""
    return ctypes.c_void_p(0x10000000 + 16 * MB * i + off)


@pytest.fixture(scope="module")
def lib():
    from delta_rule_sequence_b200 import build

    build.build()
    return P.load_library()


def shape(q=(0, 0, 0), k=(0, 0, 0), v=(0, 0, 0), **kw):
    d = dict(B=2, H=4, T=100, Hkv=2, dk=64, dv=32, io=P.PRISM_BF16)
    d.update(kw)
    mk = lambda s: (ctypes.c_longlong * 3)(*s)  # noqa: E731
    return P.PrismDecayShape(*[d[n] for n in ("B", "H", "T", "Hkv", "dk", "dv", "io")], mk(q), mk(k), mk(v))


def fwd(lib, s, ws_bytes=None, **kw):
    need = ctypes.c_size_t(0)
    lib.prism_decay_scan_fwd_workspace_size(ctypes.byref(s), ctypes.byref(need))
    a = dict(q=ptr(1), k=ptr(2), v=ptr(3), decay=ptr(4), S0=ptr(5), lengths=ptr(6), o=ptr(7), S_final=ptr(8), ws=ptr(20))
    a.update(kw)
    return lib.prism_decay_scan_fwd(ctypes.byref(s), *a.values(), need.value if ws_bytes is None else ws_bytes, None)


def bwd(lib, s, **kw):
    need = ctypes.c_size_t(0)
    lib.prism_decay_scan_bwd_workspace_size(ctypes.byref(s), ctypes.byref(need))
    a = dict(q=ptr(1), k=ptr(2), v=ptr(3), decay=ptr(4), S0=ptr(5), lengths=ptr(6), dO=ptr(7), dS=ptr(8), dq=ptr(9),
             dk=ptr(10), dv=ptr(11), dS0=ptr(12), ws=ptr(20))
    a.update(kw)
    return lib.prism_decay_scan_bwd(ctypes.byref(s), *a.values(), need.value, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dk=48), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(dk=0), INVALID), (dict(T=-1), INVALID),
    (dict(B=-1), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID), (dict(io=2), INVALID),
    (dict(T=(1 << 26) + 1), UNSUPPORTED), (dict(q=(1 << 36, 256, 64)), INVALID), (dict(B=70000), UNSUPPORTED), (dict(H=65536, Hkv=1), UNSUPPORTED), (dict(B=60000, H=400), UNSUPPORTED),
    (dict(q=(25600, 256, 60)), INVALID),    # a head stride that is no multiple of 16 bytes
    (dict(k=(12800, 0, 64)), INVALID),      # every token the same key
    (dict(v=(-6400, 64, 32)), INVALID),
])
def test_decay_scan_refuses_shapes(lib, kw, want):
    s = shape(**kw)
    assert fwd(lib, s, ws_bytes=1 << 40) == want
    assert bwd(lib, s) == want
    if not {"T", "k", "q"} & set(kw):  # (a token stride of zero is fine where there is one token)
        assert lib.prism_decay_step(ctypes.byref(shape(T=1, **kw)), *[ptr(i) for i in range(6)], None) == want


def test_decay_scan_refuses_pointers(lib):
    s = shape()
    for name in ("q", "k", "v", "decay", "o", "ws"):
        assert fwd(lib, s, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "S0", "o", "S_final", "ws"):
        assert fwd(lib, s, **{name: ptr(9, 8)}) == INVALID, name
    for name in ("decay", "lengths"):
        assert fwd(lib, s, **{name: ptr(9, 2)}) == INVALID, name
    assert fwd(lib, s, ws_bytes=16) == INVALID
    for name in ("q", "k", "v", "decay", "dO", "dq", "dk", "dv", "ws"):
        assert bwd(lib, s, **{name: None}) == INVALID, name
    for name in ("S0", "dO", "dS", "dq", "dk", "dv", "dS0"):
        assert bwd(lib, s, **{name: ptr(13, 8)}) == INVALID, name
    assert lib.prism_decay_scan_fwd(None, *[None] * 9, 0, None) == INVALID
    assert lib.prism_decay_scan_fwd_workspace_size(ctypes.byref(s), None) == INVALID


def test_decay_scan_refuses_overlap(lib):
    s = shape()
    # q is 2 * 100 * 4 * 64 bf16 = 102400 bytes: an output that begins inside it, or in another output
    assert fwd(lib, s, o=ptr(1, 102400 - 16)) == INVALID
    assert fwd(lib, s, S_final=ptr(7, 16)) == INVALID
    assert fwd(lib, s, S_final=ptr(5, 16)) == INVALID  # partly S0 (S_final == S0 itself is allowed)
    assert fwd(lib, s, S0=ptr(7)) == INVALID
    assert fwd(lib, s, ws=ptr(7, 256)) == INVALID
    assert bwd(lib, s, dq=ptr(1)) == INVALID
    assert bwd(lib, s, dv=ptr(10, 32)) == INVALID
    assert bwd(lib, s, dS0=ptr(8)) == INVALID
    assert fwd(lib, shape(T=0), S_final=ptr(5, 16)) == INVALID  # without tokens, too
    # a view's extent counts, not its dense size: batch stride 1 MB
    wide = shape(q=(MB // 2, 256, 64))
    assert fwd(lib, wide, o=ptr(1, MB + 1024)) == INVALID


def test_decay_step_refuses(lib):
    def step(s, **kw):
        a = dict(q=ptr(1), k=ptr(2), v=ptr(3), decay=ptr(4), S=ptr(5), o=ptr(6))
        a.update(kw)
        return lib.prism_decay_step(ctypes.byref(s), *a.values(), None)

    one = shape(T=1)
    assert step(shape(T=2)) == INVALID
    assert step(shape(T=0)) == INVALID
    for name in ("q", "k", "v", "decay", "S", "o"):
        assert step(one, **{name: None}) == INVALID, name
        assert step(one, **{name: ptr(9, 2)}) == INVALID, name
    assert step(one, o=ptr(5, 16)) == INVALID
    assert step(one, S=ptr(1)) == INVALID
    assert step(shape(T=1, B=0), S=None, o=None) == OK


def test_decay_empty_calls_do_nothing(lib):
    assert fwd(lib, shape(B=0), q=None, k=None, v=None, o=None, S_final=None) == OK
    assert fwd(lib, shape(T=0), q=None, k=None, v=None, o=None, S_final=None) == OK
    assert bwd(lib, shape(T=0), q=None, k=None, v=None, dO=None, dq=None, dk=None, dv=None, dS0=None) == OK


def nshape(**kw):
    d = dict(N=4, S=6, C=32, G=4, io=P.PRISM_BF16, act=1, eps=1e-5)
    d.update(kw)
    return P.PrismNormShape(*d.values())


def nfwd(lib, s, ws_bytes=1 << 30, **kw):
    a = dict(x=ptr(1), w=ptr(2), b=ptr(3), gate=ptr(4), y=ptr(5), mean=ptr(6), rstd=ptr(7), ws=ptr(20))
    a.update(kw)
    return lib.prism_group_norm_fwd(ctypes.byref(s), *a.values(), ws_bytes, None)


def nbwd(lib, s, ws_bytes=1 << 30, **kw):
    a = dict(x=ptr(1), w=ptr(2), b=ptr(3), gate=ptr(4), mean=ptr(5), rstd=ptr(6), dy=ptr(7), dx=ptr(8), dgate=ptr(9),
             dw=ptr(10), db=ptr(11), ws=ptr(20))
    a.update(kw)
    return lib.prism_group_norm_bwd(ctypes.byref(s), *a.values(), ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(G=5), INVALID), (dict(G=0), INVALID), (dict(C=0), INVALID), (dict(N=-1), INVALID), (dict(S=-1), INVALID),
    (dict(io=3), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(C=1 << 21), UNSUPPORTED), (dict(N=1 << 25), UNSUPPORTED),
    (dict(S=(1 << 30) + 1), UNSUPPORTED), (dict(N=1 << 24, S=1 << 30, C=1 << 20, G=1), UNSUPPORTED),
])
def test_group_norm_refuses_shapes(lib, kw, want):
    assert nfwd(lib, nshape(**kw)) == want
    assert nbwd(lib, nshape(**kw)) == want
    assert lib.prism_group_norm_fwd_workspace_size(ctypes.byref(nshape(**kw)), ctypes.byref(ctypes.c_size_t())) == want


def test_group_norm_refuses_pointers_and_overlap(lib):
    s = nshape()
    for name in ("x", "y", "ws"):
        assert nfwd(lib, s, **{name: None}) == INVALID, name
    for name in ("x", "y", "gate", "ws"):
        assert nfwd(lib, s, **{name: ptr(9, 8)}) == INVALID, name
    assert nfwd(lib, s, y=ptr(1)) == INVALID          # in place
    assert nfwd(lib, s, mean=ptr(7, 4)) == INVALID
    assert nfwd(lib, s, ws_bytes=16) == INVALID
    for name in ("x", "mean", "rstd", "dy", "dx", "dgate", "gate", "ws"):
        assert nbwd(lib, s, **{name: None}) == INVALID, name
    assert nbwd(lib, s, dx=ptr(7)) == INVALID
    assert nbwd(lib, s, dw=ptr(11)) == INVALID
    assert nbwd(lib, s, ws_bytes=16) == INVALID
    assert nfwd(lib, nshape(N=0), x=None, y=None) == OK


def test_wrappers_refuse_cpu_tensors():
    q = torch.zeros(1, 2, 2, 32)
    a = torch.ones(2)
    with pytest.raises(TypeError):
        P.prism_decay_scan_fwd(q, q, q, a)
    with pytest.raises(TypeError):
        P.prism_decay_step(q[:, :1], q[:, :1], q[:, :1], a, torch.zeros(1, 2, 32, 32))
    with pytest.raises(TypeError):
        P.prism_decay_scan_bwd(q, q, q, a, dO=q)
    with pytest.raises(TypeError):
        P.prism_group_norm_fwd(q, 2)
    with pytest.raises(TypeError):
        P.prism_group_norm_bwd(q, 2, a, a, dy=q)


def test_wrappers_refuse_sizes_beyond_c_ints():
    """2^32 + 1 would arrive in the library as 1."""
    with pytest.raises(ValueError):
        P._norm_shape(((1 << 32) + 1, 1, 8, 2, P.PRISM_BF16, 0, 1e-5))
    with pytest.raises(ValueError):
        P._decay_shape((1, 1, (1 << 32) + 1, 1, 32, 32, P.PRISM_BF16), P._DENSE, P._DENSE, P._DENSE)
