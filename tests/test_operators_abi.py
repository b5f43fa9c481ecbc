"""Refusals of the norm, rotation and chunk entry points on the host: every bad
argument is turned into its status before anything is launched (the addresses
are never read), and the binding's own checks raise."""
import ctypes

import pytest
import torch

from parameterized_local_linear_b200 import binding as pl
from parameterized_local_linear_b200 import build

OK, ENULL, ESHAPE, EHEAD, EDTYPE, EALIGN, EWS = 0, -1, -2, -3, -4, -5, -6
i, p, f, d, ll, z = (ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_double,
                     ctypes.c_longlong, ctypes.c_size_t)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pl.load_library()


def caller(lib, name, fields):
    """fields: (argument, type, default) in order -> a call with overrides."""
    fn = getattr(lib, name)
    proto = ctypes.CFUNCTYPE(i, *[t for _, t, _ in fields])(ctypes.cast(fn, p).value)

    def call(**kw):
        vals = {n: v for n, _, v in fields}
        assert set(kw) <= set(vals), set(kw) - set(vals)
        vals.update(kw)
        return proto(*[vals[n] for n, _, _ in fields])

    return call


HEAD = [("tokens", i, 8), ("Hq", i, 4), ("Hkv", i, 2), ("D", i, 64), ("rot", i, 64), ("inter", i, 0),
        ("maxpos", i, 100), ("eps", f, 1e-6)]
TAIL = [("dtype", i, 0), ("stream", p, None), ("ws", p, 16), ("wsb", z, 100)]
PTRS = lambda *names: [(n, p, 16) for n in names]


def test_forward_refusals(lib):
    call = caller(lib, "parallax_qk_norm_rope",
                  PTRS("q", "r", "k", "qw", "rw", "kw", "cs", "pos", "qo", "ro", "ko") + HEAD +
                  [("sq", ll, 256), ("sr", ll, 256), ("sk", ll, 128), ("L", i, 0)] + TAIL)
    assert call() == EWS
    kw = dict(wsb=256)
    for name in ("q", "k", "cs", "qo", "ro", "ko", "ws"):
        assert call(**{name: None, **kw}) == ENULL, name
    for name in ("q", "r", "k", "qw", "rw", "kw", "cs", "qo", "ro", "ko", "ws"):
        assert call(**{name: 24, **kw}) == EALIGN, name
    assert call(pos=18, **kw) == EALIGN
    for bad in (dict(tokens=0), dict(Hq=3), dict(Hq=0), dict(Hkv=0), dict(rot=0), dict(rot=24),
                dict(rot=80), dict(maxpos=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(sq=255), dict(sq=252), dict(sq=258), dict(sk=127),
                dict(sr=128), dict(L=-1), dict(L=3)):
        assert call(**bad, **kw) == ESHAPE, bad
    assert call(D=96, **kw) == EHEAD
    assert call(dtype=2, **kw) == EDTYPE
    assert call(sq=260, dtype=1, wsb=100) == EWS  # fp32: 16 bytes are four elements


def test_backward_refusals(lib):
    call = caller(lib, "parallax_qk_norm_rope_backward",
                  PTRS("gq", "gr", "gk", "q", "r", "k", "qw", "rw", "kw", "cs", "pos", "dq", "dr",
                       "dk", "dqw", "drw", "dkw") + HEAD +
                  [("sq", ll, 256), ("sr", ll, 256), ("sk", ll, 128), ("tq", ll, 256),
                   ("tr", ll, 256), ("tk", ll, 128), ("L", i, 0)] + TAIL)
    assert call() == EWS
    kw = dict(wsb=256)  # refused before the device is asked for the full size
    for name in ("gq", "gr", "gk", "q", "k", "cs", "dq", "dr", "dk", "dqw", "drw", "dkw", "ws"):
        assert call(**{name: None, **kw}) == ENULL, name
    for name in ("gq", "gr", "gk", "q", "r", "k", "qw", "rw", "kw", "cs", "dq", "dr", "dk", "ws"):
        assert call(**{name: 24, **kw}) == EALIGN, name
    assert call(dqw=18, **kw) == EALIGN
    for bad in (dict(tokens=0), dict(rot=8), dict(eps=0.0), dict(tq=255), dict(tk=132), dict(L=5)):
        assert call(**bad, **kw) == ESHAPE, bad
    assert call(D=32, **kw) == EHEAD
    f = lib.parallax_qk_norm_rope_backward_workspace_bytes
    f.restype = z
    for bad in ((0, 4, 2, 64), (8, 3, 2, 64), (8, 4, 2, 96)):
        assert f(*bad) == 0


def test_append_refusals(lib):
    call = caller(lib, "parallax_norm_rope_append",
                  PTRS("q", "r", "k", "v", "qw", "rw", "kw", "cs", "pos", "cu", "lens", "table",
                       "qo", "ro", "kp", "vp") + [("B", i, 2)] + HEAD +
                  [("sq", ll, 256), ("sr", ll, 256), ("sk", ll, 128), ("sv", ll, 128),
                   ("pages", i, 4), ("ps", i, 16), ("maxp", i, 2)] + TAIL)
    assert call() == EWS
    kw = dict(wsb=256)
    for name in ("q", "k", "v", "cs", "lens", "table", "qo", "ro", "kp", "vp", "ws"):
        assert call(**{name: None, **kw}) == ENULL, name
    for name in ("q", "r", "k", "v", "qw", "qo", "ro", "kp", "vp"):
        assert call(**{name: 24, **kw}) == EALIGN, name
    for name in ("cu", "lens", "table", "pos"):
        assert call(**{name: 18, **kw}) == EALIGN, name
    for bad in (dict(B=0), dict(cu=None), dict(pages=0), dict(ps=0), dict(maxp=0), dict(sv=64),
                dict(ps=1 << 20, maxp=1 << 12)):
        assert call(**bad, **kw) == ESHAPE, bad


def test_chunk_refusals(lib):
    call = caller(lib, "parallax_prefill_paged",
                  PTRS("q", "r", "kp", "vp", "table", "cu", "lens", "out") +
                  [("B", i, 2), ("total", i, 8), ("Hq", i, 4), ("Hkv", i, 2), ("D", i, 64),
                   ("scale", f, 0.1), ("causal", i, 1), ("stream", p, None), ("pages", i, 4),
                   ("ps", i, 64), ("maxp", i, 2), ("probe", i, 1), ("ws", p, 16), ("wsb", z, 100)])
    for name in ("q", "r", "kp", "vp", "table", "lens", "out", "ws"):
        assert call(**{name: None}) == ENULL, name
    for name in ("q", "r", "kp", "vp", "out", "ws"):
        assert call(**{name: 24}) == EALIGN, name
    for name in ("table", "cu", "lens"):
        assert call(**{name: 18}) == EALIGN, name
    for bad in (dict(B=0), dict(total=0), dict(Hq=3), dict(Hq=258), dict(pages=0), dict(ps=32),
                dict(ps=96), dict(maxp=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(cu=None), dict(ps=1 << 20, maxp=1 << 12)):
        assert call(**bad) == ESHAPE, bad
    assert call(D=96) == EHEAD
    f2 = lib.parallax_prefill_paged_workspace_bytes
    f2.restype = z
    for bad in ((0, 8, 4, 2, 64), (2, 0, 4, 2, 64), (2, 8, 3, 2, 64), (2, 8, 258, 2, 64),
                (2, 8, 4, 2, 96)):
        assert f2(*bad) == 0


def test_table_refusals(lib):
    call = caller(lib, "parallax_rope_table",
                  [("cs", p, 16), ("n", i, 10), ("rot", i, 64), ("base", d, 1e4), ("s", p, None)])
    assert call(cs=None) == ENULL and call(cs=24) == EALIGN
    for bad in (dict(n=0), dict(rot=8), dict(rot=40), dict(rot=144), dict(base=0.0),
                dict(base=float("inf")), dict(base=float("nan"))):
        assert call(**bad) == ESHAPE, bad


def test_status_string(lib):
    assert "position" in pl.parallax_status_string(-13)


def test_binding_needs_cuda_tensors():
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        pl.parallax_qk_norm_rope(x, None, x, x)
    with pytest.raises(ValueError):
        pl.parallax_prefill_paged(x, None, x, x, x, x)


def test_stream_of_another_device_is_refused():
    class Fake:
        def __init__(self, device):
            self.device, self.cuda_stream = torch.device(device), 0

    with pytest.raises(ValueError):
        pl._call("prefill_paged", (Fake("cuda:0"),), Fake("cuda:1"))
    with pytest.raises(ValueError):
        pl.parallax_rope_table(16, 64, device="cuda:0", stream=Fake("cuda:1"))
    s = Fake("cuda:1")
    assert pl._stream_on(torch.device("cuda:1"), s) is s


def test_workspace_status_refuses_what_is_no_workspace():
    for bad in (torch.zeros(256, dtype=torch.uint8), torch.zeros(256)):
        with pytest.raises(ValueError):
            pl.parallax_workspace_status(bad)


def test_stall_hook_bounds_its_timeout(lib):
    fn = lib.parallax_testing_norm_rope_stall_next
    assert [fn(t) for t in (0, -1, 10001)] == [ESHAPE] * 3
