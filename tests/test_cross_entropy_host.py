"""Host side of the linear head's cross entropy (no GPU): refused heads and
calls, workspace sizes, and the binding's argument checks."""
import ctypes

import pytest
import torch

import silent_corruption_detection_amd as sdc

INVALID, DTYPE, ALIGN, WORKSPACE, RANGE = -1, -2, -3, -4, -7


def head(**kw):
    h = sdc._Head(0x1000, 0x2000, 0x3000, 100, 64, 1000, 64, 64, sdc.BF16, 0)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def sizes(h):
    lib = ctypes.CDLL(sdc.LIB_PATH)
    f, g = ctypes.c_uint64(0), ctypes.c_uint64(0)
    st = lib.sdc_cross_entropy_ws_bytes(ctypes.byref(h) if h is not None else None, ctypes.byref(f), ctypes.byref(g))
    return st, f.value, g.value


BAD = [
    (dict(dtype=sdc.F32), DTYPE), (dict(dtype=99), DTYPE), (dict(flags=1), INVALID),
    (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(target=0), INVALID), (dict(d=0), INVALID),
    (dict(vocab=0), INVALID), (dict(x_stride=63), INVALID), (dict(w_stride=63), INVALID),
    (dict(x=0x1001), ALIGN), (dict(w=0x2001), ALIGN), (dict(target=0x3004), ALIGN),
    (dict(n=1 << 24), RANGE), (dict(vocab=1 << 24), RANGE), (dict(d=1 << 20, x_stride=1 << 20, w_stride=1 << 20), RANGE),
    (dict(x_stride=1 << 40), RANGE), (dict(n=(1 << 24) - 1, vocab=(1 << 24) - 1), RANGE),
]


@pytest.mark.parametrize("bad, status", BAD)
def test_refused_heads(bad, status):
    assert sizes(head(**bad))[0] == status


def test_sizes():
    assert sizes(None)[0] == INVALID
    st, f, g = sizes(head())
    assert st == 0 and 100 * 4 * 8 <= f < 1 << 20 and g >= 4 * 100 * 64
    # the gradient's workspace holds a piece of the vocabulary, not the logits
    st, f, g = sizes(head(n=32768, d=8192, vocab=1 << 20, x_stride=8192, w_stride=8192))
    assert st == 0 and g < 4 * 32768 * (1 << 20) / 16
    # an empty batch and a head whose rows need a copy are fine
    assert sizes(head(n=0, x=0, target=0))[0] == 0
    assert sizes(head(d=63, w=0x2002))[0] == 0


def test_refused_calls():
    lib = ctypes.CDLL(sdc.LIB_PATH)
    P, U64 = ctypes.c_void_p, ctypes.c_uint64
    fwd, bwd = lib.sdc_cross_entropy, lib.sdc_cross_entropy_grad
    fwd.argtypes = [P, P, U64, P, P, P, P, P, P]
    bwd.argtypes = [P, P, P, P, U64, P, P, P, ctypes.c_uint32, P, P, P]
    h = head()
    hp, big = ctypes.addressof(h), 1 << 40

    def f(ws=0x10000, nbytes=big, loss=0x4000, lse=0x5000, total=0x6000, count=None, row=None):
        return fwd(hp, ws, nbytes, loss, lse, total, count, row, None)

    def g(lse=0x4000, grad=0x5000, ws=0x10000, nbytes=big, dx=0x6000, dw=0x7000, ref=None, mask=15, row=None, mis=None):
        return bwd(hp, lse, grad, ws, nbytes, dx, dw, ref, mask, row, mis, None)

    for k in ("ws", "loss", "lse", "total"):
        assert f(**{k: None}) == INVALID, k
    assert f(nbytes=16) == WORKSPACE
    for k, v in (("ws", 0x10008), ("row", 0x8008), ("loss", 0x4002), ("lse", 0x5002), ("total", 0x6001),
                 ("count", 0x8004)):
        assert f(**{k: v}) == ALIGN, k
    for k in ("lse", "grad", "ws"):
        assert g(**{k: None}) == INVALID, k
    assert g(dx=None, dw=None) == INVALID
    assert g(nbytes=1000) == WORKSPACE
    for k, v in (("ws", 0x10008), ("lse", 0x4002), ("grad", 0x5001), ("dx", 0x6001), ("dw", 0x7001),
                 ("row", 0x8008)):
        assert g(**{k: v}) == ALIGN, k
    assert g(ref=0x9000) == INVALID                              # a compare needs a row and a counter
    assert g(ref=0x9000, row=0x8000) == INVALID
    assert g(ref=0x9000, row=0x8000, mis=0x100, mask=0) == INVALID
    assert g(ref=0x9000, row=0x8000, mis=0x100, mask=16) == INVALID
    assert g(ref=0x9008, row=0x8000, mis=0x100) == ALIGN
    assert g(ref=0x9000, row=0x8000, mis=0x102) == ALIGN
    for bad, status in BAD:
        h2 = head(**bad)
        assert fwd(ctypes.addressof(h2), 0x10000, big, 0x4000, 0x5000, 0x6000, None, None, None) == status
        assert bwd(ctypes.addressof(h2), 0x4000, 0x5000, 0x10000, big, 0x6000, 0x7000, None, 15, None, None, None) == status


def test_binding_refuses_host_tensors():
    x, w, t = torch.zeros(4, 8).bfloat16(), torch.zeros(16, 8).bfloat16(), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="not on a GPU"):
        sdc.sdc_cross_entropy(x, w, t)
    with pytest.raises(TypeError):
        sdc.sdc_cross_entropy(x.float(), w, t)
    with pytest.raises(ValueError, match="2-D"):
        sdc.sdc_cross_entropy(x[0], w, t)
