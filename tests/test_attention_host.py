"""Host side of attention and the gated feed-forward block (no GPU): refused
descriptions and calls, workspace sizes, and the binding's argument checks."""
import ctypes
import math

import pytest
import torch

import silent_corruption_detection_amd as sdc

OK, INVALID, DTYPE, ALIGN, WORKSPACE, RANGE = 0, -1, -2, -3, -4, -7
BIG = 1 << 40
P, U64, U32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32


def attn(**kw):
    step = U64 * 3
    h = sdc._Attn(0x1000, 0x2000, 0x3000, None, None, 2, 100, 200, 8, 2, 64, step(100 * 512, 512, 64),
                  step(200 * 128, 128, 64), step(200 * 128, 128, 64), 0, 0.125, 0, sdc.BF16, 0)
    for k, v in kw.items():
        setattr(h, k, step(*v) if k.endswith("stride") else v)
    return h


def ffn(**kw):
    b = sdc._Ffn(0x1000, 0x2000, 0x3000, 100, 64, 300, 64, 64, 64, sdc.BF16, 0)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def sizes(name, h):
    f, g = U64(0), U64(0)
    st = getattr(ctypes.CDLL(sdc.LIB_PATH), name)(ctypes.byref(h) if h is not None else None, ctypes.byref(f),
                                                  ctypes.byref(g))
    return st, f.value, g.value


BAD_ATTN = [
    (dict(dtype=sdc.F32), DTYPE), (dict(dtype=99), DTYPE), (dict(flags=1), INVALID), (dict(causal=2), INVALID),
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(d=0), INVALID), (dict(heads_q=0), INVALID),
    (dict(heads_k=0), INVALID), (dict(heads_k=3), INVALID), (dict(heads_q=1), INVALID), (dict(window=5), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=1e-30), INVALID), (dict(scale=1e30), INVALID), (dict(seq_q=0x4000), INVALID), (dict(seq_k=0x4000), INVALID),
    (dict(d=60), RANGE), (dict(d=136), RANGE), (dict(batch=1 << 24), RANGE), (dict(len_q=1 << 31), RANGE),
    (dict(len_k=1 << 30), RANGE), (dict(batch=1 << 20, len_q=1 << 20), RANGE), (dict(heads_q=1 << 20, heads_k=1), RANGE),
    (dict(batch=1 << 23, len_q=1, len_k=1), RANGE), (dict(q=0x1008), ALIGN), (dict(k=0x2002), ALIGN), (dict(v=0x3008), ALIGN),
    (dict(q_stride=(100 * 512 + 4, 512, 64)), ALIGN), (dict(k_stride=(200 * 128, 132, 64)), ALIGN),
    (dict(v_stride=(200 * 128, 128, 65)), ALIGN), (dict(q_stride=(1 << 40, 512, 64)), RANGE),
    (dict(k_stride=(200 * 128, 1 << 23, 64)), RANGE), (dict(v_stride=(200 * 128, 128, 1 << 40)), RANGE),
    (dict(seq_q=0x4002, seq_k=0x5000), ALIGN), (dict(seq_q=0x4000, seq_k=0x5001), ALIGN)]


@pytest.mark.parametrize("bad, status", BAD_ATTN)
def test_refused_attention(bad, status):
    assert sizes("sdc_attention_ws_bytes", attn(**bad))[0] == status


def test_attention_sizes():
    assert sizes("sdc_attention_ws_bytes", None)[0] == INVALID
    st, f, g = sizes("sdc_attention_ws_bytes", attn())
    assert st == OK and f >= 256 and g >= 2 * 4 * 2 * 100 * 8
    # strides of one entry, row or head mean nothing, neither do pointers to no rows
    assert sizes("sdc_attention_ws_bytes", attn(batch=1, q_stride=(3, 512, 64)))[0] == OK
    assert sizes("sdc_attention_ws_bytes", attn(len_q=1, q_stride=(512, 1 << 50, 64)))[0] == OK
    assert sizes("sdc_attention_ws_bytes", attn(heads_k=1, k_stride=(200 * 128, 128, 7)))[0] == OK
    assert sizes("sdc_attention_ws_bytes", attn(len_q=0, q=0))[0] == OK
    assert sizes("sdc_attention_ws_bytes", attn(len_k=0, k=0, v=0))[0] == OK
    assert sizes("sdc_attention_ws_bytes", attn(batch=0, q=0, k=0, v=0))[0] == OK
    # scores are in no workspace
    st, f, g = sizes("sdc_attention_ws_bytes", attn(len_q=65536, len_k=65536, causal=1))
    assert st == OK and max(f, g) < 64 << 20
    # one query of many keys: splits, whose sums are in fp32
    st, f, _ = sizes("sdc_attention_ws_bytes", attn(batch=1, len_q=1, len_k=1 << 20))
    assert st == OK and 4 * 8 * 64 * 8 < f < 64 << 20
    assert sizes("sdc_attention_ws_bytes", attn(seq_q=0x4000, seq_k=0x5000, batch=7))[0] == OK


def test_refused_attention_calls():
    lib = ctypes.CDLL(sdc.LIB_PATH)
    fwd, bwd = lib.sdc_attention, lib.sdc_attention_grad
    fwd.argtypes = [P, P, U64, P, P, P, P]
    bwd.argtypes = [P, P, P, P, P, U64, P, P, P, P, U32, P, P, P]
    h = attn()

    def f(h=ctypes.addressof(h), ws=0x10000, nbytes=BIG, out=0x4000, lse=0x5000, row=None):
        return fwd(h, ws, nbytes, out, lse, row, None)

    def g(h=ctypes.addressof(h), out=0x4000, lse=0x5000, dout=0x6000, ws=0x10000, nbytes=BIG, dq=0x7000, dk=0x8000,
          dv=0x9000, ref=None, mask=15, row=None, mis=None):
        return bwd(h, out, lse, dout, ws, nbytes, dq, dk, dv, ref, mask, row, mis, None)

    for k in ("h", "ws", "out", "lse"):
        assert f(**{k: None}) == INVALID, k
    assert f(nbytes=16) == WORKSPACE and g(nbytes=1000) == WORKSPACE
    for k, v in (("ws", 0x10008), ("row", 0x8008), ("out", 0x4008), ("lse", 0x5002)):
        assert f(**{k: v}) == ALIGN, k
    for k in ("h", "out", "lse", "dout", "ws", "dk", "dv"):
        assert g(**{k: None}) == INVALID, k
    assert g(dq=None, dk=None, dv=None) == INVALID
    for k, v in (("ws", 0x10008), ("out", 0x4008), ("lse", 0x5001), ("dout", 0x6002), ("dq", 0x7008), ("dk", 0x8004),
                 ("dv", 0x9008), ("row", 0x8008)):
        assert g(**{k: v}) == ALIGN, k
    assert g(ref=0x9000) == INVALID                              # a compare needs a row and a counter
    assert g(ref=0x9000, row=0x8000) == INVALID
    assert g(ref=0x9000, row=0x8000, mis=0x100, mask=0) == INVALID
    assert g(ref=0x9000, row=0x8000, mis=0x100, mask=16) == INVALID
    assert g(ref=0x9008, row=0x8000, mis=0x100) == ALIGN
    assert g(ref=0x9000, row=0x8000, mis=0x102) == ALIGN
    for bad, status in BAD_ATTN:
        b = attn(**bad)
        assert f(h=ctypes.addressof(b)) == status and g(h=ctypes.addressof(b)) == status, bad


BAD_FFN = [
    (dict(dtype=sdc.F32), DTYPE), (dict(dtype=99), DTYPE), (dict(act=2), INVALID), (dict(x=0), INVALID),
    (dict(w_gate=0), INVALID), (dict(w_up=0), INVALID), (dict(d=0), INVALID), (dict(f=0), INVALID),
    (dict(x_stride=63), INVALID), (dict(w_gate_stride=63), INVALID), (dict(w_up_stride=63), INVALID),
    (dict(x=0x1001), ALIGN), (dict(w_gate=0x2001), ALIGN), (dict(w_up=0x3001), ALIGN), (dict(n=1 << 24), RANGE),
    (dict(f=1 << 23), RANGE), (dict(d=1 << 20, x_stride=1 << 20, w_gate_stride=1 << 20, w_up_stride=1 << 20), RANGE),
    (dict(x_stride=1 << 40), RANGE), (dict(w_up_stride=1 << 40), RANGE), (dict(n=(1 << 24) - 1, f=(1 << 23) - 1), RANGE)]


@pytest.mark.parametrize("bad, status", BAD_FFN)
def test_refused_ffn(bad, status):
    assert sizes("sdc_gated_ffn_ws_bytes", ffn(**bad))[0] == status


def test_ffn_sizes():
    assert sizes("sdc_gated_ffn_ws_bytes", None)[0] == INVALID
    st, f, g = sizes("sdc_gated_ffn_ws_bytes", ffn())
    assert st == OK and f < 1 << 16 and g >= 4 * 100 * 300
    assert sizes("sdc_gated_ffn_ws_bytes", ffn(n=0, x=0))[0] == OK
    assert sizes("sdc_gated_ffn_ws_bytes", ffn(d=63, w_gate=0x2002))[0] == OK
    # the forward pass keeps neither projection
    st, f, g = sizes("sdc_gated_ffn_ws_bytes", ffn(n=32768, d=8192, f=28672, x_stride=8192, w_gate_stride=8192,
                                                   w_up_stride=8192))
    assert st == OK and f < 2 << 20 and g < 5 * 32768 * 28672


def test_refused_ffn_calls():
    lib = ctypes.CDLL(sdc.LIB_PATH)
    fwd, bwd = lib.sdc_gated_ffn, lib.sdc_gated_ffn_grad
    fwd.argtypes = [P, P, U64, P, P, P]
    bwd.argtypes = [P, P, U64, P, U64, P, P, P, P, U32, P, P, P]
    b0 = ffn()

    def f(b=ctypes.addressof(b0), ws=0x10000, nbytes=BIG, h=0x4000, row=None):
        return fwd(b, ws, nbytes, h, row, None)

    def g(b=ctypes.addressof(b0), dh=0x4000, stride=300, ws=0x10000, nbytes=BIG, dx=0x5000, dwg=0x6000, dwu=0x7000,
          ref=None, mask=15, row=None, mis=None):
        return bwd(b, dh, stride, ws, nbytes, dx, dwg, dwu, ref, mask, row, mis, None)

    for k in ("b", "ws", "h"):
        assert f(**{k: None}) == INVALID, k
    assert f(nbytes=16) == WORKSPACE and g(nbytes=1000) == WORKSPACE
    for k, v in (("ws", 0x10008), ("row", 0x8008), ("h", 0x4001)):
        assert f(**{k: v}) == ALIGN, k
    for k in ("b", "dh", "ws", "dwg", "dwu"):
        assert g(**{k: None}) == INVALID, k
    assert g(dx=None, dwg=None, dwu=None) == INVALID and g(stride=299) == INVALID and g(stride=1 << 40) == RANGE
    for k, v in (("ws", 0x10008), ("dh", 0x4001), ("dx", 0x5001), ("dwg", 0x6001), ("dwu", 0x7001), ("row", 0x8008)):
        assert g(**{k: v}) == ALIGN, k
    assert g(ref=0x9000) == INVALID
    assert g(ref=0x9000, row=0x8000) == INVALID
    assert g(ref=0x9000, row=0x8000, mis=0x100, mask=16) == INVALID
    assert g(ref=0x9008, row=0x8000, mis=0x100) == ALIGN
    for bad, status in BAD_FFN:
        b = ffn(**bad)
        assert f(b=ctypes.addressof(b)) == status and g(b=ctypes.addressof(b)) == status, bad


def test_binding_refuses_host_tensors_and_shapes():
    q = torch.zeros(2, 5, 4, 64).bfloat16()
    with pytest.raises(ValueError, match="not on a GPU"):
        sdc.sdc_attention(q, q, q)
    with pytest.raises(TypeError):
        sdc.sdc_attention(q.float(), q, q)
    with pytest.raises(ValueError, match="q must be"):
        sdc.sdc_attention(q[0, 0], q, q)
    with pytest.raises(ValueError, match="packed sequences need"):
        sdc.sdc_attention(q[0], q[0], q[0])
    with pytest.raises(ValueError, match="packed sequences need"):
        sdc.sdc_attention(q, q, q, seq_q=torch.zeros(3, dtype=torch.int32))
    x, w = torch.zeros(4, 8).bfloat16(), torch.zeros(16, 8).bfloat16()
    with pytest.raises(ValueError, match="not on a GPU"):
        sdc.sdc_gated_ffn(x, w, w)
    with pytest.raises(TypeError):
        sdc.sdc_gated_ffn(x.float(), w, w)
    with pytest.raises(ValueError, match="act must be"):
        sdc.sdc_gated_ffn(x, w, w, act="relu")
    with pytest.raises(ValueError, match="2-D"):
        sdc.sdc_gated_ffn(x[0], w, w)
