"""Host side of the AdamW step (no GPU): every refused list and call, the
plan's size, and the binding's argument checks."""
import ctypes

import pytest
import torch

import silent_corruption_detection_amd as sdc

INVALID, DTYPE, ALIGN, WORKSPACE, PLAN, RANGE = -1, -2, -3, -4, -6, -7


class T(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_sq", "master",
                                               "exp_avg_scale", "exp_avg_sq_scale")] + [
        ("numel", ctypes.c_uint64)] + [(n, ctypes.c_uint32) for n in
                                       ("param_dtype", "grad_dtype", "state_dtype", "group")]


def tensor(**kw):
    t = T(param=0x1000, grad=0x2000, exp_avg=0x3000, exp_avg_sq=0x4000, numel=1000,
          param_dtype=sdc.BF16, grad_dtype=sdc.BF16, state_dtype=sdc.F32, group=0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def nbytes(ts, n_groups=1, n=None):
    lib = ctypes.CDLL(sdc.LIB_PATH)
    f = lib.sdc_adamw_plan_bytes
    f.argtypes = [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_void_p]
    arr = (T * max(len(ts), 1))(*ts)
    out = ctypes.c_uint64(0)
    return f(arr, len(ts) if n is None else n, n_groups, ctypes.byref(out)), out.value


def test_plan_bytes_grow_with_the_list():
    assert nbytes([])[0] == 0
    st, one = nbytes([tensor()])
    st2, two = nbytes([tensor(), tensor(numel=10_000_000)])
    assert st == st2 == 0 and one > 0
    assert two >= one + 80 + (10_000_000 // 65536) * (32 + 32)
    assert nbytes([tensor(numel=0, param=0, exp_avg=0, exp_avg_sq=0)])[0] == 0
    assert nbytes([tensor(grad=0)])[0] == 0
    assert nbytes([tensor(master=0x5000)])[0] == 0
    assert nbytes([tensor(group=6)], n_groups=7)[0] == 0
    assert nbytes([tensor(state_dtype=sdc.FP8_E4M3, exp_avg=0x3001, exp_avg_sq=0x4003,
                          exp_avg_scale=0x5001, exp_avg_sq_scale=0x6001)])[0] == 0


@pytest.mark.parametrize("bad, status", [
    (dict(param=0), INVALID), (dict(exp_avg=0), INVALID), (dict(exp_avg_sq=0), INVALID),
    (dict(group=1), INVALID),
    (dict(param_dtype=sdc.F64), DTYPE), (dict(grad_dtype=sdc.U16), DTYPE),
    (dict(state_dtype=sdc.BF16), DTYPE), (dict(state_dtype=sdc.FP8_E5M2), DTYPE),
    (dict(state_dtype=sdc.FP8_E4M3), INVALID),                         # no scale bytes
    (dict(state_dtype=sdc.FP8_E4M3, exp_avg_scale=0x5000), INVALID),   # only one of the two
    (dict(exp_avg_scale=0x5000), INVALID),                             # scale bytes of an fp32 state
    (dict(param_dtype=sdc.F32, master=0x5000), INVALID),
    (dict(param=0x1001), ALIGN), (dict(grad=0x2001), ALIGN), (dict(exp_avg=0x3002), ALIGN),
    (dict(exp_avg_sq=0x4002), ALIGN), (dict(master=0x5002), ALIGN),
    (dict(grad_dtype=sdc.F32, grad=0x2002), ALIGN),
    (dict(numel=1 << 48), RANGE),
])
def test_refused_tensors(bad, status):
    assert nbytes([tensor(), tensor(**bad)])[0] == status


def test_refused_lists():
    assert nbytes([tensor()], n_groups=0)[0] == INVALID
    assert nbytes([tensor()], n_groups=65537)[0] == INVALID
    assert nbytes([tensor(numel=(1 << 48) - 1)] * 2)[0] == RANGE
    assert nbytes([tensor()], n=1 << 25)[0] == RANGE     # before any entry is read
    lib = ctypes.CDLL(sdc.LIB_PATH)
    assert lib.sdc_adamw_plan_bytes(None, ctypes.c_uint64(1), 1, ctypes.byref(ctypes.c_uint64())) == INVALID
    assert lib.sdc_adamw_plan_bytes(None, ctypes.c_uint64(0), 1, None) == INVALID


def test_refused_calls():
    """The step's own checks come before anything is queued, so they need no GPU."""
    lib = ctypes.CDLL(sdc.LIB_PATH)
    f = lib.sdc_adamw_step
    f.argtypes = [ctypes.c_void_p] * 6 + [ctypes.c_double] * 2 + [ctypes.c_void_p] * 2
    info = sdc._AdamwInfo()
    info.magic, info.n_groups = 0x31766D6164414453, 1
    info.plan_bytes = 1 << 20
    ok = [0x1000, ctypes.addressof(info), 0x2000, 0x3000, 0x4000, 0x5000]

    def call(at=None, value=None, max_norm=0.0, scale=1.0, rows=None):
        args = list(ok)
        if at is not None:
            args[at] = value
        return f(*args, max_norm, scale, rows, None)

    for at in (0, 1, 2, 3):
        assert call(at, None) == INVALID
    assert call(4, None, max_norm=1.0) == INVALID
    for bad in (-1.0, float("nan"), float("inf")):
        assert call(max_norm=bad) == INVALID
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=bad) == INVALID
    for at in (2, 3, 4):
        assert call(at, 0x2004) == ALIGN
    assert call(5, 0x5002) == ALIGN
    assert call(rows=0x6008) == ALIGN
    for field, value in (("magic", 0), ("n_groups", 0), ("n_items", 5), ("n_split", 1), ("n_slots", 1),
                         ("plan_bytes", 8)):
        before = getattr(info, field)
        setattr(info, field, value)
        assert call() == PLAN, field
        setattr(info, field, before)


def test_binding_refuses_host_tensors_and_bad_lists():
    p = torch.zeros(8)
    with pytest.raises(ValueError, match="not on a GPU"):
        sdc.sdc_adamw_plan_build([p], [p], [p], [p])
    with pytest.raises(ValueError, match="empty"):
        sdc.sdc_adamw_plan_build([], [], [], [])
    with pytest.raises(ValueError):
        sdc.sdc_adamw_control("cpu", step=-1)
    assert sdc.sdc_adamw_control("cpu", step=3, seed=9).tolist() == [3, 0, 9, 0]
