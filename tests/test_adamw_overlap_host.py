"""Lists whose memory overlaps (no GPU): the plan refuses what a step would write
while it reads or writes it as another tensor's.

The library compares spans of addresses only, so made-up ones do.  A plan buffer
of no bytes gives SDC_ERR_WORKSPACE where the list is right, before anything is
queued."""
import ctypes

import numpy as np
import pytest

import silent_corruption_detection_amd as sdc

INVALID, WORKSPACE = -1, -4
COLUMNS = ("param", "grad", "exp_avg", "exp_avg_sq", "master", "exp_avg_scale", "exp_avg_sq_scale")


def tensor(base, numel=1000, dtype=sdc.BF16, state=sdc.F32, **kw):
    """A tensor whose streams lie 64 KiB apart from `base` on."""
    t = np.zeros(1, dtype=sdc._ADAMW_DESC)
    for k, name in enumerate(COLUMNS):
        t[name] = base + k * 0x10000
    if state == sdc.F32:
        t["exp_avg_scale"] = t["exp_avg_sq_scale"] = 0
    t["numel"], t["param_dtype"], t["grad_dtype"], t["state_dtype"] = numel, dtype, sdc.BF16, state
    for name, v in kw.items():
        t[name] = v
    return t


def build(*tensors):
    table = np.concatenate(tensors)
    f = sdc._lib.sdc_adamw_plan_build
    info = sdc._AdamwInfo()
    got = f(ctypes.c_void_p(table.ctypes.data), len(table), 1, 0x10000, 0, ctypes.byref(info), None)
    clear = sdc._adamw_overlap(table) is None
    assert (got == WORKSPACE) == clear and (got == INVALID) == (not clear)
    return clear


A, B = 0x1000000, 0x2000000


def test_apart():
    assert build(tensor(A))
    assert build(tensor(A), tensor(B), tensor(A + 0x100000, state=sdc.FP8_E4M3))
    # back to back, in any order: 2000 bytes of bf16, 4000 of fp32, 8 scale bytes
    assert build(tensor(A, param=0x7000 + 2000), tensor(B, param=0x7000))
    assert build(tensor(A, exp_avg=0x8000), tensor(B, exp_avg=0x8000 + 4000), tensor(B + 0x100000, exp_avg=0x8000 - 4000))
    assert build(tensor(A, state=sdc.FP8_E4M3, exp_avg_scale=0x7001), tensor(B, state=sdc.FP8_E4M3, exp_avg_scale=0x7009))


@pytest.mark.parametrize("name, state", [(c, sdc.FP8_E4M3) for c in COLUMNS if c != "grad"]
                         + [(c, sdc.F32) for c in COLUMNS if c != "grad" and "scale" not in c])
def test_one_element_shared(name, state):
    """Two tensors whose streams of one kind share their last and first element."""
    size = 2 if name == "param" else 4 if name == "master" or (state == sdc.F32 and "scale" not in name) else 1
    n = 8 if "scale" in name else 1000
    first, at = tensor(A, state=state, **{name: 0x700000}), 0x700000 + size * (n - 1)
    assert not build(first, tensor(B, state=state, **{name: at}))
    assert not build(tensor(B, state=state, **{name: at}), first)
    assert build(first, tensor(B, state=state, **{name: at + size}))


def test_across_streams_and_inside():
    assert not build(tensor(A, exp_avg=A))                          # a tensor's own param and exp_avg
    assert not build(tensor(A), tensor(B, master=A + 4))            # a master inside another's param
    assert not build(tensor(A, numel=30000), tensor(B, numel=10, param=A + 2000))   # a small one inside a large one
    assert not build(tensor(A, exp_avg=0x700000), tensor(B, exp_avg_sq=0x700000))
    # behind a long span that begins first, past a short one in between
    assert not build(tensor(A, numel=30000), tensor(B, numel=2, param=A + 100), tensor(B + 0x100000, numel=2, param=A + 300))


def test_what_is_only_read():
    # one gradient for two tensors is read twice
    assert build(tensor(A, grad=0x700000), tensor(B, grad=0x700000))
    # a gradient that the step overwrites is not
    assert not build(tensor(A, grad=A + 1000))
    assert not build(tensor(A), tensor(B, grad=A + 0x20000 + 3998))
    # tensors without a gradient are not stepped: they may share memory with each other
    frozen = dict(grad=0, exp_avg=A, exp_avg_sq=A, master=0)
    assert build(tensor(A, **frozen), tensor(A, **frozen), tensor(B))
    # but their weights are read for their rows, so no step may write them
    assert not build(tensor(B), tensor(A, **dict(frozen, param=B + 100)))


def test_empty_tensors_lie_nowhere():
    assert build(tensor(A, numel=0), tensor(A, numel=0), tensor(A))


def test_long_lists():
    """100,000 tensors in shuffled order, then one that shares an element with another."""
    n, rng = 100_000, np.random.default_rng(1)
    table = np.zeros(n, dtype=sdc._ADAMW_DESC)
    numel = rng.integers(1, 300, n).astype(np.uint64)
    at = np.concatenate([[0], np.cumsum(numel)]).astype(np.uint64)
    for k, (name, size) in enumerate((("param", 2), ("grad", 2), ("exp_avg", 4), ("exp_avg_sq", 4))):
        table[name] = np.uint64((k + 1) << 32) + at[:-1] * np.uint64(size)
    table["numel"], table["param_dtype"], table["grad_dtype"] = numel, sdc.BF16, sdc.BF16
    table["state_dtype"] = sdc.F32
    assert build(table)
    order = rng.permutation(n)
    assert build(table[order])
    table["exp_avg_sq"][1234] -= 4
    assert not build(table) and not build(table[order])


def test_the_binding_names_the_tensors():
    table = np.concatenate([tensor(A), tensor(A + 0x100000), tensor(B, master=A + 0x100000 + 4)])
    assert sdc._adamw_overlap(table) == (("param", 1), ("master", 2))
