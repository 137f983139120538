"""GPU tests of the AdamW step against the formulas in 64 bits.

Tolerances, with u = 2^-24 the largest relative rounding of fp32:
- m = fma(b1, m0, omb1 * g): the rounded b1, omb1 and scaled g, the product and
  the sum: at most 5 u (|b1 m0| + |omb1 g|).
- v, a sum of terms above zero: 8 u v.
- p = fma(-size, q, p0 * decay): the rounded decay, the product and the sum,
  4 u |p0|; q = m / (sqrt(v) rbc2 + eps) with sqrt and reciprocal off by at
  most 2 u each and seven more roundings, 16 u |update|, and what m's own error
  moves.  A 16-bit weight is off by half a step more.
- An 8-bit state is one of the two neighbours of the exact value, and the one
  that the element's random bits choose, except where the choice hangs on less
  than the errors above.
"""
import ctypes

import numpy as np
import pytest
import torch

import silent_corruption_detection_amd as sdc
from _util import assert_rows_equal, oracle_rows, say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HYPER = [[3e-4, 0.9, 0.95, 1e-8, 0.1], [1e-2, 0.8, 0.999, 1e-6, 0.0]]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def blocks(n):
    return -(-n // 128)


class List:
    """Tensors of the given sizes carved one after the other from one buffer
    per stream (so they start at odd element offsets), and their plan."""

    def __init__(self, sizes, param, grad, master, state, seed=1, control_step=10, offset=0, frozen=()):
        g = gen(seed)
        n = sum(sizes)
        rnd = lambda std: torch.empty(n + offset, device=DEV).normal_(0, std, generator=g)[offset:]  # noqa: E731
        w = rnd(0.02)
        self.p = torch.empty(n + offset, dtype=TYPES[param], device=DEV)[offset:].copy_(w)
        self.w = w if master else None
        self.g = torch.empty(n + offset, dtype=TYPES[grad], device=DEV)[offset:].copy_(
            rnd(1e-3) * torch.rand(n, device=DEV, generator=g))
        nb = sum(blocks(s) for s in sizes)
        self.ms = self.vs = None
        if state == 32:
            self.m, self.v = rnd(3e-4), rnd(1.0).exp_().mul_(3e-7)
        else:
            self.m = torch.empty(n + offset, dtype=E4M3, device=DEV)[offset:].copy_(rnd(80).clamp(-200, 200))
            self.v = torch.empty(n + offset, dtype=E4M3, device=DEV)[offset:].copy_(
                rnd(0.7).exp_().mul_(40).clamp_(0.05, 230))
            self.ms = torch.randint(105, 112, (nb,), dtype=torch.uint8, device=DEV, generator=g)
            self.vs = torch.randint(106, 112, (nb,), dtype=torch.uint8, device=DEV, generator=g)
        self.sizes, self.state, self.frozen = sizes, state, frozen
        self.group = [k % 2 for k in range(len(sizes))]
        split = lambda t: list(t.split(sizes))  # noqa: E731
        scales = None if state == 32 else [list(t.split([blocks(s) for s in sizes])) for t in (self.ms, self.vs)]
        grads = [None if k in frozen else t for k, t in enumerate(split(self.g))]
        self.params = split(self.p)
        self.plan = sdc.sdc_adamw_plan_build(
            self.params, grads, split(self.m), split(self.v), master=split(w) if master else None,
            exp_avg_scale=scales and scales[0], exp_avg_sq_scale=scales and scales[1],
            group=self.group, n_groups=2)
        self.groups = torch.tensor(HYPER, dtype=torch.float64, device=DEV)
        self.control = sdc.sdc_adamw_control(DEV, step=control_step, seed=77 + seed)

    def streams(self):
        return [t for t in (self.p, self.w, self.m, self.v, self.ms, self.vs) if t is not None]

    def snapshot(self):
        """Copies of everything a step reads, as host float64 (bytes for scales)."""
        f = lambda t: None if t is None else (t.cpu().numpy().copy() if t.dtype == torch.uint8  # noqa: E731
                                              else t.float().cpu().numpy().astype(np.float64))
        return {k: f(getattr(self, k)) for k in ("p", "w", "g", "m", "v", "ms", "vs")}

    def per_element(self):
        """(group, block index, index over the list) of every element."""
        grp = np.repeat(np.array(self.group), self.sizes)
        base = np.cumsum([0] + [blocks(s) for s in self.sizes])
        blk = np.concatenate([base[k] + np.arange(s) // 128 for k, s in enumerate(self.sizes)] or [np.zeros(0, int)])
        live = np.concatenate([np.full(s, k not in self.frozen) for k, s in enumerate(self.sizes)])
        return grp, blk, live


def random_bits(seed, t, index):
    m = np.uint64(0xFFFFFFFF)
    index = index.astype(np.uint64)
    k0 = ((seed & 0xFFFFFFFF) * 0x9E3779B1 + (t & 0xFFFFFFFF) * 0x85157AF5) & 0xFFFFFFFF
    k1 = ((seed >> 32) * 0x9E3779B1 + (t >> 32) * 0x85157AF5 + 0x6C8E9CF5) & 0xFFFFFFFF
    a = ((index & m) + np.uint64(k0)) & m
    a = ((a ^ (a >> np.uint64(16))) * np.uint64(0x7FEB352D)) & m
    a ^= (np.uint64(k1) + (index >> np.uint64(32)) * np.uint64(0x2C1B3C6D)) & m
    a = ((a ^ (a >> np.uint64(15))) * np.uint64(0x846CA68B)) & m
    return (a ^ (a >> np.uint64(16))).astype(np.int64)


def neighbours(t):
    """The e4m3 values below (or at) and above each t in [0, 448)."""
    e = np.maximum(np.floor(np.log2(np.maximum(t, 2.0 ** -30))), -6)
    e = np.where(2.0 ** e > np.maximum(t, 2.0 ** -6), e - 1, e)
    step = 2.0 ** (np.maximum(e, -6) - 3)
    lo = np.floor(t / step) * step
    return lo, lo + step


def check_codes(got, scale, want, tol, blk, bits, root):
    """got: held e4m3 values, scale bytes; want: the exact m or sqrt(v) with
    absolute error bounds tol; bits: the elements' random bits."""
    top = np.zeros(len(scale))
    np.maximum.at(top, blk, np.abs(want))
    e = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1))), -300) - 7
    s = np.maximum(e + 127, 1)
    assert np.array_equal(scale.astype(np.float64), s)
    unit = 2.0 ** (s[blk] - 127)
    t, tol = np.abs(want) / unit, tol / unit
    lo, hi = neighbours(t)
    if root:
        u = ((bits >> 16) + 0.5) / 65536
        gap = u * (hi * hi - lo * lo) - (t * t - lo * lo)
        margin = 2 * hi * tol + 8 * U * hi * hi
        up = gap < 0
    else:
        gap = (t - lo) / (hi - lo) + ((bits & 0xFFFF) * 16 + 8) / 2 ** 20 - 1
        margin = tol / (hi - lo) + 2.0 ** -19
        up = gap >= 0
    held = np.where(up, hi, lo)
    if root:
        held = np.where((want > 0) & (held == 0), 2.0 ** -9, held)
    sure = (np.abs(gap) > margin) | (want == 0)   # zero is held as zero whatever its bits
    mag = np.abs(got)
    assert np.array_equal(mag[sure], held[sure]), (np.flatnonzero(sure & (mag != held))[:5],)
    near = ((mag >= lo - tol - 1e-30) & (mag <= hi + (hi - lo))) if not root else (mag <= hi + (hi - lo))
    assert near.all()
    assert sure.mean() > 0.99 or sure.size < 1000
    signed = got[(mag > 0)] * want[(mag > 0)]
    assert (signed >= 0).all()


def check_step(lst, before, after, t, scale=1.0, first=0):
    grp, blk, live = lst.per_element()
    hyper = np.array(HYPER)[grp].T if len(grp) else np.zeros((5, 0))
    lr, b1, b2, eps, wd = hyper
    p0 = before["w"] if before["w"] is not None else before["p"]
    g = before["g"] * scale
    if lst.state == 32:
        m0, v0 = before["m"], before["v"]
    else:
        m0 = before["m"] * 2.0 ** (before["ms"][blk].astype(np.float64) - 127)
        v0 = (before["v"] * 2.0 ** (before["vs"][blk].astype(np.float64) - 127)) ** 2
    m = b1 * m0 + (1 - b1) * g
    v = b2 * v0 + (1 - b2) * g * g
    tol_m, tol_v = 5 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g)) + 1e-40, 8 * U * v + 1e-40
    den = np.sqrt(v / (1 - b2 ** t)) + eps
    size = lr / (1 - b1 ** t)
    upd = size * m / den
    p = p0 * (1 - lr * wd) - upd
    tol_p = 4 * U * np.abs(p0) + 16 * U * np.abs(upd) + size * tol_m / den + 1e-40
    for k, want, tol in (("w", p, tol_p), ("p", p, tol_p)):
        if after[k] is None:
            continue
        if k == "p" and lst.p.dtype != torch.float32:
            info = torch.finfo(lst.p.dtype)
            tol = tol + info.eps / 2 * np.maximum(np.abs(p) + tol, info.tiny)
        bad = np.abs(after[k] - want) > tol
        assert not (bad & live).any(), (k, np.flatnonzero(bad & live)[:5], after[k][bad & live][:5], want[bad & live][:5])
    for k in before:  # tensors without a gradient, and the gradients, are untouched
        if before[k] is not None and len(before[k]) == len(live):
            same = before[k] == after[k]
            assert same[~live].all() and (k != "g" or same.all())
    if lst.state == 32:
        assert (np.abs(after["m"] - m) <= tol_m)[live].all()
        assert (np.abs(after["v"] - v) <= tol_v)[live].all()
        return
    bits = random_bits(int(lst.control[2]), t, first + np.arange(len(live)))
    used = np.zeros(len(before["ms"]), bool)
    used[blk[live]] = True
    assert (after["ms"] == before["ms"])[~used].all() and (after["vs"] == before["vs"])[~used].all()
    if not live.any():
        return
    sub = np.cumsum(used) - 1
    check_codes(after["m"][live], after["ms"][used], m[live], tol_m[live], sub[blk[live]], bits[live], False)
    r = np.sqrt(v)
    check_codes(after["v"][live], after["vs"][used], r[live], (6 * U * r)[live], sub[blk[live]], bits[live], True)


SIZES = [1, 7, 8, 127, 128, 129, 511, 2048, 2049, 4097, 20_000, 3]


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("grad", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("param, master", [("f32", False), ("bf16", False), ("bf16", True), ("f16", False),
                                           ("f16", True)])
def test_step_matches_the_formulas(param, grad, master, state):
    lst = List(SIZES, param, grad, master, state, seed=3, offset=1)
    rows = torch.empty((len(SIZES), 4), dtype=torch.int64, device=DEV)
    for k in range(3):
        before = lst.snapshot()
        sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control, rows=rows)
        torch.cuda.synchronize()
        check_step(lst, before, lst.snapshot(), 11 + k)
        assert_rows_equal(sdc.rows_numpy(rows), oracle_rows(lst.params))
    assert lst.control.tolist()[:2] == [13, 0]


@pytest.mark.parametrize("n, state, param", [(3_000_001, 32, "f32"), (3_000_001, 8, "bf16"),
                                             (9_000_128, 8, "f16"), (9_000_003, 32, "bf16")])
def test_large_tensors_of_many_items(n, state, param):
    lst = List([5, n, 300], param, param, False, state, seed=4)
    rows = torch.empty((3, 4), dtype=torch.int64, device=DEV)
    before = lst.snapshot()
    sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control, rows=rows)
    torch.cuda.synchronize()
    check_step(lst, before, lst.snapshot(), 11)
    assert_rows_equal(sdc.rows_numpy(rows), oracle_rows(lst.params))


def test_rows_do_not_change_the_step():
    a, b = (List(SIZES, "bf16", "bf16", True, 8, seed=5) for _ in range(2))
    sdc.sdc_adamw_step(a.plan, a.groups, a.control)
    sdc.sdc_adamw_step(b.plan, b.groups, b.control, rows=torch.empty((len(SIZES), 4), dtype=torch.int64, device=DEV))
    for x, y in zip(a.streams(), b.streams()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_replayed_steps_give_the_same_bits():
    a, b = (List(SIZES, "bf16", "f32", False, 8, seed=6) for _ in range(2))
    for _ in range(4):
        for l in (a, b):
            sdc.sdc_adamw_step(l.plan, l.groups, l.control)
    for x, y in zip(a.streams(), b.streams()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_clip_and_scale_from_the_squared_norm():
    lst = List(SIZES, "f32", "f32", False, 32, seed=7)
    gplan = sdc.sdc_plan_build(list(lst.g.split(SIZES)))
    _, total, flag = sdc.sdc_sqnorm(gplan)
    norm = float(lst.g.double().square().sum().sqrt())
    for max_norm, gs in ((norm / 3, 1.0), (norm * 10, 0.5), (norm / 8, 0.25)):
        before = lst.snapshot()
        t = int(lst.control[0]) + 1
        sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control, sq_total=total, flag=flag, max_norm=max_norm,
                           grad_scale=gs)
        c = gs * min(1.0, max_norm / (norm * gs + 1e-6))
        check_step(lst, before, lst.snapshot(), t, scale=c)
        assert abs(lst.control[3:].view(torch.float32)[0].item() - c) <= 1e-6 * c


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("what", ["nan", "inf", "overflow", "flag"])
def test_a_bad_gradient_takes_no_step(what, state):
    lst = List(SIZES, "bf16", "f32", True, state, seed=8)
    gplan = sdc.sdc_plan_build(list(lst.g.split(SIZES)))
    total = flag = None
    if what == "flag":
        flag = torch.ones(1, dtype=torch.int32, device=DEV)
    else:
        lst.g[1000] = {"nan": float("nan"), "inf": float("-inf"), "overflow": 3e38}[what]
        _, total, flag = sdc.sdc_sqnorm(gplan)
        if what != "overflow":
            flag = None   # the total alone decides
    kept = [t.clone() for t in lst.streams()]
    rows = torch.zeros((len(SIZES), 4), dtype=torch.int64, device=DEV)
    sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control, sq_total=total, flag=flag, rows=rows)
    for x, y in zip(kept, lst.streams()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert lst.control.tolist()[:2] == [10, 1] and lst.control[3].item() >> 32 == 1
    assert_rows_equal(sdc.rows_numpy(rows), oracle_rows(lst.params))
    # the next good gradient takes step 11
    lst.g[1000] = 1e-3
    before = lst.snapshot()
    sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control)
    check_step(lst, before, lst.snapshot(), 11)
    assert lst.control.tolist()[:2] == [11, 1]


def test_an_ungated_nan_stays_in_its_block():
    for state in (32, 8):
        lst = List([512, 640], "f32", "f32", False, state, seed=9)
        lst.g[130], lst.g[700] = float("nan"), float("inf")
        sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control)
        bad = ~torch.isfinite(lst.p)
        assert bad.nonzero().flatten().tolist() == [130, 700]
        m = torch.isfinite(lst.m.float())
        assert (~m).nonzero().flatten().tolist() == [130, 700]


def test_tensors_without_a_gradient_and_empty_ones():
    for state in (32, 8):
        lst = List([100, 0, 5000, 300, 0], "bf16", "bf16", True, state, seed=10, frozen=(0, 2))
        rows = torch.full((5, 4), -1, dtype=torch.int64, device=DEV)
        before = lst.snapshot()
        sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control, rows=rows)
        check_step(lst, before, lst.snapshot(), 11)
        assert_rows_equal(sdc.rows_numpy(rows), oracle_rows(lst.params))


def test_from_the_empty_state():
    """All-zero 8-bit states and step 0; gradients of zero leave zero states and only decay the weights."""
    lst = List([1000, 4000], "f32", "f32", False, 8, seed=11, control_step=0)
    for t in (lst.m, lst.v, lst.ms, lst.vs):
        t.view(torch.uint8).zero_()
    lst.g[:128].zero_()
    before = lst.snapshot()
    sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control)
    after = lst.snapshot()
    check_step(lst, before, after, 1)
    assert not after["m"][:128].any() and not after["v"][:128].any()
    assert (after["v"][128:] > 0).all()   # a second moment above zero is never held as zero


def test_random_bits_beyond_32_bits_of_the_list():
    """The element counter passes 2^32 inside the second tensor; the first has no gradient."""
    n0 = (1 << 32) - 1000
    big = torch.zeros(n0, dtype=torch.bfloat16, device=DEV)
    code = torch.zeros(n0, dtype=torch.uint8, device=DEV)
    scale = torch.zeros(blocks(n0), dtype=torch.uint8, device=DEV)
    lst = List([5000], "bf16", "bf16", False, 8, seed=12)
    plan = sdc.sdc_adamw_plan_build([big, lst.p], [None, lst.g], [code.view(E4M3), lst.m], [code.view(E4M3), lst.v],
                                    exp_avg_scale=[scale, lst.ms], exp_avg_sq_scale=[scale, lst.vs], n_groups=2)
    before = lst.snapshot()
    sdc.sdc_adamw_step(plan, lst.groups, lst.control)
    check_step(lst, before, lst.snapshot(), 11, first=n0)
    assert not code.any()


def test_captured_steps_follow_the_schedule():
    """A captured step with rows replays with the learning rate of its time,
    beside eager work on the same tensors."""
    a, b = (List(SIZES, "bf16", "bf16", True, 8, seed=13) for _ in range(2))
    rows = torch.empty((len(SIZES), 4), dtype=torch.int64, device=DEV)
    gplan = sdc.sdc_plan_build(list(a.g.split(SIZES)))
    sq, total, flag = sdc.sdc_sqnorm(gplan)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sdc.sdc_sqnorm(gplan, sq, total, flag)
        sdc.sdc_adamw_step(a.plan, a.groups, a.control, sq_total=total, flag=flag, max_norm=0.05, rows=rows)
    assert a.control[0].item() == 10
    for k in range(4):
        lr = 1e-3 / (k + 1)
        for l in (a, b):
            l.groups[:, 0] = lr
            l.g.copy_(torch.empty_like(l.g, dtype=torch.float32).normal_(0, 1e-3, generator=gen(100 + k)))
        graph.replay()
        torch.cuda.synchronize()
        _, tot, flg = sdc.sdc_sqnorm(sdc.sdc_plan_build(list(b.g.split(SIZES))))
        sdc.sdc_adamw_step(b.plan, b.groups, b.control, sq_total=tot, flag=flg, max_norm=0.05)
        for x, y in zip(a.streams(), b.streams()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), k
        assert_rows_equal(sdc.rows_numpy(rows), oracle_rows(a.params))
    assert a.control[0].item() == 14


def test_on_another_stream():
    lst = List(SIZES, "f32", "f32", False, 32, seed=14)
    before = lst.snapshot()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control, stream=s)
    s.synchronize()
    check_step(lst, before, lst.snapshot(), 11)


def test_two_plans_at_once_on_two_streams():
    a, b = List([200_000, 77], "bf16", "bf16", False, 8, seed=15), List([150_000, 5], "f32", "f32", False, 32, seed=16)
    ba, bb = a.snapshot(), b.snapshot()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    sdc.sdc_adamw_step(a.plan, a.groups, a.control, stream=s1)
    sdc.sdc_adamw_step(b.plan, b.groups, b.control, stream=s2)
    torch.cuda.synchronize()
    check_step(a, ba, a.snapshot(), 11)
    check_step(b, bb, b.snapshot(), 11)


def test_mixed_list_in_one_plan():
    """fp32 norms with fp32 states beside 16-bit matrices with 8-bit states."""
    g = gen(17)
    r = lambda n, std=1e-2: torch.empty(n, device=DEV).normal_(0, std, generator=g)  # noqa: E731
    p = [r(5000).bfloat16(), r(64), r(300).half()]
    gr = [r(5000, 1e-3).bfloat16(), r(64, 1e-3), r(300, 1e-3)]
    z = lambda n: torch.zeros(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    m = [z(5000).view(E4M3), torch.zeros(64, device=DEV), torch.zeros(300, device=DEV)]
    v = [z(5000).view(E4M3), torch.zeros(64, device=DEV), torch.zeros(300, device=DEV)]
    ms, vs = [z(40), None, None], [z(40), None, None]
    plan = sdc.sdc_adamw_plan_build(p, gr, m, v, exp_avg_scale=ms, exp_avg_sq_scale=vs)
    groups = torch.tensor([HYPER[0]], dtype=torch.float64, device=DEV)
    rows = torch.empty((3, 4), dtype=torch.int64, device=DEV)
    want = [x.double() * (1 - 3e-5) - 3e-4 * y.double() / (y.double().abs() + 1e-8) for x, y in zip(p, gr)]
    sdc.sdc_adamw_step(plan, groups, sdc.sdc_adamw_control(DEV), rows=rows)
    for x, w in zip(p, want):
        # the first step's update is lr * sign(g); fp32 errors as above, then half a step of the type
        tol = 20 * U * (w.abs() + 1e-3) + torch.finfo(x.dtype).eps / 2 * w.abs() + 2.0 ** -25
        assert ((x.double() - w).abs() <= tol).all()
    assert_rows_equal(sdc.rows_numpy(rows), oracle_rows(p))


def test_more_tensors_than_one_launch_takes():
    """2^23 + 70 tensors of one weight each, through the C entry points: their
    items need two launches, as a grid has fewer than 2^32 threads."""
    n = (1 << 23) + 70
    say(f"case adamw of {n} tensors")
    g = gen(19)
    p, gr, m, v = (torch.empty(n, device=DEV).normal_(generator=g) for _ in range(4))
    v.abs_()
    p0 = p.double()
    want_m = 0.9 * m.double() + (1 - 0.9) * gr.double()
    want_v = 0.99 * v.double() + (1 - 0.99) * gr.double() ** 2
    den = want_v.sqrt() / (1 - 0.99) ** 0.5 + 1e-8
    update = 1e-2 / (1 - 0.9) * want_m / den
    tol_m = 5 * U * (0.9 * m.double().abs() + 0.1 * gr.double().abs())
    table = np.zeros(n, dtype=sdc._ADAMW_DESC)
    for name, t in (("param", p), ("grad", gr), ("exp_avg", m), ("exp_avg_sq", v)):
        table[name] = np.arange(n, dtype=np.uint64) * 4 + t.data_ptr()
    table["numel"] = 1
    table["param_dtype"] = table["grad_dtype"] = table["state_dtype"] = sdc.F32
    h, nbytes, info = ctypes.c_void_p(table.ctypes.data), ctypes.c_uint64(0), sdc._AdamwInfo()
    assert sdc._lib.sdc_adamw_plan_bytes(h, n, 1, ctypes.byref(nbytes)) == 0
    buf = torch.empty(nbytes.value, dtype=torch.uint8, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    assert sdc._lib.sdc_adamw_plan_build(h, n, 1, buf.data_ptr(), buf.numel(), ctypes.byref(info), s) == 0
    assert sum(info.n_wave) == n
    groups = torch.tensor([[1e-2, 0.9, 0.99, 1e-8, 0.0]], dtype=torch.float64, device=DEV)
    rows = torch.zeros((n, 4), dtype=torch.int64, device=DEV)
    sdc.sdc_adamw_step(sdc.AdamwPlan(buf, info, [], torch.device(DEV, 0)), groups, sdc.sdc_adamw_control(DEV), rows=rows)
    assert ((m.double() - want_m).abs() <= tol_m).all()
    assert ((v.double() - want_v).abs() <= 8 * U * want_v).all()
    tol_p = 4 * U * p0.abs() + 16 * U * update.abs() + 1e-2 / (1 - 0.9) * tol_m / den
    assert ((p.double() - (p0 - update)).abs() <= tol_p).all()
    bits = p.view(torch.int32).long() & 0xFFFFFFFF
    assert torch.equal(rows[:, 0], bits) and torch.equal(rows[:, 1], bits) and torch.equal(rows[:, 2], bits)
    assert not rows[:, 3].any()


def test_binding_refuses():
    lst = List([100], "bf16", "bf16", False, 32, seed=18)
    P, G, M, V = [lst.p], [lst.g], [lst.m], [lst.v]
    build = sdc.sdc_adamw_plan_build
    with pytest.raises(TypeError):
        build([lst.p.double()], G, M, V)
    with pytest.raises(TypeError):
        build(P, G, [lst.m.bfloat16()], V)
    with pytest.raises(TypeError):
        build(P, G, M, [lst.v.to(E4M3)])
    with pytest.raises(ValueError):
        build(P, [lst.g[:50]], M, V)
    with pytest.raises(ValueError):
        build(P, [lst.g.cpu()], M, V)
    with pytest.raises(ValueError):
        build(P, [], M, V)
    for twice in ((P * 2, G * 2, M + [M[0].clone()], V + [V[0].clone()]),
                  (P, G, M, M),
                  (P + [P[0].clone()], G * 2, M * 2, V + [V[0].clone()])):
        with pytest.raises(ValueError, match="listed twice"):
            build(*twice)
    with pytest.raises(ValueError):
        build([torch.zeros(10, 20, device=DEV).bfloat16().t()[:, :10]], G, M, V)
    with pytest.raises(sdc.SdcError):
        build(P, G, M, V, group=[3], n_groups=2)
    with pytest.raises(sdc.SdcError):   # 8-bit states need their scale bytes
        build(P, G, [lst.m.to(E4M3)], [lst.v.to(E4M3)])
    with pytest.raises(ValueError):
        sdc.sdc_adamw_step(lst.plan, lst.groups[:1], lst.control)
    with pytest.raises(ValueError):
        sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control.cpu())
    with pytest.raises(ValueError):
        sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control, rows=torch.empty(2, dtype=torch.int64, device=DEV))
    with pytest.raises(sdc.SdcError):
        sdc.sdc_adamw_step(lst.plan, lst.groups, lst.control, max_norm=1.0)
    assert lst.control.tolist() == [10, 0, 95, 0]
