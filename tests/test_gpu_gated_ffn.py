"""GPU tests of the gated feed-forward block and its gradient against the formulas in
64 bits.

Tolerances (u = 2^-24, h = half a step of the 16-bit type, eps / 2):
- a projection, d products summed in fp32 in some order: (d + 8) u A with A the sum of
  the products' magnitudes;
- y = 1 / (1 + exp(-t)): t is g, or for gelu_tanh a polynomial of it (8 u |t|), times
  log2(e), and the exponential, sum and reciprocal: u (10 |t| + 8) of y and of 1 - y;
- the activation is at most 1.2 times as steep as g, its derivative at most 1.2 times;
- h = act(g) u: its factors' errors, 4 u, and h of the result;
- dg, du: the same and rounded to 16 bits (h, in fp16 at least half a subnormal step,
  2^-25); dx, dw: those through the products, (terms + 64) u of the magnitudes' sum for the
  fp32 additions, and h of the result.
"""
import math

import pytest
import torch

import silent_corruption_detection_amd as sdc
from _util import assert_rows_equal, oracle_rows, say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float16
ACTS = ("silu", "gelu_tanh")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make(n, d, f, dtype, seed=1, scale=1.0):
    g = gen(seed)
    r = lambda std, *s: torch.empty(s, device=DEV).normal_(0, std, generator=g).to(dtype)  # noqa: E731
    return r(scale, n, d), r(d ** -0.5, f, d), r(d ** -0.5, f, d), r(1.0, n, f)


def activation(act, g):
    """(act(g), its derivative, |t|) in 64 bits."""
    if act == "silu":
        y = torch.sigmoid(g)
        return g * y, y + g * y * (1 - y), g.abs()
    c = math.sqrt(2 / math.pi)
    t = c * (g + 0.044715 * g ** 3)
    th = torch.tanh(t)
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g), 2 * t.abs()


def exact(x, wg, wu, dh, act):
    """{name: (value, tolerance)}"""
    X, G, Up, DH = x.double(), wg.double(), wu.double(), dh.double()
    n, d = x.shape
    f, h = wg.shape[0], torch.finfo(x.dtype).eps / 2
    sub = 2.0 ** -25 if x.dtype == FP else 0.0
    g, u = X @ G.t(), X @ Up.t()
    eg, eu = ((d + 8) * U * (X.abs() @ w.abs().t()) for w in (G, Up))
    a, slope, t = activation(act, g)
    ey = U * (10 * t + 8)
    # far out the activation is 0 or g to within less than the smallest terms here
    ea = 1.2 * eg + a.abs() * ey + 1e-38
    es = 1.2 * eg + (slope.abs() + 1) * ey * (t < 80)
    hh = a * u
    done = {"h": (hh, ea * u.abs() + a.abs() * eu + hh.abs() * (h * 1.01 + 4 * U) + ea * eu + sub)}
    dg, du = DH * u * slope, DH * a
    edg = DH.abs() * (slope.abs() * eu + u.abs() * es + es * eu) + dg.abs() * (h * 1.01 + 4 * U) + sub
    edu = DH.abs() * ea + du.abs() * (h * 1.01 + 4 * U) + sub
    mdg, mdu = dg.abs() + edg, du.abs() + edu
    dx = dg @ G + du @ Up
    done["dx"] = (dx, (edg + (2 * f + 64) * U * mdg) @ G.abs() + (edu + (2 * f + 64) * U * mdu) @ Up.abs()
                  + h * 1.01 * dx.abs() + sub)
    for name, w, e, m in (("dw_gate", dg, edg, mdg), ("dw_up", du, edu, mdu)):
        dw = w.t() @ X
        done[name] = (dw, (e + (n + 64) * U * m).t() @ X.abs() + h * 1.01 * dw.abs() + sub)
    return done


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol * 1.001 + 1e-37)
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist(),
                           tol[bad][:4].tolist())


def check(x, wg, wu, dh, act):
    got = {"h": sdc.sdc_gated_ffn(x, wg, wu, act=act)}
    torch.cuda.synchronize()
    got["dx"], got["dw_gate"], got["dw_up"] = sdc.sdc_gated_ffn_grad(x, wg, wu, dh, act=act)
    torch.cuda.synchronize()
    for name, (want, tol) in exact(x, wg, wu, dh, act).items():
        close(got[name], want, tol, name)
    return got


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n, d, f", [
    (1, 1, 1), (1, 8, 2), (2, 7, 3), (1, 64, 300), (3, 65, 15), (17, 63, 16), (16, 128, 17), (32, 72, 33), (33, 200, 100),
    (64, 72, 129), (65, 200, 1000), (255, 256, 129), (256, 64, 512), (257, 320, 257), (300, 1000, 777), (33, 33, 2049),
    (1037, 264, 751), (5, 2048, 1003), (100, 328, 9000), (700, 200, 6011), (4000, 136, 999), (129, 9, 4500), (2000, 72, 5000)])
def test_sizes(n, d, f, act, dtype):
    say(f"case ffn n={n} d={d} f={f} {act} {dtype}")
    check(*make(n, d, f, dtype, seed=n + d + f), act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_large_projections(act, dtype):
    """Projections of +-100 and more, where exp overflows on one side."""
    x, wg, wu, dh = make(130, 64, 200, dtype, seed=2, scale=60.0)
    got = check(x, wg, wu, (dh.float() * 1e-2).to(dtype), act)
    assert got["h"].isfinite().all() and got["dx"].isfinite().all()


@pytest.mark.parametrize("act", ACTS)
def test_projections_of_any_size(act):
    """Up to fp32's end: the activation is 0 or g, its derivative 0 or 1."""
    g = torch.tensor([-1e30, -3e19, -1e10, -200.0, 200.0, 1e10, 3e19, 1e30], device=DEV)
    x = torch.ones(40, 8, dtype=BF, device=DEV)
    wg, wu = torch.zeros(8, 8, dtype=BF, device=DEV), torch.zeros(8, 8, dtype=BF, device=DEV)
    wg[:, 0] = g.to(BF)
    wu[:, 0] = 1.0
    h = sdc.sdc_gated_ffn(x, wg, wu, act=act)
    assert torch.equal(h, torch.where(g > 0, g, 0.0).to(BF).expand(40, 8))
    _, dwg, dwu = sdc.sdc_gated_ffn_grad(x, wg, wu, torch.ones(40, 8, dtype=BF, device=DEV), act=act)
    assert torch.equal(dwg[:, 0], torch.where(g > 0, 40.0, 0.0).to(BF)) and dwu.isfinite().all()


def test_strides_and_misaligned_rows():
    """Halves of one matrix, wide rows, odd offsets: the bits of contiguous tensors."""
    for n, d, f in ((300, 200, 130), (20, 200, 130), (300, 203, 77), (20, 203, 77), (40, 5, 70)):
        x, wg, wu, dh = make(n, d, f, BF, seed=n + d)
        want = (sdc.sdc_gated_ffn(x, wg, wu),) + sdc.sdc_gated_ffn_grad(x, wg, wu, dh)

        def tried(x, wg, wu, dh):
            got = (sdc.sdc_gated_ffn(x, wg, wu),) + sdc.sdc_gated_ffn_grad(x, wg, wu, dh)
            torch.cuda.synchronize()
            for a, b, name in zip(got, want, ("h", "dx", "dw_gate", "dw_up")):
                assert torch.equal(a, b), (name, n, d, f)
        both = torch.cat([wg, wu])
        tried(x, both[:f], both[f:], dh)
        for pad, off in ((3, 1), (8, 0), (1, 6)):
            def lay(t):
                buf = torch.full((t.shape[0] * (t.shape[1] + pad) + off + 8,), math.inf, dtype=BF, device=DEV)
                return buf[off:off + t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], -1)[:, :t.shape[1]].copy_(t)
            tried(*(lay(t) for t in (x, wg, wu, dh)))
        tried(*(t.t().contiguous().t() for t in (x, wg, wu, dh)))
        tried(x, wg, lay(wu), dh)


def test_what_lies_behind_the_rows_has_no_effect():
    """Rows of NaN right behind x, the weights and dh."""
    x, wg, wu, dh = make(70, 72, 50, FP, seed=5)
    want = (sdc.sdc_gated_ffn(x, wg, wu),) + sdc.sdc_gated_ffn_grad(x, wg, wu, dh)
    more = lambda t: torch.cat([t, torch.full_like(t, math.nan)])[:t.shape[0]]  # noqa: E731
    got = (sdc.sdc_gated_ffn(more(x), more(wg), more(wu)),) + sdc.sdc_gated_ffn_grad(more(x), more(wg), more(wu), more(dh))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens():
    x, wg, wu, dh = make(0, 40, 30, BF)
    row = torch.full((1, 4), 7, dtype=torch.int64, device=DEV)
    assert sdc.sdc_gated_ffn(x, wg, wu, row=row).shape == (0, 30) and (row == 0).all()
    dx, dwg, dwu = sdc.sdc_gated_ffn_grad(x, wg, wu, dh)
    assert dx.shape == (0, 40) and (dwg == 0).all() and (dwu == 0).all()
    assert sdc.sdc_gated_ffn_grad(x, wg, wu, dh, need_dw=False)[0].shape == (0, 40)


def test_only_what_is_needed():
    x, wg, wu, dh = make(300, 136, 500, BF, seed=6)
    dx, dwg, dwu = sdc.sdc_gated_ffn_grad(x, wg, wu, dh)
    a = sdc.sdc_gated_ffn_grad(x, wg, wu, dh, need_dw=False)
    b = sdc.sdc_gated_ffn_grad(x, wg, wu, dh, need_dx=False)
    assert a[1] is None and b[0] is None
    assert torch.equal(a[0], dx) and torch.equal(b[1], dwg) and torch.equal(b[2], dwu)


def test_rows_are_those_of_the_projections():
    """Small whole numbers make every projection exact, so the row is the scan's row of
    them in memory; the gradient's recomputed ones have it too."""
    for n, d, f, dtype in ((1, 8, 3, BF), (300, 64, 350, BF), (257, 200, 255, FP), (9, 33, 525, BF), (100, 72, 9000, FP),
                           (400, 64, 12011, BF), (9, 65, 16500, FP), (2000, 64, 4000, BF)):
        g = gen(n)
        x = torch.randint(-4, 5, (n, d), device=DEV, generator=g).to(dtype)
        wg, wu = (torch.randint(-4, 5, (f, d), device=DEV, generator=g).to(dtype) for _ in range(2))
        dh = torch.ones(n, f, dtype=dtype, device=DEV)
        z = torch.stack([x.float() @ wg.float().t(), x.float() @ wu.float().t()], 1)
        want = oracle_rows([z])
        row, again = (torch.empty((1, 4), dtype=torch.int64, device=DEV) for _ in range(2))
        mis = torch.zeros(1, dtype=torch.int32, device=DEV)
        sdc.sdc_gated_ffn(x, wg, wu, row=row)
        sdc.sdc_gated_ffn_grad(x, wg, wu, dh, row=again, ref=row, mismatch=mis)
        torch.cuda.synchronize()
        assert_rows_equal(sdc.rows_numpy(row), want)
        assert_rows_equal(sdc.rows_numpy(again), want)
        assert mis.item() == 0
        wu[f // 2, d // 2] += 1   # a weight changed between the passes
        x[:, d // 2] = 1
        sdc.sdc_gated_ffn_grad(x, wg, wu, dh, row=again, ref=row, mismatch=mis)
        assert mis.item() == 1


def test_rows_do_not_change_the_results_and_runs_repeat():
    for n, act in ((500, "silu"), (20, "gelu_tanh")):
        x, wg, wu, dh = make(n, 192, 1100, BF, seed=10)
        want = (sdc.sdc_gated_ffn(x, wg, wu, act),) + sdc.sdc_gated_ffn_grad(x, wg, wu, dh, act)
        rows = torch.empty((2, 4), dtype=torch.int64, device=DEV)
        mis = torch.zeros(1, dtype=torch.int32, device=DEV)
        for _ in range(3):
            got = (sdc.sdc_gated_ffn(x, wg, wu, act, row=rows[:1]),) + sdc.sdc_gated_ffn_grad(
                x, wg, wu, dh, act, row=rows[1:], ref=rows[:1], mismatch=mis)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert mis.item() == 0 and torch.equal(rows[0], rows[1])


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(act):
    x, wg, wu, dh = make(40, 64, 90, FP, seed=11)
    grads = sdc.sdc_gated_ffn_grad(x, wg, wu, dh, act)
    g = gen(12)
    base = [t.double() for t in (x, wg, wu)]
    loss = lambda x, wg, wu: (activation(act, x @ wg.t())[0] * (x @ wu.t()) * dh.double()).sum()  # noqa: E731
    for i in range(3):
        step = torch.empty(base[i].shape, device=DEV, dtype=torch.float64).normal_(0, 1, generator=g)
        at = lambda e: loss(*[t + e * step if j == i else t for j, t in enumerate(base)])  # noqa: E731
        slope = (at(1e-5) - at(-1e-5)) / 2e-5
        got = (grads[i].double() * step).sum()
        # each gradient is off by its rounding, twice (its own and its factors'), in a sum of random signs
        assert (got - slope).abs() <= 8 * torch.finfo(FP).eps * (grads[i].double() * step).norm() + 1e-6


def test_outputs_workspace_another_stream_and_graphs():
    x, wg, wu, dh = make(300, 203, 411, BF, seed=13)
    want = (sdc.sdc_gated_ffn(x, wg, wu),) + sdc.sdc_gated_ffn_grad(x, wg, wu, dh)
    need = sdc.sdc_gated_ffn_ws_bytes(x, wg, wu)
    ws = [torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV) for n in need]
    given = [torch.empty_like(t) for t in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (sdc.sdc_gated_ffn(x, wg, wu, out=given[0], ws=ws[0], stream=side),) + sdc.sdc_gated_ffn_grad(
        x, wg, wu, dh, dx=given[1], dw_gate=given[2], dw_up=given[3], ws=ws[1], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) and b.data_ptr() == c.data_ptr() for a, b, c in zip(want, got, given))
    assert all((w[n:] == 0xFF).all() for w, n in zip(ws, need))
    y = make(9, 136, 300, FP, seed=14)
    graphs = []
    for a in ((x, wg, wu, dh), y):
        sdc.sdc_gated_ffn_grad(*a)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = (sdc.sdc_gated_ffn(*a[:3]),) + sdc.sdc_gated_ffn_grad(*a)
        graphs.append((g, a, got))
    for turn in range(3):
        for g, a, got in graphs:
            a[0].copy_(a[0].roll(1, 0))
            g.replay()
            want = (sdc.sdc_gated_ffn(*a[:3]),) + sdc.sdc_gated_ffn_grad(*a)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(want, got)), turn
