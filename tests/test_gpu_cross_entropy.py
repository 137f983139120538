"""GPU tests of the linear head's cross entropy and its gradient against the
formulas in 64 bits.

Tolerances (u = 2^-24, h = half a step of the 16-bit type, eps / 2):
- a logit, d products summed in fp32 in some order: (d + 8) u A with A the sum
  of the products' magnitudes;
- lse: the largest logit's error; each exponential's argument rounds log2(e),
  the product and the shift (3 u |z| each way) and the exponential itself 2 u;
  up to 64 additions and the logarithm: u (6 |z| + 80 + 2 |lse|);
- dz = (p - onehot) as a 16-bit number: p (error of z and lse, 4 u) + h |dz|
  (fp16 holds dz 2^15 times as large: its subnormal step is 2^-40 there);
- dx, dw: those errors through the products, (terms + 8) u of the magnitudes'
  sum for the fp32 additions, and h of the result.
"""
import numpy as np
import pytest
import torch

import silent_corruption_detection_amd as sdc
from _util import assert_rows_equal, oracle_rows, say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make(n, d, v, dtype, seed=1, ignored=0.0, scale=1.0):
    g = gen(seed)
    x = torch.empty(n, d, device=DEV).normal_(0, scale, generator=g).to(dtype)
    w = torch.empty(v, d, device=DEV).normal_(0, d ** -0.5, generator=g).to(dtype)
    t = torch.randint(0, v, (n,), device=DEV, generator=g)
    t = torch.where(torch.rand(n, device=DEV, generator=g) < ignored, torch.full_like(t, -100), t)
    return x, w, t


class Exact:
    """The definition in 64 bits, with each result's error bound."""

    def __init__(self, x, w, t, g=1.0):
        n, d, v = x.shape[0], x.shape[1], w.shape[0]
        X, W = x.double(), w.double()
        live = (t >= 0) & (t < v)
        X = torch.where(live[:, None], X, torch.zeros_like(X)) if n else X
        z = X @ W.t()
        A = X.abs() @ W.abs().t()
        ez = ((d + 8) * U * A).amax(1)
        zmax = z.abs().amax(1)
        self.live = live
        self.lse = torch.logsumexp(z, 1)
        self.tol_lse = ez + U * (6 * zmax + 80 + 2 * self.lse.abs())
        hit = torch.where(live, t, 0)
        at = z.gather(1, hit[:, None])[:, 0]
        self.loss = torch.where(live, self.lse - at, 0.0)
        self.tol_loss = self.tol_lse + ez + 2 * U * (at.abs() + self.loss.abs())
        p = (z - self.lse[:, None]).exp()
        dz = p.clone()
        dz[torch.arange(n, device=DEV), hit] -= 1.0
        dz *= live[:, None]
        h = torch.finfo(x.dtype).eps / 2
        e = (p * (ez + self.tol_lse + 6 * U * (1 + zmax))[:, None] + 2 * U + h * dz.abs() + 2.0 ** -41) * live[:, None]
        self.dx, self.dw = g * dz @ W, g * dz.t() @ X
        mag = dz.abs() + e
        tiny = torch.finfo(x.dtype).tiny * h if x.dtype == FP else 0.0
        gg = abs(g)
        self.tol_dx = gg * ((e + (v + 8) * U * mag) @ W.abs()) + (h + 4 * U) * self.dx.abs() + tiny * 2
        self.tol_dw = gg * ((e + (n + 8) * U * mag).t() @ X.abs()) + (h + 4 * U) * self.dw.abs() + tiny * 2


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol * 1.001 + 1e-30)
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def check(x, w, t, g=0.25, ex=None):
    ex = ex or Exact(x, w, t, g)
    count = torch.empty(1, dtype=torch.int64, device=DEV)
    loss, lse, total = sdc.sdc_cross_entropy(x, w, t, count=count)
    live = ex.live
    close(lse[live], ex.lse[live], ex.tol_lse[live], "lse")
    close(loss, ex.loss, ex.tol_loss * live, "loss")
    assert count.item() == int(live.sum())
    s = loss.double().sum().item()
    assert abs(total.item() - s) <= (U + 1e-12) * abs(s) + 1e-30
    dx, dw = sdc.sdc_cross_entropy_grad(x, w, t, lse, torch.tensor([g], device=DEV))
    torch.cuda.synchronize()
    close(dx, ex.dx, ex.tol_dx, "dx")
    close(dw, ex.dw, ex.tol_dw, "dw")
    return loss, lse, total, dx, dw


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("n, d, v", [
    (1, 1, 1), (1, 8, 2), (2, 7, 3), (1, 64, 300), (3, 65, 255), (17, 63, 256), (16, 128, 257), (64, 72, 511),
    (65, 200, 1000), (255, 256, 129), (256, 64, 512), (257, 320, 513), (300, 1000, 777), (33, 33, 4097),
    (1037, 264, 1501), (5, 2048, 1003), (100, 328, 30000), (400, 200, 25011), (400, 203, 25011), (300, 1027, 30001), (129, 9, 24500)])
def test_sizes(n, d, v, dtype):
    say(f"case xent n={n} d={d} v={v} {dtype}")
    check(*make(n, d, v, dtype, seed=n + d + v, ignored=0.3 if n > 2 else 0.0))


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_large_logits_and_a_sure_row(dtype):
    """Logits of +-100 (sums that overflow without the running maximum), and a
    row whose target holds all the probability."""
    x, w, t = make(130, 64, 700, dtype, seed=2, scale=30.0)
    w[5] = 0
    w[5, :8] = 4.0
    x[3] = 0
    x[3, :8] = 4.0
    t[3] = 5
    loss, *_ = check(x, w, t)
    assert loss[3].item() < 1e-6


def test_strides_and_misaligned_rows():
    x0, w0, t = make(70, 96, 333, BF, seed=3)
    want = check(x0, w0, t)
    for pad, off in ((8, 0), (8, 8), (3, 0), (1, 1), (0, 5)):
        bx = torch.full((70 * (96 + pad) + off + 8,), float("nan"), dtype=BF, device=DEV)
        bw = torch.full((333 * (96 + pad) + off + 8,), float("nan"), dtype=BF, device=DEV)
        x = bx[off:off + 70 * (96 + pad)].view(70, 96 + pad)[:, :96]
        w = bw[off:off + 333 * (96 + pad)].view(333, 96 + pad)[:, :96]
        x.copy_(x0)
        w.copy_(w0)
        got = check(x, w, t)
        for a, b in zip(got, want):   # the same arithmetic whatever the layout
            assert torch.equal(a, b)
    # columns apart: the binding copies
    xt = x0.t().contiguous().t()
    assert torch.equal(sdc.sdc_cross_entropy(xt, w0, t)[1], want[1])


def test_rows_without_a_target_hold_anything():
    x, w, t = make(90, 80, 400, BF, seed=4, ignored=0.4)
    t[0], t[1], t[2] = -1, 400, 1 << 40
    t[3] = -(1 << 40)
    dead = (t < 0) | (t >= 400)
    assert dead.sum() > 10
    ex = Exact(x, w, t, 0.25)
    x = torch.where(dead[:, None], torch.full_like(x, float("nan")), x)
    x[0] = float("inf")
    loss, lse, total, dx, dw = check(x, w, t, ex=ex)
    assert not dx[dead].any() and not loss[dead].any()


def test_no_row_has_a_target_and_no_rows():
    x, w, t = make(40, 64, 300, BF, seed=5, ignored=2.0)
    loss, lse, total, dx, dw = check(x, w, t)
    assert total.item() == 0 and not dx.any() and not dw.any()
    x, w, t = x[:0], w, t[:0]
    count = torch.full((1,), 7, dtype=torch.int64, device=DEV)
    row = torch.full((1, 4), 7, dtype=torch.int64, device=DEV)
    loss, lse, total = sdc.sdc_cross_entropy(x, w, t, count=count, row=row)
    dx, dw = sdc.sdc_cross_entropy_grad(x, w, t, lse, torch.ones(1, device=DEV))
    assert loss.numel() == 0 and total.item() == 0 and count.item() == 0 and not row.any()
    assert dx.shape == (0, 64) and dw.shape == w.shape and not dw.any()


def test_infinite_and_nan_logits():
    x, w, t = make(4, 16, 50, BF, seed=6)
    w[7, 0] = float("inf")
    x[0, 0], x[1, 0], x[2, 0] = 1.0, -1.0, float("nan")
    x[3, 0] = 1.0
    t[:] = 3
    loss, lse, _ = sdc.sdc_cross_entropy(x, w, t)
    assert lse[0].item() == float("inf") and lse[3].item() == float("inf")
    want = torch.logsumexp((x[1:2].double() @ w.double().t()), 1).item()   # -inf among finite logits
    assert abs(lse[1].item() - want) < 1e-4
    assert torch.isnan(lse[2])


def test_several_pieces_of_the_vocabulary():
    """A workspace smaller than the logits: pieces, with a short last one, and a split sum of dx."""
    x, w, t = make(16000, 64, 13001, BF, seed=7, ignored=0.1)
    need = sdc.sdc_cross_entropy_ws_bytes(x, w, t)[1]
    assert need < 16000 * 13001 * 4
    check(x, w, t, g=1.0 / 16000)


def test_pieces_of_copied_operands():
    x, w, t = make(5, 4095, 66000, FP, seed=8)
    check(x, w, t)


def test_split_sum_of_dx():
    check(*make(40, 128, 30011, BF, seed=9))


def test_logit_rows_are_those_of_the_logits():
    """Small whole numbers make every logit exact, so the row is the scan's row
    of the logits in memory; the gradient's recomputed logits have it too."""
    for n, d, v, dtype in ((1, 8, 3, BF), (300, 64, 700, BF), (257, 200, 511, FP), (9, 33, 1025, BF),
                           (100, 72, 30000, FP), (400, 64, 25011, BF), (9, 65, 33000, FP)):
        g = gen(n)
        x = torch.randint(-4, 5, (n, d), device=DEV, generator=g).to(dtype)
        w = torch.randint(-4, 5, (v, d), device=DEV, generator=g).to(dtype)
        t = torch.randint(0, v, (n,), device=DEV, generator=g)
        z = x.float() @ w.float().t()
        want = oracle_rows([z])
        row, again = (torch.empty((1, 4), dtype=torch.int64, device=DEV) for _ in range(2))
        mis = torch.zeros(1, dtype=torch.int32, device=DEV)
        _, lse, _ = sdc.sdc_cross_entropy(x, w, t, row=row)
        one = torch.ones(1, device=DEV)
        sdc.sdc_cross_entropy_grad(x, w, t, lse, one, row=again, ref=row, mismatch=mis)
        torch.cuda.synchronize()
        assert_rows_equal(sdc.rows_numpy(row), want)
        assert_rows_equal(sdc.rows_numpy(again), want)
        assert mis.item() == 0
        w[v // 2, d // 2] += 1   # the head changed between the passes
        x[:, d // 2] = 1
        sdc.sdc_cross_entropy_grad(x, w, t, lse, one, row=again, ref=row, mismatch=mis)
        assert mis.item() == 1


def test_rows_do_not_change_the_results_and_runs_repeat():
    x, w, t = make(500, 192, 5000, BF, seed=10, ignored=0.2)
    g = torch.full((1,), 0.5, device=DEV)
    a = sdc.sdc_cross_entropy(x, w, t)
    da = sdc.sdc_cross_entropy_grad(x, w, t, a[1], g)
    rows = torch.empty((2, 4), dtype=torch.int64, device=DEV)
    mis = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(3):
        b = sdc.sdc_cross_entropy(x, w, t, row=rows[0:1])
        db = sdc.sdc_cross_entropy_grad(x, w, t, b[1], g, row=rows[1:2], ref=rows[0:1], mismatch=mis)
        for p, q in zip(a + da, b + db):
            assert torch.equal(p, q)
    assert mis.item() == 0 and torch.equal(rows[0], rows[1])


@pytest.mark.parametrize("n", [1, 31, 32, 33])
@pytest.mark.parametrize("d", [7, 8, 9, 64, 130, 193, 320])
def test_few_tokens_wherever_their_rows_lie(n, d):
    """Around the smallest tile's 32 tokens, with one to six steps of k: rows of
    x and w at odd element offsets give the bits of aligned ones, and the logits'
    row too, in both passes."""
    say(f"case few n={n} d={d}")
    x0, w0, t = make(n, d, 301, BF, seed=n * d, ignored=0.2 if n > 1 else 0.0)
    want = check(x0, w0, t)
    rows = []
    for pad, off in ((0, 0), (3, 1), (1, 6)):
        bx = torch.full((n * (d + pad) + off + 8,), float("inf"), dtype=BF, device=DEV)
        bw = torch.full((301 * (d + pad) + off + 8,), float("inf"), dtype=BF, device=DEV)
        x = bx[off:off + n * (d + pad)].view(n, d + pad)[:, :d].copy_(x0)
        w = bw[off:off + 301 * (d + pad)].view(301, d + pad)[:, :d].copy_(w0)
        row, again = (torch.zeros(1, 4, dtype=torch.int64, device=DEV) for _ in range(2))
        mismatch = torch.zeros(1, dtype=torch.int32, device=DEV)
        loss, lse, total = sdc.sdc_cross_entropy(x, w, t, row=row)
        dx, dw = sdc.sdc_cross_entropy_grad(x, w, t, lse, torch.tensor([0.25], device=DEV), row=again, ref=row,
                                            mismatch=mismatch)
        assert mismatch.item() == 0 and torch.equal(row, again)
        rows.append(row)
        for got, ref, what in zip((loss, lse, total, dx, dw), want, ("loss", "lse", "total", "dx", "dw")):
            assert torch.equal(got, ref), (what, pad, off)
    assert torch.equal(rows[0], rows[1]) and torch.equal(rows[0], rows[2])


def test_more_tiles_than_one_launch_takes():
    """2^21 tokens over 2^18 + 300 words (8.4 million tiles: a grid has fewer than
    2^32 threads), the word that a token's logit stands out at in the first, a
    middle and the last rows of the vocabulary."""
    n, v = 1 << 21, (1 << 18) + 300
    say(f"case xent n={n} v={v}")
    words = (3, v // 2, v - 1)
    x = torch.zeros(n, 8, dtype=BF, device=DEV)
    w = torch.zeros(v, 8, dtype=BF, device=DEV)
    kind = torch.arange(n, device=DEV) % 3
    x[torch.arange(n, device=DEV), kind] = 8.0
    for j, at in enumerate(words):
        w[at, j] = 1.0
    t = torch.tensor(words, device=DEV)[kind]
    row = torch.empty((1, 4), dtype=torch.int64, device=DEV)
    loss, lse, total = sdc.sdc_cross_entropy(x, w, t, row=row)
    want = np.log(v - 1 + np.exp(8.0))
    # exact logits; the sum and the logarithm as in the note at the top
    tol = U * (6 * 8 + 80 + 2 * want)
    assert (lse.double() - want).abs().max().item() <= tol
    assert (loss.double() - (want - 8)).abs().max().item() <= tol + 2 * U * 16
    assert abs(total.item() - n * (want - 8)) <= n * (tol + 2 * U * 16) + U * n * want
    bits = 0x41000000                                            # of 8.0f
    at = np.arange(n, dtype=np.uint64) * np.uint64(v) + np.array(words, dtype=np.uint64)[np.arange(n) % 3] + np.uint64(1)
    got = sdc.rows_numpy(row)[0].tolist()
    assert got == [n * bits, int(at.sum(dtype=np.uint64)) * bits % 2 ** 64, 0, 0]


def test_gradient_against_differences():
    """Central differences of the 64-bit loss at 16-bit x and w: their error is
    the second-order remainder, e^2 / 6 times a third derivative below 1."""
    x, w, t = make(6, 16, 40, FP, seed=11)
    _, lse, _ = sdc.sdc_cross_entropy(x, w, t)
    dx, dw = sdc.sdc_cross_entropy_grad(x, w, t, lse, torch.ones(1, device=DEV))
    ex = Exact(x, w, t)
    f = lambda X, W: torch.nn.functional.cross_entropy(X @ W.t(), t, reduction="sum").item()  # noqa: E731
    X, W, e = x.double(), w.double(), 1e-4
    for i, k in ((0, 0), (3, 5), (5, 15)):
        P, M = X.clone(), X.clone()
        P[i, k] += e
        M[i, k] -= e
        assert abs((f(P, W) - f(M, W)) / (2 * e) - dx[i, k].item()) <= ex.tol_dx[i, k].item() + 1e-6
    for i, k in ((0, 0), (17, 5), (39, 15)):
        P, M = W.clone(), W.clone()
        P[i, k] += e
        M[i, k] -= e
        assert abs((f(X, P) - f(X, M)) / (2 * e) - dw[i, k].item()) <= ex.tol_dw[i, k].item() + 1e-6


def test_caller_buffers_and_streams():
    x, w, t = make(100, 64, 600, BF, seed=12)
    g = torch.ones(1, device=DEV)
    want = sdc.sdc_cross_entropy(x, w, t)
    dwant = sdc.sdc_cross_entropy_grad(x, w, t, want[1], g)
    fb, gb = sdc.sdc_cross_entropy_ws_bytes(x, w, t)
    ws, wg = (torch.empty(b, dtype=torch.uint8, device=DEV) for b in (fb, gb))
    dx, dw = torch.full_like(x, 9.0), torch.full_like(w, 9.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sdc.sdc_cross_entropy(x, w, t, ws=ws, stream=s)
    sdc.sdc_cross_entropy_grad(x, w, t, got[1], g, dx=dx, dw=dw, ws=wg, stream=s)
    s.synchronize()
    for p, q in zip(want + dwant, got + (dx, dw)):
        assert torch.equal(p, q)
    # two calls at once, each with its own workspace
    x2, w2, t2 = make(700, 64, 900, BF, seed=13)
    want2 = sdc.sdc_cross_entropy(x2, w2, t2)
    torch.cuda.synchronize()
    s2 = torch.cuda.Stream()
    a = sdc.sdc_cross_entropy(x, w, t, stream=s)
    b = sdc.sdc_cross_entropy(x2, w2, t2, stream=s2)
    torch.cuda.synchronize()
    for p, q in zip(want + want2, a + b):
        assert torch.equal(p, q)


def test_captured_and_replayed():
    x, w, t = make(300, 128, 2000, BF, seed=14)
    g = torch.full((1,), 0.5, device=DEV)
    fb, gb = sdc.sdc_cross_entropy_ws_bytes(x, w, t)
    ws, wg = (torch.empty(b, dtype=torch.uint8, device=DEV) for b in (fb, gb))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    row = torch.empty((1, 4), dtype=torch.int64, device=DEV)
    mis = torch.zeros(1, dtype=torch.int32, device=DEV)
    sdc.sdc_cross_entropy(x, w, t, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse, total = sdc.sdc_cross_entropy(x, w, t, ws=ws, row=row)
        sdc.sdc_cross_entropy_grad(x, w, t, lse, g, dx=dx, dw=dw, ws=wg, ref=row, mismatch=mis)
    for k in range(4):
        x2, w2, t2 = make(300, 128, 2000, BF, seed=20 + k, ignored=0.1 * k)
        x.copy_(x2)
        w.copy_(w2)
        t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        want = sdc.sdc_cross_entropy(x2, w2, t2)
        dwant = sdc.sdc_cross_entropy_grad(x2, w2, t2, want[1], g)
        for p, q in zip(want + dwant, (loss, lse, total, dx, dw)):
            assert torch.equal(p, q), k
        assert mis.item() == 0


def test_binding_refuses():
    x, w, t = make(10, 64, 100, BF, seed=15)
    lse, g = torch.zeros(10, device=DEV), torch.ones(1, device=DEV)
    for bad in ((x.float(), w, t), (x, w.half(), t), (x, w[:, :32], t), (x, w, t[:5]), (x, w, t.int()),
                (x, w.cpu(), t), (x, w, t.cpu()), (x[0], w, t)):
        with pytest.raises((ValueError, TypeError)):
            sdc.sdc_cross_entropy(*bad)
    with pytest.raises(ValueError):
        sdc.sdc_cross_entropy(x, w, t, ws=torch.empty(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        sdc.sdc_cross_entropy_grad(x, w, t, lse[:3], g)
    with pytest.raises(ValueError):
        sdc.sdc_cross_entropy_grad(x, w, t, lse, g.double())
    with pytest.raises(ValueError):
        sdc.sdc_cross_entropy_grad(x, w, t, lse, g, dw=torch.empty(99, 64, dtype=BF, device=DEV))
    with pytest.raises(ValueError):
        sdc.sdc_cross_entropy_grad(x, w, t, lse, g, ref=torch.zeros(1, 4, dtype=torch.int64, device=DEV))
    with pytest.raises(sdc.SdcError):
        sdc.sdc_cross_entropy(x[:, :0], w[:, :0], t)
    with pytest.raises(sdc.SdcError):
        sdc.sdc_cross_entropy(x, w[:0], t)
