"""GPU tests of the linear head's cross entropy at logits of any magnitude.

In the first tests each logit is one product of two numbers of at most 8 significant bits, so it is
exact in fp32, and what is tested is the softmax alone.  A row's largest logit
stands so far above the others that its probability is 1 and theirs 0 to far
below fp32: lse is that logit, rounded once (u = 2^-24 of it), and the gradient
is a difference of two rows of w (of x), rounded once.
"""
import pytest
import torch

import silent_corruption_detection_amd as sdc
from _util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float16


def exact_rows(n, d, v, dtype, a, b, seed=0):
    """x, w, target and the logits: row n of x has +-a in its first place, word k
    has b times one of 1, 7/8, .. 1/8, -1/8, .. -1 there, so the logits' magnitudes
    are a b k / 8; half the rows have their largest at the positive end, half at the
    other."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    step = torch.randint(1, 8, (v,), device=DEV, generator=g) * (torch.randint(0, 2, (v,), device=DEV, generator=g) * 2 - 1)
    step[v // 3], step[v // 2] = 8, -8                     # each end once
    x = torch.zeros(n, d, dtype=dtype, device=DEV)
    w = torch.zeros(v, d, dtype=dtype, device=DEV)
    x[:, 0] = a
    x[1::2, 0] = -a
    w[:, 0] = (step.double() * (b / 8)).to(dtype)
    t = torch.randint(0, v, (n,), device=DEV, generator=g)
    t[::5] = v // 3
    return x, w, t, x[:, :1].double() @ w[:, :1].double().t()


def check_sure_rows(x, w, t, z):
    n = x.shape[0]
    top, best = z.max(1)
    loss, lse, _ = sdc.sdc_cross_entropy(x, w, t)
    # the sum of the others: at most v exp(-a b / 8), nothing in fp32
    assert ((lse.double() - top).abs() <= U * top.abs()).all(), (lse[:4], top[:4])
    at = z.gather(1, t[:, None])[:, 0]
    # lse - z_target: one more rounding.  Where it passes fp32's largest number,
    # 3.403e38 (2.85e38 - -2.14e38 = 4.99e38), that rounding gives Inf.
    want = top - at
    over = want > 3.4028235677973366e38
    assert (loss[over] == float("inf")).all()
    assert ((loss.double() - want).abs()[~over] <= 2 * U * (top.abs() + at.abs())[~over]).all(), (loss[:4], want[:4])
    dx, dw = sdc.sdc_cross_entropy_grad(x, w, t, lse, torch.ones(1, device=DEV))
    torch.cuda.synchronize()
    h = torch.finfo(x.dtype).eps / 2
    tiny = torch.finfo(x.dtype).tiny * h
    one = torch.zeros_like(z)
    rows = torch.arange(n, device=DEV)
    one[rows, best] += 1.0
    one[rows, t] -= 1.0                                    # dz: -1, 0 and 1, exact in 16 bits
    for got, want, mag, terms in ((dx, one @ w.double(), one.abs() @ w.double().abs(), z.shape[1]),
                                  (dw, one.t() @ x.double(), one.abs().t() @ x.double().abs(), n)):
        # sums of few-bit numbers: 2 u of the magnitudes for each addition, h of the result
        tol = h * want.abs() + (terms + 8) * U * mag + tiny
        # beyond the 16-bit type's largest number (sums of many rows) the result is Inf
        over = want.abs() > torch.finfo(x.dtype).max * (1 - h)
        bad = ~((got.double() - want).abs() <= tol) & ~over
        assert not bad.any(), (got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("n, d, v", [(5, 8, 301), (70, 9, 700), (400, 8, 25011), (2000, 16, 8000)],
                         ids=["32", "64", "128", "256"])   # tokens of a tile
@pytest.mark.parametrize("a, b, dtype", [
    (1000.0, 1000.0, BF), (1000.0, 1000.0, FP), (53248.0, 57344.0, FP), (60000.0, 50176.0, BF),
    (1e5, 1e5, BF), (60416.0, 60416.0, FP), (1.5e19, 1.9e19, BF)], ids=str)
def test_logits_of_any_magnitude(a, b, dtype, n, d, v):
    """Magnitudes of 1e6, 3e9, 1e10 and 3e38, both signs, in each shape of tile."""
    say(f"case xent a={a} b={b} n={n} d={d} v={v} {dtype}")
    a, b = (float(torch.tensor(q).to(dtype)) for q in (a, b))
    check_sure_rows(*exact_rows(n, d, v, dtype, a, b))


@pytest.mark.parametrize("value", [30000.0, 40000.0])
def test_the_largest_half_precision_products(value):
    """d = 8, a row and a word all of one large number: the logit is the loss' lse."""
    x = torch.full((3, 8), value, dtype=FP, device=DEV)
    w = torch.zeros(50, 8, dtype=FP, device=DEV)
    w[7] = value
    t = torch.tensor([7, 3, -100], device=DEV)
    v = float(x[0, 0])
    loss, lse, _ = sdc.sdc_cross_entropy(x, w, t)
    z = 8 * v * v
    assert (lse.double() - z).abs().max().item() <= 9 * U * z
    # 30000^2 = 1875^2 2^8 has 22 bits, five times that 25: sums of these products
    # round, each by at most 7 u z, so lse and the target's logit may differ by twice that
    assert abs(loss[0].item()) <= 15 * U * z and abs(loss[1].item() - z) <= 10 * U * z and loss[2].item() == 0
    dx, dw = sdc.sdc_cross_entropy_grad(x, w, t, lse, torch.ones(1, device=DEV))
    assert not dx[0].any() and not dx[2].any() and torch.equal(dx[1], w[7])
    want = torch.zeros_like(w)
    want[7], want[3] = x[0], -x[0]
    assert torch.equal(dw, want)


def test_neighbouring_logits_of_a_million():
    """Sixteen words share the largest logit, 1e6, exactly: the sum of exponentials is 16.
    lse is held in fp32, half a step of 2^-4 there, so that is what p is off by."""
    x = torch.zeros(40, 8, dtype=BF, device=DEV)
    w = torch.zeros(300, 8, dtype=BF, device=DEV)
    x[:, 0], w[:, 0] = 1000.0, -1000.0
    w[16:32, 0] = 1000.0
    t = torch.full((40,), 17, dtype=torch.int64, device=DEV)
    _, lse, _ = sdc.sdc_cross_entropy(x, w, t)
    want = 1e6 + torch.log(torch.tensor(16.0, dtype=torch.float64)).item()
    # ln 16 to a few u, then the rounding of the sum
    assert (lse.double() - want).abs().max().item() <= U * want + 1e-5


SHAPES = [(5, 301), (70, 700), (400, 25011), (2000, 8000)]   # a tile of 32, 64, 128 and 256 tokens


@pytest.mark.parametrize("n, v", SHAPES)
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_a_sure_row_loses_nothing(n, v, dtype):
    """Rows of d = 3001 random elements whose target's logit is about 40, the others' about
    +-1: the loss, below v exp(-35), is 0 in fp32.  It is taken from the logit that is in
    the sum: one summed in another order would be off by some u 40 either way."""
    d = 3001
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.empty(n, d, device=DEV).normal_(0, 1, generator=g).to(dtype)
    w = torch.empty(v, d, device=DEV).normal_(0, d ** -0.5, generator=g).to(dtype)
    t = torch.randperm(v, device=DEV, generator=g)[:min(n, v // 4)]
    t = t.repeat(-(-n // len(t)))[:n]
    first = torch.arange(len(t.unique()), device=DEV)        # rows that share a word share their x
    for k in range(0, n, len(first)):
        x[k:k + len(first)] = x[first][:min(len(first), n - k)]
    w[t[first]] = (x[first].double() * (40 / x[first].double().square().sum(1, keepdim=True))).to(dtype)
    z = x.double() @ w.double().t()
    want = torch.nn.functional.cross_entropy(z, t, reduction="none")
    assert want.max().item() < 1e-11
    loss, lse, total = sdc.sdc_cross_entropy(x, w, t)
    assert not loss.any() and total.item() == 0, (loss.min(), loss.max())
    top = z.amax(1)
    assert ((lse.double() - top).abs() <= (d + 8) * U * (x.double().abs() @ w.double().abs().t()).amax(1)).all()


@pytest.mark.parametrize("n", [1, 33, 500])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_a_vocabulary_of_one(n, dtype):
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.empty(n, 777, device=DEV).normal_(0, 3, generator=g).to(dtype)
    w = torch.empty(1, 777, device=DEV).normal_(0, 3, generator=g).to(dtype)
    t = torch.zeros(n, dtype=torch.int64, device=DEV)
    loss, lse, total = sdc.sdc_cross_entropy(x, w, t)
    assert not loss.any() and total.item() == 0
    dx, dw = sdc.sdc_cross_entropy_grad(x, w, t, lse, torch.ones(1, device=DEV))
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("n, v", SHAPES)
def test_equal_logits_of_a_million(n, v):
    """All logits 1e6, exactly: the loss is ln v although lse, in fp32, has steps of 1/16."""
    x = torch.zeros(n, 8, dtype=BF, device=DEV)
    w = torch.zeros(v, 8, dtype=BF, device=DEV)
    x[:, 0], w[:, 0] = 1000.0, 1000.0
    t = torch.arange(n, device=DEV) * 7 % v
    loss, _, _ = sdc.sdc_cross_entropy(x, w, t)
    want = torch.log(torch.tensor(float(v), dtype=torch.float64)).item()
    # a sum of ones below 2^24 is exact; the logarithm and its factor, 4 u
    assert (loss.double() - want).abs().max().item() <= 4 * U * want


def test_losses_are_never_below_zero():
    """Random rows of large width, half of them nearly sure of their target."""
    n, d, v = 300, 4097, 2000
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty(n, d, device=DEV).normal_(0, 1, generator=g).to(BF)
    w = torch.empty(v, d, device=DEV).normal_(0, 0.01, generator=g).to(BF)
    t = torch.randperm(v, device=DEV, generator=g)[:n]
    for k in range(0, n, 2):
        w[t[k]] = (x[k].double() * ((10 + k / 5) / x[k].double().square().sum())).to(BF)
    z = x.double() @ w.double().t()
    want = torch.nn.functional.cross_entropy(z, t, reduction="none")
    loss, _, _ = sdc.sdc_cross_entropy(x, w, t)
    assert (loss >= 0).all()
    # each logit is off by ez, the exponentials' relative error is twice that and 2 u,
    # 11 levels of sums (2000 words) and the logarithm near 1: 16 u
    ez = ((d + 8) * U * (x.double().abs() @ w.double().abs().t())).amax(1)
    assert ((loss.double() - want).abs() <= 2 * ez * (-torch.expm1(-want)).clamp(min=0) * 1.01 + 2 * ez * ez
            + 16 * U * (1 + want)).all()
