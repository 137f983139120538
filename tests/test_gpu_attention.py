"""GPU tests of softmax attention and its gradient against the formulas in 64 bits.

Tolerances (u = 2^-24, h = half a step of the 16-bit type, eps / 2):
- a score, d products summed in fp32 in some order: (d + 8) u A with A the sum of the
  products' magnitudes; scaled, and u for the scaling;
- a probability relative to its row: twice the row's largest error of a scaled score,
  the exponent's rounding (4 u |z|), the exponential, up to lk additions of the row's sum
  and up to lk / 64 rescalings (u (2 lk + 40)); lse the same and 2 u |lse|;
- out: the probabilities' errors and their rounding (h; in fp16 at least half a subnormal
  step, 2^-25 of the largest), through the product with |v|, lk u of it for the
  additions, and h of the result;
- the gradient takes out and lse as they are: p is off by the score's and lse's errors,
  delta by out's rounding, dz = p (dp - delta) by those of its factors and h of itself (fp16
  holds dz 2^e times as large with 2^e above 2^13 / B, B twice the largest norms'
  product, so a subnormal step is B 2^-37 at most, and p 2^14 times: 2^-38); dq, dk,
  dv: those through the products, the additions, and h of the result.
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


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make(b, lq, lk, hq, hk, d, dtype, seed=1, scale=1.0):
    g = gen(seed)
    r = lambda *s: torch.empty(s, device=DEV).normal_(0, 1, generator=g)  # noqa: E731
    return ((r(b, lq, hq, d) * scale).to(dtype), (r(b, lk, hk, d) * scale).to(dtype), r(b, lk, hk, d).to(dtype),
            r(b, lq, hq, d).to(dtype))


def attended(lq, lk, causal, window):
    i = torch.arange(lq, device=DEV)[:, None] + lk - lq
    j = torch.arange(lk, device=DEV)[None, :]
    ok = torch.ones(lq, lk, dtype=torch.bool, device=DEV)
    if causal:
        ok = j <= i
        if window:
            ok = ok & (j > i - window)
    return ok


def exact(q, k, v, do, causal, window, scale, out=None, lse=None):
    """One sequence ([rows, heads, d]): {name: (value, tolerance)} of the forward pass, or,
    with its out and lse, of the gradient."""
    lq, hq, d = q.shape
    lk, hk = k.shape[:2]
    G, h = hq // hk, torch.finfo(q.dtype).eps / 2
    half, sub = q.dtype == FP, 2.0 ** -25
    ok = attended(lq, lk, causal, window)
    Q = q.double().transpose(0, 1)
    K, V = (t.double().transpose(0, 1).repeat_interleave(G, 0) for t in (k, v))
    s, A = Q @ K.transpose(1, 2), Q.abs() @ K.abs().transpose(1, 2)
    z = (s * scale).masked_fill(~ok, -math.inf)
    zmax = (z.abs().masked_fill(~ok, 0)).amax(2) if lk else torch.zeros(hq, lq, device=DEV, dtype=torch.float64)
    es = (((d + 8) * U * A * scale + U * (s * scale).abs()) * ok)
    esmax = es.amax(2) if lk else torch.zeros_like(zmax)
    exact_lse = torch.logsumexp(z, 2) if lk else torch.full((hq, lq), -math.inf, device=DEV, dtype=torch.float64)
    empty = exact_lse == -math.inf
    back = lambda t: t.transpose(0, 1)  # noqa: E731
    if out is None:
        p = torch.where(ok, (z - exact_lse.masked_fill(empty, 0)[..., None]).exp(), 0.0)
        ep = 2 * esmax + U * (4 * zmax + 2 * lk + 40)
        o = p @ V
        mag = p @ V.abs()
        tol = mag * (2 * ep[..., None] + h * 1.01 + lk * U) + h * 1.01 * o.abs() + 1e-30
        if half:
            tol = tol + sub * (ok.double() @ V.abs()) + sub
        tl = (ep + 2 * U * exact_lse.abs()).masked_fill(empty, 0.0)
        return {"out": (back(o), back(tol)), "lse": (back(exact_lse), back(tl))}
    DO, O = do.double().transpose(0, 1), out.double().transpose(0, 1)
    L = lse.double().transpose(0, 1)
    p = torch.where(ok, (z - L.masked_fill(empty, 0)[..., None]).exp(), 0.0)
    ep = es + U * (4 * zmax + 4 * L.masked_fill(empty, 0).abs() + 16)[..., None]
    dp, Adp = DO @ V.transpose(1, 2), DO.abs() @ V.abs().transpose(1, 2)
    delta = (DO * O).sum(2, keepdim=True)
    diff = dp - delta
    dz = p * diff
    ediff = (d + 8) * U * (Adp + (DO * O).abs().sum(2, keepdim=True)) + U * diff.abs()
    B = 2 * (DO.norm(dim=2).amax() * V.norm(dim=2).amax()).item() if lq and lk else 0.0
    edz = (p * ediff + dz.abs() * (ep + 4 * U) + dz.abs() * h * 1.01 + (B * 2.0 ** -37 if half else 0)) * ok
    epv = (p * (ep + h * 1.01) + (2.0 ** -38 if half else 0)) * ok
    fold = lambda t: t.reshape(hk, G, *t.shape[1:]).sum(1)  # noqa: E731
    n = lq * G
    done = {}
    for name, w, ew, m, terms, by_key in (("dv", p, epv, DO, n, True), ("dk", dz * scale, edz * scale, Q, n, True),
                                          ("dq", dz * scale, edz * scale, K, lk, False)):
        if by_key:
            w, ew = w.transpose(1, 2), ew.transpose(1, 2)
        x, tol = w @ m, (ew + (terms + 64) * U * w.abs()) @ m.abs()
        if by_key:
            x, tol = fold(x), fold(tol)
        done[name] = (back(x), back(tol + 1.01 * h * x.abs() + (sub if half else 0) + 1e-30))
    return done


def close(got, want, tol, what):
    got = got.double()
    same = (got == want) | ((got - want).abs() <= tol * 1.001)
    bad = ~same
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist(),
                           tol.expand_as(got)[bad][:4].tolist())


def check(q, k, v, do, causal=False, window=0, scale=None, seq=None, **kw):
    """Both passes of a batch (or of packed sequences: seq, lists of offsets) against exact()."""
    how = dict(causal=causal, window=window, scale=scale)
    if seq is not None:
        how.update(seq_q=torch.tensor(seq[0], dtype=torch.int32, device=DEV),
                   seq_k=torch.tensor(seq[1], dtype=torch.int32, device=DEV))
    out, lse = sdc.sdc_attention(q, k, v, **how, **kw)
    torch.cuda.synchronize()
    dq, dk, dv = sdc.sdc_attention_grad(q, k, v, out, lse, do, **how)
    torch.cuda.synchronize()
    sc = q.shape[-1] ** -0.5 if scale is None else scale
    if seq is None:
        parts = [((b,), (b,)) for b in range(q.shape[0])]
    else:
        parts = [(slice(*seq[0][i:i + 2]), slice(*seq[1][i:i + 2])) for i in range(len(seq[0]) - 1)]
    for iq, ik in parts:
        iq, ik = (iq[0] if isinstance(iq, tuple) else iq), (ik[0] if isinstance(ik, tuple) else ik)
        a = (q[iq], k[ik], v[ik], do[iq], causal, window, sc)
        for name, (x, tol) in exact(*a).items():
            close({"out": out, "lse": lse}[name][iq], x, tol, (name, iq))
        for name, (x, tol) in exact(*a, out[iq], lse[iq]).items():
            close({"dq": dq, "dk": dk, "dv": dv}[name][iq if name == "dq" else ik], x, tol, (name, iq))
    return out, lse, dq, dk, dv


SIZES = [  # batch, queries, keys, heads of each, d, causal, window
    (1, 1, 1, 1, 1, 8, False, 0), (1, 1, 1, 1, 1, 128, True, 0), (2, 1, 63, 1, 1, 64, False, 0),
    (1, 2, 64, 2, 1, 72, True, 0), (3, 31, 65, 3, 1, 80, True, 0), (1, 33, 32, 4, 4, 96, False, 0),
    (2, 64, 64, 2, 2, 64, True, 0), (1, 65, 65, 5, 1, 128, True, 0), (1, 127, 129, 2, 1, 104, True, 0),
    (1, 128, 128, 1, 1, 128, True, 0), (2, 130, 257, 6, 2, 40, True, 0), (1, 257, 130, 7, 1, 24, False, 0),
    (1, 300, 300, 2, 2, 128, True, 1), (1, 300, 300, 4, 2, 64, True, 64), (1, 200, 500, 3, 3, 16, True, 77),
    (1, 500, 333, 2, 1, 120, True, 1000), (1, 1, 5000, 8, 1, 128, True, 0), (2, 3, 3001, 4, 2, 64, True, 100),
    (1, 2, 2500, 24, 1, 96, False, 0), (1, 3000, 40, 2, 1, 64, False, 0), (1, 1100, 1100, 2, 1, 128, True, 0),
    (33, 5, 7, 2, 1, 32, True, 0), (1, 40, 700, 1, 1, 128, True, 0)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("b, lq, lk, hq, hk, d, causal, window", SIZES)
def test_sizes(b, lq, lk, hq, hk, d, causal, window, dtype):
    say(f"case attention {b} {lq} {lk} {hq} {hk} {d} {causal} {window} {dtype}")
    check(*make(b, lq, lk, hq, hk, d, dtype, seed=lq + lk + d), causal, window)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_queries_without_keys(dtype):
    """More queries than keys under the causal mask: the first attend nothing."""
    q, k, v, do = make(2, 150, 70, 4, 2, 64, dtype, seed=3)
    out, lse, dq, *_ = check(q, k, v, do, True)
    assert (out[:, :80] == 0).all() and (lse[:, :80] == -math.inf).all() and (dq[:, :80] == 0).all()
    q, k, v, do = make(2, 9, 0, 4, 2, 64, dtype, seed=4)
    out, lse, dq, dk, dv = check(q, k, v, do)
    assert (out == 0).all() and (lse == -math.inf).all() and (dq == 0).all() and dk.numel() == 0
    q, k, v, do = make(2, 0, 9, 4, 2, 64, dtype, seed=5)
    out, lse, dq, dk, dv = check(q, k, v, do)
    assert (dk == 0).all() and (dv == 0).all() and out.numel() == 0
    q, k, v, do = make(0, 5, 9, 4, 2, 64, dtype, seed=5)
    check(q, k, v, do)


@pytest.mark.parametrize("scale", [0.02, 3.0, 400.0, 1e9])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_scores_of_any_size(scale, dtype):
    """From nearly equal probabilities to scores of 10^10, where one key has them all; the
    formulas' own bounds say what fp32 scores can give there.  Beyond |lse| of 10^4 lse's
    last bit is a whole exponent, and only the forward pass is checked."""
    q, k, v, do = make(1, 70, 190, 2, 1, 64, dtype, seed=6)
    out, lse = sdc.sdc_attention(q, k, v, scale=scale)
    torch.cuda.synchronize()
    assert out.isfinite().all() and lse.isfinite().all()
    if scale < 1e3:
        check(q, k, v, do, scale=scale)
    else:
        # whole numbers: the scores are exact, and each row's largest is far above the others
        g = gen(7)
        q, k = (torch.randint(-8, 9, t.shape, device=DEV, generator=g).to(dtype) for t in (q, k))
        out, lse = sdc.sdc_attention(q, k, v, scale=scale)
        s = (q[0].double().transpose(0, 1) @ k[0, :, 0].double().t())
        top = s.amax(2)
        p = (s == top[..., None]).double()
        want = ((p / p.sum(2, keepdim=True)) @ v[0, :, 0].double()).transpose(0, 1)
        close(out[0], want, 4 * torch.finfo(dtype).eps * torch.ones_like(want) * v.abs().max().double(), "out")
        close(lse[0], top.t() * scale, 4 * U * (top.t() * scale).abs() + 2, "lse")


PACKED = [([0, 1, 1, 64, 65, 200], None), ([0, 130, 131, 400], [0, 20, 300, 300]), ([5, 9, 40], [0, 65, 129]),
          ([0, 0, 0], [0, 3, 70]), (list(range(0, 700, 7)), None), ([0, 333], [0, 50])]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("causal, window", [(False, 0), (True, 0), (True, 17)])
@pytest.mark.parametrize("n", range(len(PACKED)))
def test_packed_sequences(n, causal, window, dtype):
    """Sequences of zero, one and more rows, of different lengths on both sides; rows of
    none are neither read (they hold NaN) nor, in given outputs, written."""
    sq, sk = PACKED[n]
    sk = sq if sk is None else sk
    say(f"case packed {n} {causal} {window} {dtype}")
    hq, hk, d = ((6, 2, 72), (3, 3, 128), (4, 1, 64))[n % 3]
    q, k, v, do = (t[0] for t in make(1, sq[-1] + 9, sk[-1] + 5, hq, hk, d, dtype, seed=n))
    for t, s in ((q, sq), (k, sk), (v, sk), (do, sq)):
        t[:s[0]] = math.nan
        t[s[-1]:] = math.nan
    out, lse, dq, dk, dv = check(q, k, v, do, causal, window, seq=(sq, sk))
    for t, s in ((out, sq), (lse, sq), (dq, sq), (dk, sk), (dv, sk)):
        assert (t[:s[0]] == 0).all() and (t[s[-1]:] == 0).all()
    how = dict(causal=causal, window=window, seq_q=torch.tensor(sq, dtype=torch.int32, device=DEV),
               seq_k=torch.tensor(sk, dtype=torch.int32, device=DEV))
    given = [torch.full_like(t, 7.0) for t in (out, lse, dq, dk, dv)]
    sdc.sdc_attention(q, k, v, out=given[0], lse=given[1], **how)
    sdc.sdc_attention_grad(q, k, v, out, lse, do, dq=given[2], dk=given[3], dv=given[4], **how)
    torch.cuda.synchronize()
    for t, g, s in zip((out, lse, dq, dk, dv), given, (sq, sq, sq, sk, sk)):
        assert torch.equal(t[s[0]:s[-1]], g[s[0]:s[-1]])
        assert (g[:s[0]] == 7).all() and (g[s[-1]:] == 7).all()


def test_few_packed_queries_split_over_keys():
    sk = [0, 3000, 3001, 9000]
    q, k, v, do = (t[0] for t in make(1, 7, 9000, 4, 2, 128, BF, seed=11))
    check(q, k, v, do, True, seq=([0, 3, 4, 7], sk))
    out, lse = sdc.sdc_attention(q, k, v, seq_q=torch.tensor([1, 3, 4, 6], dtype=torch.int32, device=DEV),
                                 seq_k=torch.tensor(sk, dtype=torch.int32, device=DEV),
                                 out=torch.full_like(q, 7.0), lse=torch.full((7, 4), 7.0, device=DEV))
    assert (out[0] == 7).all() and (out[6] == 7).all() and (lse[0] == 7).all() and (out[1:6] != 7).any()


def test_offsets_outside_the_rows_count_as_the_nearest_inside():
    q, k, v, _ = (t[0] for t in make(1, 90, 90, 2, 1, 64, BF, seed=12))
    seq = lambda *s: torch.tensor(s, dtype=torch.int32, device=DEV)  # noqa: E731
    a = sdc.sdc_attention(q, k, v, True, seq_q=seq(-5, 40, 1 << 30), seq_k=seq(-5, 40, 1 << 30))
    b = sdc.sdc_attention(q, k, v, True, seq_q=seq(0, 40, 90), seq_k=seq(0, 40, 90))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("hold", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("lq, window", [(300, 0), (300, 50), (2, 0)])
def test_what_masked_places_hold_has_no_effect(hold, dtype, lq, window):
    """Infinities and NaN in keys, values and queries that a mask keeps apart from the rest:
    everything else is what it is without them.  (Not to the bit: a tile that holds them is
    multiplied pair by pair, which adds the same fp32 products in another order; the bounds
    hold for any order.)"""
    lk, at = 300, 150
    q, k, v, do = make(1, lq, lk, 4, 2, 128, dtype, seed=13)
    how = dict(causal=True, window=window)
    out, lse = sdc.sdc_attention(q, k, v, **how)
    clean = (q[0], k[0], v[0], do[0], True, window, 128 ** -0.5)
    want = {**exact(*clean), **exact(*clean, out[0], lse[0])}

    def near(got, name, rows):
        x, tol = want[name]
        close(got[0][rows], x[rows], tol[rows], name)
    for which in ("k", "v"):
        t = {"k": k, "v": v}[which].clone()
        t[:, at] = hold
        args = (t, v) if which == "k" else (k, t)
        got = sdc.sdc_attention(q, *args, **how)
        i = torch.arange(lq, device=DEV) + lk - lq     # queries that attend key `at`
        sees = (i >= at) & ((i < at + window) if window else torch.ones_like(i, dtype=torch.bool))
        near(got[0], "out", ~sees)
        near(got[1], "lse", ~sees)
        dq, dk, dv = sdc.sdc_attention_grad(q, *args, out, lse, do, **how)
        near(dq, "dq", ~sees)
    if lq != lk:
        return
    # a query's rows reach the keys it attends only
    for which in ("q", "do"):
        t = {"q": q, "do": do}[which].clone()
        t[:, at] = hold
        args = (t, do) if which == "q" else (q, t)
        dq, dk, dv = sdc.sdc_attention_grad(args[0], k, v, out, lse, args[1], **how)
        j = torch.arange(lk, device=DEV)
        seen = (j <= at) & ((j > at - window) if window else torch.ones_like(j, dtype=torch.bool))
        near(dk, "dk", ~seen)
        near(dv, "dv", ~seen)
        near(dq, "dq", torch.arange(lq, device=DEV) != at)


def test_what_attended_places_hold_is_not_lost():
    q, k, v, do = make(1, 200, 200, 2, 1, 64, BF, seed=14)
    v[0, 100, 0, 5] = math.nan
    v[0, 120, 0, 6] = math.inf
    out, lse = sdc.sdc_attention(q, k, v, True)
    assert out[0, 100:, :, 5].isnan().all() and out[0, 120:, :, 6].isinf().all() and lse.isfinite().all()
    assert out[0, :100].isfinite().all() and out[0, :, :, 7].isfinite().all()


def test_layouts():
    """One projection's output, heads before rows, rows off 16-byte boundaries, heads
    repeated without memory: the bits of contiguous tensors."""
    q, k, v, do = make(2, 150, 150, 4, 2, 64, BF, seed=15)
    want = sdc.sdc_attention(q, k, v, True)
    wants = sdc.sdc_attention_grad(q, k, v, *want, do, True)
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731

    def tried(q, k, v, do):
        got = sdc.sdc_attention(q, k, v, True)
        assert same(got, want) and same(sdc.sdc_attention_grad(q, k, v, *got, do, True), wants)

    tried(*torch.cat([q, k, v], 2).split((4, 2, 2), 2), do)
    tried(*(t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v, do)))
    odd = lambda t: torch.full((t.numel() + 3,), math.nan, dtype=BF, device=DEV)[3:].view(t.shape).copy_(t)  # noqa: E731
    tried(*(odd(t) for t in (q, k, v, do)))
    wide = lambda t: torch.full(t.shape[:-1] + (72,), math.nan, dtype=BF, device=DEV)[..., :64].copy_(t)  # noqa: E731
    tried(*(wide(t) for t in (q, k, v)), do)
    shared = lambda t: t[:, :, :1].expand(-1, -1, 2, -1)  # noqa: E731
    a = sdc.sdc_attention(q, shared(k), shared(v), True)
    b = sdc.sdc_attention(q, shared(k).contiguous(), shared(v).contiguous(), True)
    assert same(a, b)
    one = sdc.sdc_attention(q[:1, :1], k[:1, :1], v[:1, :1])  # one row: its strides mean nothing
    assert same(one, sdc.sdc_attention(*(t[:1, :1].contiguous() for t in (q, k, v))))


def scores(q, k, causal, window):
    """fp32 [rows, heads, keys] scores of whole-number inputs, zero where not attended."""
    G = q.shape[2] // k.shape[2]
    s = q.double().transpose(1, 2) @ k.double().repeat_interleave(G, 2).permute(0, 2, 3, 1)
    s = s.masked_fill(~attended(q.shape[1], k.shape[1], causal, window), 0.0)
    return s.transpose(1, 2).float().contiguous()


@pytest.mark.parametrize("b, lq, lk, hq, hk, d, causal, window", [
    (1, 1, 1, 1, 1, 8, False, 0), (2, 70, 70, 4, 2, 64, True, 0), (1, 200, 130, 3, 1, 96, True, 0),
    (1, 150, 300, 6, 3, 128, True, 40), (1, 1, 5000, 8, 2, 128, True, 0), (2, 600, 40, 2, 1, 80, False, 0)])
def test_rows_are_those_of_the_scores(b, lq, lk, hq, hk, d, causal, window):
    """Small whole numbers make every score exact, so the row is the scan's row of the
    scores in memory; both of the gradient's launches have it too."""
    g = gen(lq)
    q, k, v = (torch.randint(-4, 5, s, device=DEV, generator=g).to(BF) for s in ((b, lq, hq, d), (b, lk, hk, d), (b, lk, hk, d)))
    want = oracle_rows([scores(q, k, causal, window)])
    row, again = (torch.zeros((1, 4), dtype=torch.int64, device=DEV) for _ in range(2))
    mis = torch.zeros(1, dtype=torch.int32, device=DEV)
    how = dict(causal=causal, window=window)
    out, lse = sdc.sdc_attention(q, k, v, row=row, **how)
    torch.cuda.synchronize()
    assert_rows_equal(sdc.rows_numpy(row), want)
    do = torch.ones_like(q)
    for need in ((True, True), (True, False), (False, True)):
        again.zero_()
        sdc.sdc_attention_grad(q, k, v, out, lse, do, row=again, ref=row, mismatch=mis, need_dq=need[0], need_dkv=need[1],
                               **how)
        assert_rows_equal(sdc.rows_numpy(again), want)
    assert mis.item() == 0
    q[0, lq - 1, 0, 0] = 1
    k[0, 0 if not window else lk - 1, 0, 0] += 1    # a key changed between the passes
    sdc.sdc_attention_grad(q, k, v, out, lse, do, row=again, ref=row, mismatch=mis, **how)
    assert mis.item() == 2


def test_packed_rows_are_those_of_the_scores():
    g = gen(3)
    sq, sk = [0, 40, 41, 130], [0, 70, 170, 200]
    q, k, v = (torch.randint(-4, 5, s, device=DEV, generator=g).to(FP) for s in ((140, 6, 72), (210, 2, 72), (210, 2, 72)))
    want = torch.zeros(140, 6, 210, device=DEV)
    for i in range(3):
        a, c = slice(*sq[i:i + 2]), slice(*sk[i:i + 2])
        want[a, :, :sk[i + 1] - sk[i]] = scores(q[None, a], k[None, c], True, 0)[0]
    row, again = (torch.zeros((1, 4), dtype=torch.int64, device=DEV) for _ in range(2))
    mis = torch.zeros(1, dtype=torch.int32, device=DEV)
    how = dict(causal=True, seq_q=torch.tensor(sq, dtype=torch.int32, device=DEV),
               seq_k=torch.tensor(sk, dtype=torch.int32, device=DEV))
    out, lse = sdc.sdc_attention(q, k, v, row=row, **how)
    sdc.sdc_attention_grad(q, k, v, out, lse, q, row=again, ref=row, mismatch=mis, **how)
    assert_rows_equal(sdc.rows_numpy(row), oracle_rows([want]))
    assert torch.equal(row, again) and mis.item() == 0


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("b, lq, lk, hq, hk, d", [(2, 500, 500, 8, 2, 128), (1, 300, 700, 4, 4, 80), (3, 1, 2000, 16, 2, 64)])
def test_rows_agree_and_change_nothing_and_runs_repeat(b, lq, lk, hq, hk, d, dtype):
    """Scores of any values: the passes' rows agree bit for bit, results with and without
    rows too, and from run to run."""
    q, k, v, do = make(b, lq, lk, hq, hk, d, dtype, seed=16)
    want = sdc.sdc_attention(q, k, v, True)
    wants = sdc.sdc_attention_grad(q, k, v, *want, do, True)
    rows = torch.empty((2, 4), dtype=torch.int64, device=DEV)
    mis = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(3):
        got = sdc.sdc_attention(q, k, v, True, row=rows[:1])
        gots = sdc.sdc_attention_grad(q, k, v, *got, do, True, row=rows[1:], ref=rows[:1], mismatch=mis)
        for x, y in zip(want + wants, got + gots):
            assert torch.equal(x, y)
    assert mis.item() == 0 and torch.equal(rows[0], rows[1])


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_gradient_against_differences(dtype):
    """The directional derivative of sum(dout * out) from the 64-bit forward pass."""
    q, k, v, do = make(1, 40, 90, 4, 2, 64, dtype, seed=17)
    out, lse = sdc.sdc_attention(q, k, v, True)
    grads = sdc.sdc_attention_grad(q, k, v, out, lse, do, True)

    def loss(q, k, v):
        K, V = (t[0].transpose(0, 1).repeat_interleave(2, 0) for t in (k, v))
        z = (q[0].transpose(0, 1) @ K.transpose(1, 2) / 8).masked_fill(~attended(40, 90, True, 0), -math.inf)
        return ((torch.softmax(z, 2) @ V).transpose(0, 1) * do[0].double()).sum()
    g = gen(18)
    base = [t.double() for t in (q, k, v)]
    for i in range(3):
        step = torch.empty(base[i].shape, device=DEV, dtype=torch.float64).normal_(0, 1, generator=g)
        at = lambda e: loss(*[t + e * step if j == i else t for j, t in enumerate(base)])  # noqa: E731
        slope = (at(1e-5) - at(-1e-5)) / 2e-5
        got = (grads[i].double() * step).sum()
        # each gradient is off by its rounding, twice (its own and its factors'), in a sum of random signs
        assert (got - slope).abs() <= 8 * torch.finfo(dtype).eps * (grads[i].double() * step).norm() + 1e-6


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("size", [1e-6, 1e3])
def test_gradients_of_any_size(dtype, size):
    """dout's magnitude goes through as a factor; in fp16 down to its subnormals and up to
    its largest numbers."""
    q, k, v, do = make(1, 100, 100, 2, 1, 64, dtype, seed=19)
    check(q, k, v, (do.float() * size).to(dtype), True)


def test_outputs_workspace_and_another_stream():
    q, k, v, do = make(1, 300, 300, 4, 2, 64, FP, seed=20)
    want = sdc.sdc_attention(q, k, v, True)
    wants = sdc.sdc_attention_grad(q, k, v, *want, do, True)
    need = sdc.sdc_attention_ws_bytes(q, k, v, True)
    ws = [torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV) for n in need]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    given = [torch.empty_like(t) for t in want + wants]
    got = sdc.sdc_attention(q, k, v, True, out=given[0], lse=given[1], ws=ws[0], stream=side)
    gots = sdc.sdc_attention_grad(q, k, v, *got, do, True, dq=given[2], dk=given[3], dv=given[4], ws=ws[1], stream=side)
    fresh = sdc.sdc_attention(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, True, stream=side)
    side.synchronize()
    for x, y, z in zip(want + wants, got + gots, given):
        assert torch.equal(x, y) and y.data_ptr() == z.data_ptr()
    assert torch.equal(fresh[0], want[0])
    assert all((w[n:] == 0xFF).all() for w, n in zip(ws, need))


def test_graphs_share_nothing():
    """Two captured graphs replayed in turn with eager work between."""
    cases = [make(2, 200, 200, 4, 2, 128, BF, seed=21), make(1, 1, 3000, 8, 2, 64, FP, seed=22)]
    for q, k, v, do in cases:
        sdc.sdc_attention_grad(q, k, v, *sdc.sdc_attention(q, k, v, True), do, True)
    torch.cuda.synchronize()
    graphs = []
    for q, k, v, do in cases:
        g = torch.cuda.CUDAGraph()
        row = torch.zeros((1, 4), dtype=torch.int64, device=DEV)
        with torch.cuda.graph(g):
            got = sdc.sdc_attention(q, k, v, True, row=row)
            got = got + sdc.sdc_attention_grad(q, k, v, *got, do, True)
        graphs.append((g, got, row))
    for turn in range(3):
        for (q, k, v, do), (g, got, row) in zip(cases, graphs):
            q.copy_(q.roll(1, 1) if q.shape[1] > 1 else -q)
            g.replay()
            other = torch.empty((1, 4), dtype=torch.int64, device=DEV)
            want = sdc.sdc_attention(q, k, v, True, row=other)
            want = want + sdc.sdc_attention_grad(q, k, v, *want, do, True)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(want, got)) and torch.equal(row, other), turn


def test_long_cache_past_32_bit_offsets():
    """Keys whose byte offsets pass 2^32: rows of 64 KiB apart from each other in a buffer of 4.6 GiB."""
    n, step = 70_000, 32768
    buf = torch.zeros(n * step, dtype=BF, device=DEV)
    k, v = (buf.view(1, n, step)[:, :, at:at + 64].unsqueeze(2) for at in (0, 64))
    g = gen(23)
    k.copy_(torch.empty(1, n, 1, 64, device=DEV).normal_(0, 1, generator=g))
    v.copy_(torch.empty(1, n, 1, 64, device=DEV).normal_(0, 1, generator=g))
    q = torch.empty(1, 2, 4, 64, device=DEV).normal_(0, 1, generator=g).to(BF)
    got = sdc.sdc_attention(q, k, v, True)
    want = sdc.sdc_attention(q, k.contiguous(), v.contiguous(), True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


MANY = [  # single tokens and few queries of many sequences: one wave each, with and without splits
    (100, 1, 70, 8, 8, 128, True, 0), (8, 2, 3301, 16, 8, 128, True, 0), (32, 1, 1500, 16, 8, 64, False, 0),
    (100, 3, 400, 16, 8, 40, True, 90), (50, 5, 66, 32, 16, 96, True, 0), (100, 1, 1, 8, 8, 72, True, 0)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("b, lq, lk, hq, hk, d, causal, window", MANY)
def test_few_queries_of_many_sequences(b, lq, lk, hq, hk, d, causal, window, dtype):
    say(f"case many {b} {lq} {lk} {hq} {hk} {d} {causal} {window} {dtype}")
    q, k, v, do = make(b, lq, lk, hq, hk, d, dtype, seed=b + lk + d)
    out, lse, dq, *_ = check(q, k, v, do, causal, window)
    rows = torch.zeros(2, 4, dtype=torch.int64, device=DEV)
    again = sdc.sdc_attention(q, k, v, causal, window, row=rows[0])
    grads = sdc.sdc_attention_grad(q, k, v, out, lse, do, causal, window, row=rows[1])
    torch.cuda.synchronize()
    assert torch.equal(again[0], out) and torch.equal(again[1], lse) and torch.equal(grads[0], dq)
    assert torch.equal(rows[0], rows[1])


def test_few_queries_of_many_packed_sequences():
    lengths = torch.randint(0, 4, (450,), generator=torch.Generator().manual_seed(21)).tolist()
    keys = torch.randint(0, 90, (450,), generator=torch.Generator().manual_seed(22)).tolist()
    sq, sk = [0], [0]
    for a, b in zip(lengths, keys):
        sq.append(sq[-1] + a)
        sk.append(sk[-1] + b)
    q, k, v, do = (t[0] for t in make(1, sq[-1], sk[-1], 4, 2, 128, BF, seed=23))
    check(q, k, v, do, True, seq=(sq, sk))


@pytest.mark.parametrize("hold", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("b, lk", [(100, 151), (8, 3301)])
def test_masked_places_of_few_queries_of_many_sequences(hold, b, lk):
    """The last key is attended by the last query only: the first's results are those without it."""
    q, k, v, do = make(b, 2, lk, 16, 8, 128, BF, seed=24)
    k2, v2 = k.clone(), v.clone()
    k2[:, -1], v2[:, -1] = hold, hold
    out, lse = sdc.sdc_attention(q, k2, v2, True)
    torch.cuda.synchronize()
    for i in range(b):
        for name, (x, tol) in exact(q[i], k[i], v[i], do[i], True, 0, 128 ** -0.5).items():
            close({"out": out, "lse": lse}[name][i][:1], x[:1], tol[:1], (name, i))
