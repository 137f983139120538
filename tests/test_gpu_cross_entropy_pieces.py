"""GPU tests of the linear head's gradient where the vocabulary is cut into pieces:
dz of the whole vocabulary would take more than the 256 MiB that one piece may.

Every way that rows may lie (aligned, off 16-byte boundaries, copied as they are
shorter than a load), every shape of tile that can have pieces, dx added up over
pieces in vectors and element by element; and the logits' row, whose parts the
pieces leave one behind the other, against the forward pass', which has one
piece, and against a scan of the logits in memory.
"""
import pytest
import torch

import silent_corruption_detection_amd as sdc
from _util import say
from test_gpu_cross_entropy import check, make

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16
PIECE = 256 << 20


def pieces_at_least_two(x, w, t):
    """The workspace is smaller than dz of the whole vocabulary alone."""
    n, v = x.shape[0], w.shape[0]
    assert 2 * n * v > PIECE
    assert sdc.sdc_cross_entropy_ws_bytes(x, w, t)[1] < 2 * n * v


def placed(t, pad, off):
    """t with rows `pad` elements apart, the first `off` elements into its buffer."""
    n, d = t.shape
    b = torch.full((n * (d + pad) + off + 8,), float("nan"), dtype=t.dtype, device=DEV)
    return b[off:off + n * (d + pad)].view(n, d + pad)[:, :d].copy_(t)


CASES = [
    # tiles of 256 tokens
    (16000, 64, 13001, 0, 0), (16000, 65, 13001, 2, 3), (16000, 66, 13001, 0, 1), (16000, 5, 13001, 3, 1),
    # of 32: 128 words a tile
    (32, 8, 4_400_003, 0, 0), (31, 9, 4_700_001, 0, 1), (20, 5, 6_800_003, 0, 0)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("n, d, v, pad, off", CASES)
def test_the_formulas(n, d, v, pad, off, dtype):
    say(f"case pieces n={n} d={d} v={v} pad={pad} off={off} {dtype}")
    x, w, t = make(n, d, v, dtype, seed=d, ignored=0.1 if n > 100 else 0.0)
    x, w = placed(x, pad, off), placed(w, pad, off)
    pieces_at_least_two(x, w, t)
    # losses of some words need targets in the last piece too
    t[0], t[1] = v - 1, 0
    check(x, w, t, g=1.0 / n)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("n, d, v, pad, off", CASES)
def test_the_logits_row(n, d, v, pad, off, dtype):
    """Small whole numbers make every logit exact, so its row is that of the logits in memory."""
    say(f"case pieces row n={n} d={d} v={v} pad={pad} off={off} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(d)
    x = placed(torch.randint(-4, 5, (n, d), device=DEV, generator=g).to(dtype), pad, off)
    w = placed(torch.randint(-4, 5, (v, d), device=DEV, generator=g).to(dtype), pad, off)
    t = torch.randint(0, v, (n,), device=DEV, generator=g)
    pieces_at_least_two(x, w, t)
    want = sdc.sdc_fingerprint([x.float() @ w.float().t()])
    row, again = (torch.empty((1, 4), dtype=torch.int64, device=DEV) for _ in range(2))
    mis = torch.zeros(1, dtype=torch.int32, device=DEV)
    one = torch.ones(1, device=DEV)
    _, lse, _ = sdc.sdc_cross_entropy(x, w, t, row=row)
    dx, dw = sdc.sdc_cross_entropy_grad(x, w, t, lse, one, row=again, ref=row, mismatch=mis)
    assert torch.equal(row, want) and torch.equal(again, want) and mis.item() == 0
    alone = sdc.sdc_cross_entropy_grad(x, w, t, lse, one)
    assert torch.equal(dx, alone[0]) and torch.equal(dw, alone[1])
    for at in (v - 1, 0):   # a weight of the last piece, then one of the first too
        w[at, d - 1] += 1
        x[n - 1, d - 1] = 1
        sdc.sdc_cross_entropy_grad(x, w, t, lse, one, row=again, ref=row, mismatch=mis)
        assert torch.equal(again, sdc.sdc_fingerprint([x.float() @ w.float().t()]))
    assert mis.item() == 2


@pytest.mark.parametrize("need", [(True, False), (False, True)], ids=["dx", "dw"])
def test_one_of_the_two(need):
    x, w, t = make(16000, 30, 13001, BF, seed=3, ignored=0.1)
    pieces_at_least_two(x, w, t)
    _, lse, _ = sdc.sdc_cross_entropy(x, w, t)
    one = torch.ones(1, device=DEV)
    both = sdc.sdc_cross_entropy_grad(x, w, t, lse, one)
    got = sdc.sdc_cross_entropy_grad(x, w, t, lse, one, need_dx=need[0], need_dw=need[1])
    for a, b, wanted in zip(got, both, need):
        assert torch.equal(a, b) if wanted else a is None
