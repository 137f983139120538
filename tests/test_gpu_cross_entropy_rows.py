"""GPU tests of the linear head's cross entropy for weights whose rows lie off
16-byte boundaries, at sizes of many workgroups and over repeated runs: bit for
bit what the same numbers give in aligned rows (padded with zeros, which change
no sum).
"""
import pytest
import torch

import silent_corruption_detection_amd as sdc
from _util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16


def padded(t):
    d = -(-t.shape[1] // 8) * 8
    out = torch.zeros(t.shape[0], d, dtype=t.dtype, device=DEV)
    out[:, :t.shape[1]] = t
    return out


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("n, d, v", [
    (400, 203, 25011), (2000, 331, 8000), (2000, 204, 8000), (1500, 71, 20001),   # tiles of 256 tokens
    (300, 205, 16001), (100, 202, 50304),                                         # of 128
    (70, 206, 3001), (100, 207, 8000),                                            # of 64
    (32, 201, 50304), (7, 999, 9001)])                                            # of 32
def test_rows_off_their_boundaries(n, d, v, dtype):
    say(f"case rows n={n} d={d} v={v} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(n + d)
    x = torch.empty(n, d, device=DEV).normal_(0, 1, generator=g).to(dtype)
    w = torch.empty(v, d, device=DEV).normal_(0, d ** -0.5, generator=g).to(dtype)
    t = torch.randint(-v // 5, v, (n,), device=DEV, generator=g)
    xa, wa = padded(x), padded(w)
    row = [torch.zeros(1, 4, dtype=torch.int64, device=DEV) for _ in range(3)]
    want = sdc.sdc_cross_entropy(xa, wa, t, row=row[0])
    one = torch.ones(1, device=DEV)
    dx, dw = sdc.sdc_cross_entropy_grad(xa, wa, t, want[1], one)
    want += dx[:, :d], dw[:, :d]
    for k in range(10):
        got = sdc.sdc_cross_entropy(x, w, t)
        got += sdc.sdc_cross_entropy_grad(x, w, t, got[1], one)
        for a, b, what in zip(got, want, ("loss", "lse", "total", "dx", "dw")):
            assert torch.equal(a, b), (what, k, (a != b).sum().item())
    sdc.sdc_cross_entropy(x, w, t, row=row[1])
    sdc.sdc_cross_entropy_grad(x, w, t, got[1], one, row=row[2])
    assert torch.equal(row[0], row[1]) and torch.equal(row[0], row[2])
