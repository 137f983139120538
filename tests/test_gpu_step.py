"""GPU tests of the loss, the audits and the optimizer step together, as a
training step uses them: a checkpointed bf16 model with a linear head over a
vocabulary, three replicas that must stay bit-identical.

- linear_cross_entropy's gradients equal the library call's and, within 16-bit
  rounding, autograd's in 64 bits.
- The audit counts a flipped bit in what the head's recomputation reads, and
  nothing on a clean step.
- The step takes its gate and clip from the squared norms of the gradients, its
  rows are the weights' fingerprints, replicas agree, a replay gives the same
  bits, a NaN gradient takes no step, a flip after the step names its replica.
"""
import pytest
import torch
import torch.utils.checkpoint as cp

import silent_corruption_detection_amd as sdc
from silent_corruption_detection_amd.loss import linear_cross_entropy
from silent_corruption_detection_amd.recompute import RecomputeAudit
import workloads as W
from _util import assert_rows_equal, oracle_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
D, V, TOKENS, BLOCKS = 96, 1003, 70, 2


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def batch(seed):
    g = gen(seed)
    ids = torch.randint(0, V, (2, TOKENS), device=DEV, generator=g)
    target = torch.randint(0, V, (2, TOKENS), device=DEV, generator=g)
    target[0, :5] = -100
    return ids, target


class Replica:
    """Embedding (also the head), residual blocks with a LayerNorm each."""

    def __init__(self, seed, state=8):
        g = gen(seed)
        r = lambda *s, std=0.05: torch.empty(s, device=DEV).normal_(0, std, generator=g).to(BF)  # noqa: E731
        self.params = [r(V, D)]
        for _ in range(BLOCKS):
            self.params += [torch.ones(D, device=DEV, dtype=BF), torch.zeros(D, device=DEV, dtype=BF), r(D, D), r(D)]
        for p in self.params:
            p.requires_grad_()
            p.grad = torch.zeros_like(p)
        P = [p.detach() for p in self.params]
        self.master = [p.float() for p in P]
        if state == 8:
            z = lambda p: torch.zeros(p.numel(), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # noqa: E731
            s = lambda: [torch.zeros(-(-p.numel() // 128), dtype=torch.uint8, device=DEV) for p in P]  # noqa: E731
            kw = dict(exp_avg_scale=s(), exp_avg_sq_scale=s())
        else:
            z = lambda p: torch.zeros(p.shape, device=DEV)  # noqa: E731
            kw = {}
        self.states = [z(p) for p in P], [z(p) for p in P]
        grads = [p.grad for p in self.params]
        self.plan = sdc.sdc_adamw_plan_build(P, grads, *self.states, master=self.master,
                                             group=[0 if p.dim() == 2 else 1 for p in P], n_groups=2, **kw)
        self.gplan = sdc.sdc_plan_build(grads)
        self.groups = torch.tensor([[3e-3, 0.9, 0.95, 1e-8, 0.1], [3e-3, 0.9, 0.95, 1e-8, 0.0]], dtype=torch.float64,
                                   device=DEV)
        self.control = sdc.sdc_adamw_control(DEV, seed=5)
        self.rows = torch.empty((len(P), 4), dtype=torch.int64, device=DEV)
        self.audit = RecomputeAudit(BLOCKS + 1, device=DEV)

    def block(self, i, h):
        a, b, w, c = self.params[1 + 4 * i:5 + 4 * i]
        return h + torch.nn.functional.gelu(torch.nn.functional.layer_norm(h, (D,), a, b) @ w.t() + c)

    def loss(self, ids, target):
        self.audit.begin_step()
        h = self.params[0][ids]
        for i in range(BLOCKS):
            h = cp.checkpoint(self.audit.wrap(lambda x, i=i: self.block(i, x), i), h, use_reentrant=True)
        return self.audit.cross_entropy(BLOCKS, h, self.params[0], target)

    def backward(self, ids, target):
        for p in self.params:
            p.grad.zero_()
        loss = self.loss(ids, target)
        loss.backward()
        return loss

    def step(self):
        _, total, flag = sdc.sdc_sqnorm(self.gplan)
        sdc.sdc_adamw_step(self.plan, self.groups, self.control, sq_total=total, flag=flag, max_norm=1.0,
                           rows=self.rows)

    def bits(self):
        return [t.detach().view(torch.uint8).clone() for t in self.params + self.master + self.states[0] + self.states[1]]


@pytest.mark.parametrize("reduction", ["mean", "sum"])
@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_autograd_of_the_loss(dtype, reduction):
    g = gen(1)
    x = torch.empty(2, 33, 72, device=DEV).normal_(0, 1, generator=g).to(dtype).requires_grad_()
    w = torch.empty(700, 72, device=DEV).normal_(0, 0.1, generator=g).to(dtype).requires_grad_()
    t = torch.randint(0, 700, (2, 33), device=DEV, generator=g)
    t[1, 3:9] = -100
    loss = linear_cross_entropy(x, w, t, reduction)
    (loss * 3.0).backward()
    xd, wd = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    ref = torch.nn.functional.cross_entropy((xd @ wd.t()).flatten(0, 1), t.flatten(), reduction=reduction)
    (ref * 3.0).backward()
    # fp32 sums of 72 products of size 1 and of 60 losses below 20
    assert abs(loss.item() - ref.item()) <= 2e-5 * abs(ref.item())
    _, lse, _ = sdc.sdc_cross_entropy(x.detach().flatten(0, 1), w.detach(), t.flatten())
    coef = torch.tensor([3.0 / 60 if reduction == "mean" else 3.0], device=DEV)
    dx, dw = sdc.sdc_cross_entropy_grad(x.detach().flatten(0, 1), w.detach(), t.flatten(), lse, coef)
    assert torch.equal(x.grad.flatten(0, 1), dx) and torch.equal(w.grad, dw)
    # dz and the result are rounded once each: 2 half steps of the sums' magnitudes
    h = torch.finfo(dtype).eps / 2
    z = (xd @ wd.t()).detach().flatten(0, 1)
    dz = torch.softmax(z, 1)
    hit = t.flatten().clamp(min=0)
    dz[torch.arange(66, device=DEV), hit] -= 1
    dz = (dz * (t.flatten() >= 0)[:, None]).abs() * coef.double()
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0
    tol = 2.05 * h * (dz @ wd.detach().abs()) + 2 ** -18 * coef.double() * 0.1 + tiny
    assert ((x.grad.flatten(0, 1).double() - xd.grad.flatten(0, 1)).abs() <= tol).all()
    tol = 2.05 * h * (dz.t() @ xd.detach().flatten(0, 1).abs()) + 2 ** -18 * coef.double() + tiny
    assert ((w.grad.double() - wd.grad).abs() <= tol).all()


def test_one_gradient_alone_and_no_targets():
    g = gen(2)
    x = torch.empty(20, 64, device=DEV).normal_(0, 1, generator=g).to(BF)
    w = torch.empty(300, 64, device=DEV).normal_(0, 0.1, generator=g).to(BF)
    t = torch.randint(0, 300, (20,), device=DEV, generator=g)
    both = [v.clone().requires_grad_() for v in (x, w)]
    linear_cross_entropy(*both, t).backward()
    a = x.clone().requires_grad_()
    linear_cross_entropy(a, w, t).backward()
    b = w.clone().requires_grad_()
    linear_cross_entropy(x, b, t).backward()
    assert torch.equal(a.grad, both[0].grad) and torch.equal(b.grad, both[1].grad)
    c = [v.clone().requires_grad_() for v in (x, w)]
    loss = linear_cross_entropy(*c, torch.full_like(t, -100))
    loss.backward()
    assert torch.isnan(loss) and not c[0].grad.any() and not c[1].grad.any()
    with pytest.raises(ValueError):
        linear_cross_entropy(x, w, t, "none")
    with pytest.raises(ValueError):
        linear_cross_entropy(x, w, t[:5])


def test_the_audit_covers_the_logits():
    r = Replica(3)
    ids, target = batch(3)
    r.backward(ids, target)
    res = r.audit.result()
    assert res["mismatched"] == [] and res["not_recomputed"] == [] and res["not_run"] == []
    orig, again = r.audit.rows()
    assert (orig[BLOCKS] == again[BLOCKS]).all() and orig[BLOCKS][0] != 0
    # a bit of the head's weights flips between the passes: the head alone is
    # reported if the blocks do not read it again
    for p in r.params:
        p.grad.zero_()
    loss = r.loss(ids, target)
    W.flip_bit(r.params[0].data, 777, 13)   # as memory would: autograd does not see it
    loss.backward()
    assert r.audit.result()["mismatched"] == [BLOCKS]
    # without a backward pass the segment is reported as not recomputed
    with torch.no_grad():
        r.loss(ids, target)
    assert BLOCKS in r.audit.result()["not_recomputed"]
    with pytest.raises(RuntimeError, match="begin_step"):
        r.audit.cross_entropy(BLOCKS, torch.zeros(1, D, device=DEV, dtype=BF), r.params[0],
                              torch.zeros(1, dtype=torch.int64, device=DEV))
    with pytest.raises(IndexError):
        r.audit.cross_entropy(BLOCKS + 1, torch.zeros(1, D, device=DEV, dtype=BF), r.params[0],
                              torch.zeros(1, dtype=torch.int64, device=DEV))


@pytest.mark.parametrize("state", [32, 8])
def test_replicas_step_together(state):
    reps = [Replica(4, state) for _ in range(3)]
    T = len(reps[0].params)
    for k in range(4):
        ids, target = batch(10 + k)
        losses = [r.backward(ids, target) for r in reps]
        for r in reps:
            assert r.audit.result()["mismatched"] == []
            r.step()
        # what Check 2 compares: the loss bits and the gradients' rows
        assert all(torch.equal(losses[0], l) for l in losses)
        grows = [sdc.rows_numpy(sdc.sdc_fingerprint_plan(r.gplan)) for r in reps]
        assert all((g == grows[0]).all() for g in grows)
        # what Check 3 compares: the rows that the step wrote are the weights'
        for r in reps:
            assert_rows_equal(sdc.rows_numpy(r.rows), oracle_rows([p.detach() for p in r.params]))
        table = torch.cat([r.rows for r in reps])
        assert not sdc.sdc_majority_compare(table, 3, T)["diverged"]
    assert [r.control.tolist()[:2] for r in reps] == [[4, 0]] * 3
    # a flip after the step: the rows taken from memory differ from those the step wrote
    W.flip_bit(reps[1].params[3], 4242, 9)
    now = [sdc.sdc_fingerprint([p.detach() for p in r.params]) for r in reps]
    d = sdc.sdc_fingerprint_diff(reps[1].rows, now[1])
    assert d["indices"] == [3] and d["hints"][0][:2] == (4242, 9)
    assert sdc.sdc_majority_compare(torch.cat(now), 3, T)["suspects"] == [1]


def test_a_nan_gradient_takes_no_step():
    r = Replica(5)
    ids, target = batch(20)
    r.backward(ids, target)
    before = r.bits()
    r.params[2].grad[3] = float("nan")
    r.step()
    assert all(torch.equal(a, b) for a, b in zip(before, r.bits()))
    assert r.control.tolist()[:2] == [0, 1]
    assert_rows_equal(sdc.rows_numpy(r.rows), oracle_rows([p.detach() for p in r.params]))
    r.backward(ids, target)
    r.step()
    assert r.control.tolist()[:2] == [1, 1]
    assert not all(torch.equal(a, b) for a, b in zip(before, r.bits()))
