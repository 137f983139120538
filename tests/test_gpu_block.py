"""GPU tests of attention and the gated feed-forward block as a transformer block's
halves: the differentiable operators, their audits, a checkpointed model of such blocks
with the loss, the optimizer step and the checks around them, captured and not.

- block.attention's and block.gated_ffn's gradients equal the library calls'.
- The audits store and compare the rows of scores and projections, count a flipped bit
  in what the recomputation reads, and refuse a second backward pass.
- A step of a model of such blocks is reproducible to the bit and audited clean.
"""
import math

import pytest
import torch
import torch.nn.functional as F
import torch.utils.checkpoint as cp

import silent_corruption_detection_amd as sdc
from silent_corruption_detection_amd.block import attention, gated_ffn
from silent_corruption_detection_amd.recompute import RecomputeAudit

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def leaf(std, *shape, seed=1, dtype=BF):
    return torch.empty(shape, device=DEV).normal_(0, std, generator=gen(seed)).to(dtype).requires_grad_()


def test_attention_gives_the_calls_gradients():
    qkv = leaf(1.0, 2, 90, 8, 64)
    q, k, v = qkv.split((4, 2, 2), 2)
    out = attention(q, k, v, causal=True)
    g = leaf(1.0, 2, 4, 90, 64, seed=2).detach().transpose(1, 2)   # a gradient that is not contiguous
    out.backward(g)
    with torch.no_grad():
        want, lse = sdc.sdc_attention(q, k, v, True)
        dq, dk, dv = sdc.sdc_attention_grad(q, k, v, want, lse, g.contiguous(), True)
    assert torch.equal(out, want) and torch.equal(qkv.grad, torch.cat([dq, dk, dv], 2))


def test_gradients_of_shared_and_missing_inputs():
    """The same keys as values, heads that share one by expand, inputs without a gradient."""
    q, kv = leaf(1.0, 1, 70, 4, 64), leaf(1.0, 1, 70, 1, 64, seed=3)
    shared = kv.expand(-1, -1, 2, -1)
    attention(q, shared, shared, causal=True).sum().backward()
    with torch.no_grad():
        s = shared.contiguous()
        out, lse = sdc.sdc_attention(q, s, s, True)
        dq, dk, dv = sdc.sdc_attention_grad(q, s, s, out, lse, torch.ones_like(out), True)
    assert torch.equal(q.grad, dq)
    assert torch.allclose(kv.grad.float(), (dk.float() + dv.float()).sum(2, keepdim=True), rtol=2 ** -6, atol=2 ** -4)
    q.grad = kv.grad = None
    attention(q, shared.detach(), shared.detach(), causal=True).sum().backward()
    assert torch.equal(q.grad, dq)
    attention(q.detach(), kv, kv.detach()).sum().backward()
    assert kv.grad.isfinite().all()
    x, w = leaf(1.0, 3, 5, 64), leaf(0.1, 96, 64, seed=4)
    h = gated_ffn(x, w, w)                                     # one matrix for both projections
    h.sum().backward()
    dx, dg, du = sdc.sdc_gated_ffn_grad(x.detach().view(15, 64), w.detach(), w.detach(), torch.ones(15, 96, device=DEV, dtype=BF))
    assert torch.equal(x.grad, dx.view(3, 5, 64)) and torch.equal(w.grad, dg + du)
    x.grad = None
    gated_ffn(x, w.detach(), w.detach()).sum().backward()
    assert torch.equal(x.grad, dx.view(3, 5, 64))


def test_packed_padding_gets_zero_gradients():
    q, k, v = (leaf(1.0, 100, 2, 64, seed=s) for s in (1, 2, 3))
    seq = torch.tensor([10, 40, 81], dtype=torch.int32, device=DEV)
    out = attention(q, k, v, causal=True, seq_q=seq, seq_k=seq)
    out.sum().backward()
    for t in (out, q.grad, k.grad, v.grad):
        assert (t[:10] == 0).all() and (t[81:] == 0).all() and (t[10:81] != 0).any()


D, HEADS, KV, FF, V, L = 128, 4, 2, 328, 1003, 90
EPS = 1e-5
HEAD = D // HEADS


class Model:
    """Embedding (also the head), blocks of normalised attention and gated feed-forward."""

    def __init__(self, blocks=2, seed=1):
        g = gen(seed)
        r = lambda std, *s: torch.empty(s, device=DEV).normal_(0, std, generator=g).to(BF).requires_grad_()  # noqa: E731
        self.embed = r(0.5, V, D)
        self.blocks = [dict(qkv=r(D ** -0.5, (HEADS + 2 * KV) * HEAD, D), o=r(D ** -0.5, D, D), gate=r(D ** -0.5, FF, D),
                            up=r(D ** -0.5, FF, D), down=r(FF ** -0.5, D, FF)) for _ in range(blocks)]
        self.params = [self.embed] + [p for b in self.blocks for p in b.values()]
        for p in self.params:
            p.grad = torch.zeros_like(p)

    def loss(self, ids, target, audit=None):
        x = F.embedding(ids, self.embed)
        for k, b in enumerate(self.blocks):
            q, key, v = F.linear(F.rms_norm(x, (D,), eps=EPS), b["qkv"]).unflatten(-1, (HEADS + 2 * KV, HEAD)).split((HEADS, KV, KV), -2)
            a = attention(q, key, v, causal=True) if audit is None else audit.attention(2 * k, q, key, v, causal=True)
            x = x + F.linear(a.flatten(-2), b["o"])
            y = F.rms_norm(x, (D,), eps=EPS)
            h = gated_ffn(y, b["gate"], b["up"]) if audit is None else audit.gated_ffn(2 * k + 1, y, b["gate"], b["up"])
            x = x + F.linear(h, b["down"])
        if audit is None:
            from silent_corruption_detection_amd.loss import linear_cross_entropy
            return linear_cross_entropy(x, self.embed, target)
        return audit.cross_entropy(2 * len(self.blocks), x, self.embed, target)


def batch(seed):
    g = gen(seed)
    return tuple(torch.randint(0, V, (2, L), device=DEV, generator=g) for _ in range(2))


def test_a_step_is_audited_and_reproducible():
    ids, target = batch(5)
    grads, losses, rows = [], [], []
    for turn in range(2):
        m = Model()
        audit = RecomputeAudit(5, device=DEV)
        audit.begin_step()
        loss = m.loss(ids, target, audit)
        loss.backward()
        res = audit.result()
        assert res["mismatched"] == [] and res["not_recomputed"] == [] and res["not_run"] == []
        grads.append([p.grad.clone() for p in m.params])
        losses.append(loss.detach())
        rows.append(audit.rows()[0])
        # Check 1 and the step
        plan = sdc.sdc_plan_build([p.grad for p in m.params])
        _, total, flag = sdc.sdc_sqnorm(plan)
        assert flag.item() == 0 and math.isfinite(total.item()) and total.item() > 0
    assert torch.equal(losses[0], losses[1]) and (rows[0] == rows[1]).all()
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    m = Model()
    plain = m.loss(ids, target)
    plain.backward()
    assert torch.equal(plain, losses[0]) and all(torch.equal(p.grad, g) for p, g in zip(m.params, grads[0]))


def plain_loss(P, ids, target, cast):
    """The model (of one block) in torch operations; cast: what each operator's result is rounded to."""
    e, qkv, o, gate, up, down = P
    norm = lambda x: cast(x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt())  # noqa: E731
    x = e[ids]
    q, k, v = cast(norm(x) @ qkv.t()).unflatten(-1, (HEADS + 2 * KV, HEAD)).split((HEADS, KV, KV), -2)
    k, v = (t.repeat_interleave(HEADS // KV, 2).transpose(1, 2) for t in (k, v))
    z = q.transpose(1, 2) @ k.transpose(2, 3) / math.sqrt(HEAD)
    z = z.masked_fill(torch.ones(L, L, device=DEV).triu(1).bool(), -math.inf)
    x = cast(x + cast(cast((torch.softmax(z, -1) @ v).transpose(1, 2).flatten(-2)) @ o.t()))
    y = norm(x)
    x = cast(x + cast(cast(F.silu(y @ gate.t()) * (y @ up.t())) @ down.t()))
    return F.cross_entropy((x @ e.t()).flatten(0, 1), target.flatten())


class _Rounded(torch.autograd.Function):
    """To bf16 and back, of a value and of its gradient."""
    forward = staticmethod(lambda ctx, x: x.to(BF).to(x.dtype))
    backward = staticmethod(lambda ctx, g: g.to(BF).to(g.dtype))


def test_gradients_of_the_model():
    """Against autograd in 64 bits: as near as the same model of plain operations, computed in
    64 bits and rounded to bf16 between its operators, comes (which is what the activations' 16
    bits do to these gradients), and half as much again for the operators' own inner rounding."""
    ids, target = batch(6)
    m = Model(blocks=1, seed=2)
    m.loss(ids, target).backward()
    grads = []
    for cast in (lambda x: x, _Rounded.apply):
        P = [p.detach().double().requires_grad_() for p in m.params]
        grads.append(torch.autograd.grad(plain_loss(P, ids, target, cast), P))
    for i, (p, want, rounded) in enumerate(zip(m.params, *grads)):
        off, bound = (p.grad.double() - want).norm(), (rounded - want).norm()
        assert off <= 1.5 * bound + 2 ** -8 * want.norm(), i


def test_audits_count_what_changed_between_the_passes():
    q, k, v = (leaf(1.0, 2, 70, 2, 64, seed=s) for s in (1, 2, 3))
    x, wg, wu = leaf(1.0, 70, 64, seed=4), leaf(0.1, 96, 64, seed=5), leaf(0.1, 96, 64, seed=6)
    audit = RecomputeAudit(2, device=DEV)
    for what in (None, "k", "w"):
        audit.begin_step()
        a = audit.attention(0, q, k, v, causal=True)
        h = audit.gated_ffn(1, x, wg, wu, act="gelu_tanh")
        if what == "k":
            k.data.view(torch.int16)[0, 5, 0, 3] ^= 1 << 9
        if what == "w":
            wu.data.view(torch.int16)[7, 9] ^= 1 << 8
        # (in place behind autograd's back, as a fault would be)
        torch.autograd.backward([a.sum(), h.sum()])
        res = audit.result()
        assert res["mismatched"] == {None: [], "k": [0], "w": [1]}[what], what
        assert res["not_recomputed"] == []
    audit.begin_step()
    a = audit.attention(0, q, k, v)
    with pytest.raises(RuntimeError, match="ran before"):
        audit.attention(0, q, k, v)
    a.sum().backward(retain_graph=True)
    with pytest.raises(RuntimeError, match="ran again"):
        a.sum().backward()
    h = audit.gated_ffn(1, x, wg, wu)
    audit.begin_step()
    with pytest.raises(RuntimeError, match="earlier step"):
        h.sum().backward()
    with pytest.raises(IndexError):
        audit.gated_ffn(2, x, wg, wu)


def test_inside_a_checkpointed_segment():
    """Recomputed whole: wrap() scans the segment's output, the operators run twice."""
    q, k, v = (leaf(1.0, 2, 70, 2, 64, seed=s) for s in (1, 2, 3))
    wg, wu = leaf(0.1, 96, 128, seed=5), leaf(0.1, 96, 128, seed=6)
    audit = RecomputeAudit(1, device=DEV)
    seg = lambda q, k, v: gated_ffn(attention(q, k, v, causal=True).flatten(-2), wg, wu)  # noqa: E731
    audit.begin_step()
    cp.checkpoint(audit.wrap(seg, 0), q, k, v, use_reentrant=True).sum().backward()
    assert audit.result()["mismatched"] == [] and audit.result()["not_recomputed"] == []
    got = [t.grad.clone() for t in (q, k, v, wg, wu)]
    for t in (q, k, v, wg, wu):
        t.grad = None
    seg(q, k, v).sum().backward()
    assert all(torch.equal(t.grad, g) for t, g in zip((q, k, v, wg, wu), got))


def test_a_captured_step():
    """Forward and backward pass of a model of such blocks in one graph, replayed with new
    data and eager steps of other leaves between."""
    m, other = Model(seed=3), Model(seed=3)
    ids, target = batch(7)
    audit = RecomputeAudit(5, device=DEV)

    def step(model, ids, target, audit=None):
        for p in model.params:
            p.grad.zero_()
        loss = model.loss(ids, target, audit)
        loss.backward()
        return loss.detach()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            audit.begin_step()
            step(m, ids, target, audit)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        audit.begin_step()
        loss = step(m, ids, target, audit)
    for turn in range(3):
        a, b = batch(20 + turn)
        ids.copy_(a)
        target.copy_(b)
        g.replay()
        want = step(other, a, b)
        torch.cuda.synchronize()
        assert torch.equal(loss, want), turn
        assert all(torch.equal(p.grad, q.grad) for p, q in zip(m.params, other.params)), turn
        assert audit.mismatch.sum().item() == 0 and torch.equal(audit.original, audit.recomputed)
