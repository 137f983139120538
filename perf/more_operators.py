"""The two recomputed halves of a transformer block, as measured cases: softmax
attention and the gated feed-forward block, each with its gradient, which
computes the scores (the projections) again instead of keeping them.

Each case runs either in plain elementary torch operations (`own` false) or
through the library's entry points (`own` true).
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
NONE = -math.inf


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one short sequence of a small model: the smallest call, where launches count
        dict(name="attn_short", op="attn", batch=1, lq=65, lk=65, hq=8, hkv=8, d=64, causal=True, window=0,
             packed=False, fused=False, type="fp16"),
        # generation: one new token of each of 8 sequences against 8191 keys (grouped heads)
        dict(name="attn_one_token", op="attn", batch=8, lq=1, lk=8191, hq=32, hkv=8, d=128, causal=True, window=0,
             packed=False, fused=False, type="bf16"),
        # two sequences of 2048 tokens through a layer of the GPT-style model, q, k and v from one projection
        dict(name="attn_gpt_2x2048", op="attn", batch=2, lq=2048, lk=2048, hq=16, hkv=16, d=128, causal=True,
             window=0, packed=False, fused=True, type="bf16"),
        # one long sequence through a layer of a 70B-shaped model (64 heads, 8 of keys and values)
        dict(name="attn_8k", op="attn", batch=1, lq=8192, lk=8192, hq=64, hkv=8, d=128, causal=True, window=0,
             packed=False, fused=False, type="bf16"),
        # sequences of odd lengths packed without padding, a window of 500 keys, heads of 80, grouped by 3
        dict(name="attn_grad_packed", op="attn_grad", batch=9, lq=1500, lk=1500, hq=12, hkv=4, d=80, causal=True,
             window=500, packed=True, fused=False, type="fp16"),
        # the gradient for the GPT-style layer
        dict(name="attn_grad_gpt_2x2048", op="attn_grad", batch=2, lq=2048, lk=2048, hq=16, hkv=16, d=128,
             causal=True, window=0, packed=False, fused=True, type="bf16"),
        # the gradient for the long sequence
        dict(name="attn_grad_8k", op="attn_grad", batch=1, lq=8192, lk=8192, hq=64, hkv=8, d=128, causal=True,
             window=0, packed=False, fused=False, type="bf16"),
        # one token through a 70B-shaped layer: bound by reading both weights once
        dict(name="ffn_one_token", op="ffn", n=1, d=8192, f=28672, act="silu", type="bf16"),
        # two sequences of 2048 tokens through the GPT-style layer
        dict(name="ffn_gpt_4096", op="ffn", n=4096, d=2048, f=8192, act="gelu_tanh", type="bf16"),
        # odd sizes in fp16
        dict(name="ffn_grad_ragged", op="ffn_grad", n=1037, d=1000, f=2731, act="gelu_tanh", type="fp16"),
        # the gradient for the GPT-style layer
        dict(name="ffn_grad_gpt_4096", op="ffn_grad", n=4096, d=2048, f=8192, act="silu", type="bf16"),
        # the gradient for the 70B-shaped layer, the largest weights here
        dict(name="ffn_grad_2048", op="ffn_grad", n=2048, d=8192, f=28672, act="silu", type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("bf16", "fp16"))
    if rng.random() < 0.45:
        op = rng.choice(("ffn", "ffn_grad"))
        n, d, f = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 28672)
        if rng.random() < 0.5:
            d, f = max(64, d // 64 * 64), max(64, f // 64 * 64)
        n = max(1, min(n, int(4e11 / (d * f))))
        return dict(op=op, n=n, d=d, f=f, act=rng.choice(("silu", "gelu_tanh")), type=kind)
    op = rng.choice(("attn", "attn_grad"))
    group, hkv = rng.choice((1, 1, 2, 3, 4, 8)), rng.choice((1, 2, 4, 5, 8, 16))
    d = rng.choice((128, 128, 64, 64, 96, 80, 32, 72, 120))
    packed = rng.random() < 0.35
    lk = _log(rng, 16, 8192)
    lq = lk if packed or op == "attn_grad" or rng.random() < 0.5 else _log(rng, 1, min(lk, 64))
    causal = rng.random() < 0.75
    window = _log(rng, 8, lk) if causal and rng.random() < 0.3 else 0
    # scores of one pass: at most half of the largest listed case's
    batch = max(1, min(_log(rng, 1, 32), int(2e9 / (group * hkv * lq * lk))))
    while batch * group * hkv * lq * lk > 2e9:
        group, hkv = max(1, group // 2), max(1, hkv // 2)
    return dict(op=op, batch=batch, lq=lq, lk=lk, hq=group * hkv, hkv=hkv, d=d, causal=causal, window=window,
                packed=packed, fused=lq == lk and rng.random() < 0.3, type=kind)


def _lengths(case):
    """Lengths of the packed sequences: the longest first, the others spread
    over a factor of 30, the same for every seed of the values."""
    g = random.Random(case["batch"] * 10007 + case["lq"])
    rest = [max(1, int(case["lq"] * 30 ** -g.random())) for _ in range(case["batch"] - 1)]
    return [case["lq"]] + rest


def _pairs(case):
    """(pairs of a query and a key that it attends, queries, keys), of one head."""
    pairs = tq = tk = 0
    for lq, lk in [(x, x) for x in _lengths(case)] if case["packed"] else [(case["lq"], case["lk"])] * case["batch"]:
        tq, tk = tq + lq, tk + lk
        if not case["causal"]:
            pairs += lq * lk
            continue
        # query i attends up to i + lk - lq + 1 keys (lq <= lk here), with a window at most that many
        lo, hi, w = lk - lq + 1, lk, case["window"] or lk
        short = max(0, min(hi, w) - lo + 1)       # queries with no more keys than the window
        pairs += (lo + lo + short - 1) * short // 2 + (lq - short) * w
    return pairs, tq, tk


def work(case):
    if case["op"] in ("attn", "attn_grad"):
        pairs, tq, tk = _pairs(case)
        q, kv = 2 * tq * case["hq"] * case["d"], 2 * tk * case["hkv"] * case["d"]
        lse = 4 * tq * case["hq"]
        if case["op"] == "attn":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * pairs * case["hq"] * case["d"]}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * pairs * case["hq"] * case["d"]}
    n, d, f = case["n"], case["d"], case["f"]
    if case["op"] == "ffn":
        return {"bytes": 2 * (n * d + 2 * d * f + n * f), "flops": 4 * n * d * f}
    return {"bytes": 2 * (2 * n * d + 4 * d * f + n * f), "flops": 12 * n * d * f}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(shape, std, dtype, g):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _prepare_attn(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t, d, hq, hkv = TYPES[case["type"]], case["d"], case["hq"], case["hkv"]
    if case["packed"]:
        lengths = _lengths(case)
        first, rows_q, rows_k = [0], (sum(lengths),), (sum(lengths),)
        for x in lengths:
            first.append(first[-1] + x)
        seq = torch.tensor(first, dtype=torch.int32, device=DEV)
    else:
        seq, rows_q, rows_k = None, (case["batch"], case["lq"]), (case["batch"], case["lk"])
    if case["fused"]:
        # one projection's output, heads of q, then of k, then of v
        q, k, v = _normal(rows_q + (hq + 2 * hkv, d), 1.0, t, gen).split((hq, hkv, hkv), dim=-2)
    else:
        q, k, v = (_normal(r + (h, d), 1.0, t, gen) for r, h in ((rows_q, hq), (rows_k, hkv), (rows_k, hkv)))
    s = {"op": case["op"], "q": q, "k": k, "v": v, "causal": case["causal"], "window": case["window"], "seq": seq,
         "longest": case["lq"], "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "attn_grad":
        # what the forward pass left, and the gradient of its output
        left = _plain_attn(s)
        s["out"], s["lse"] = left["out"], left["lse"]
        s["dout"] = _normal(rows_q + (hq, d), 1e-2, t, gen)
    return s


def _prepare_ffn(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n, d, f, t = case["n"], case["d"], case["f"], TYPES[case["type"]]
    s = {"op": case["op"], "act": case["act"], "x": _normal((n, d), 1.0, t, gen),
         "w_gate": _normal((f, d), 1.0 / math.sqrt(d), t, gen), "w_up": _normal((f, d), 1.0 / math.sqrt(d), t, gen)}
    if case["op"] == "ffn_grad":
        s["dh"] = _normal((n, f), 1e-2, t, gen)
    return s


def prepare(case, seed):
    return _prepare_attn(case, seed) if case["op"] in ("attn", "attn_grad") else _prepare_ffn(case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _padded(s, x):
    """A tensor's rows as [batch, heads of keys, rows of all heads that share them, d] in 32
    bits, packed sequences padded to the longest."""
    x = x.float()
    if s["seq"] is not None:
        x = x[_at(s).clamp(max=x.shape[0] - 1)]
    b, rows, h = x.shape[:3]
    g = h // s["k"].shape[-2]
    return x.unflatten(2, (h // g, g)).permute(0, 2, 3, 1, 4).reshape(b, h // g, g * rows, -1)


def _at(s):
    """Packed sequences: the row of each place of the padded batch."""
    return s["seq"][:-1].long().unsqueeze(1) + torch.arange(s["longest"], device=DEV)


def _unpadded(s, x, heads):
    """_padded's inverse: [batch, heads, rows, ...] to the rows' own layout."""
    b, hkv = x.shape[:2]
    g = heads // hkv
    x = x.unflatten(2, (g, x.shape[2] // g)).flatten(1, 2).transpose(1, 2)
    if s["seq"] is not None:
        x = x[_at(s) < s["seq"][1:].unsqueeze(1)]
    return x.contiguous()


def _attended(s, lq, lk):
    """Which keys each query attends, [batch or 1, 1, 1, lq, lk]."""
    i = torch.arange(lq, device=DEV).view(-1, 1) + (lk - lq)
    j = torch.arange(lk, device=DEV)
    ok = torch.ones(1, lq, lk, dtype=torch.bool, device=DEV)
    if s["seq"] is not None:
        # q and k have the same lengths, so only the keys behind the end go
        ok = ok & (j < (s["seq"][1:] - s["seq"][:-1]).view(-1, 1, 1))
    if s["causal"]:
        ok = ok & (j <= i)
        if s["window"]:
            ok = ok & (j > i - s["window"])
    return ok.unsqueeze(1).unsqueeze(1)


def _scores(s, q, k):
    z = (q @ k.transpose(-1, -2)) * s["scale"]
    g = s["q"].shape[-2] // s["k"].shape[-2]
    lq, lk = z.shape[2] // g, z.shape[3]
    return z.unflatten(2, (g, lq)).masked_fill_(~_attended(s, lq, lk), NONE).flatten(2, 3)


def _plain_attn(s):
    q, k, v = _padded(s, s["q"]), _padded(s, s["k"]), _padded(s, s["v"])
    z = _scores(s, q, k)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == NONE, torch.zeros_like(top), top)     # a query of the padding that attends nothing
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total
    hq = s["q"].shape[-2]
    return {"out": _unpadded(s, out, hq).to(s["q"].dtype), "lse": _unpadded(s, (top + total.log()).squeeze(-1), hq)}


def _plain_attn_grad(s):
    q, k, v = _padded(s, s["q"]), _padded(s, s["k"]), _padded(s, s["v"])
    dout = _padded(s, s["dout"])
    delta = (dout * _padded(s, s["out"])).sum(-1, keepdim=True)
    lse = _padded(s, s["lse"].unsqueeze(-1))
    p = _scores(s, q, k).sub_(lse).exp_()
    if s["seq"] is not None:
        # queries of the padding give nothing
        live = (_at(s) < s["seq"][1:].unsqueeze(1)).repeat(1, p.shape[2] // s["longest"])
        p = p * live.view(p.shape[0], 1, -1, 1)
    dv = p.transpose(-1, -2) @ dout
    ds = (dout @ v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(s["scale"])
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    hq, hkv, t = s["q"].shape[-2], s["k"].shape[-2], s["q"].dtype
    return {"dq": _unpadded(s, dq, hq).to(t), "dk": _unpadded(s, dk, hkv).to(t), "dv": _unpadded(s, dv, hkv).to(t)}


ROOT_2_OVER_PI = math.sqrt(2.0 / math.pi)


def _act(name, g):
    """(the activation, its derivative) at g."""
    if name == "silu":
        y = 1.0 / (1.0 + torch.exp(-g))
        return g * y, y * (1.0 + g * (1.0 - y))
    # 0.5 g (1 + tanh(u)) with u = sqrt(2 / pi) (g + 0.044715 g^3); 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2 u))
    y = 1.0 / (1.0 + torch.exp(-2.0 * ROOT_2_OVER_PI * (g + 0.044715 * g * g * g)))
    return g * y, y + g * y * (1.0 - y) * 2.0 * ROOT_2_OVER_PI * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_ffn(s):
    x = s["x"].float()
    a, _ = _act(s["act"], x @ s["w_gate"].float().t())
    return {"h": (a * (x @ s["w_up"].float().t())).to(s["x"].dtype)}


def _plain_ffn_grad(s):
    x, wg, wu, dh = s["x"].float(), s["w_gate"].float(), s["w_up"].float(), s["dh"].float()
    a, slope = _act(s["act"], x @ wg.t())
    dg, du = dh * (x @ wu.t()) * slope, dh * a
    t = s["x"].dtype
    return {"dx": (dg @ wg + du @ wu).to(t), "dw_gate": (dg.t() @ x).to(t), "dw_up": (du.t() @ x).to(t)}


def run(state):
    s = state
    if own:
        import silent_corruption_detection_amd as sdc
        if s["op"] in ("attn", "attn_grad"):
            how = dict(causal=s["causal"], window=s["window"], scale=s["scale"], seq_q=s["seq"], seq_k=s["seq"])
            if s["op"] == "attn":
                out, lse = sdc.sdc_attention(s["q"], s["k"], s["v"], **how)
                return {"out": out, "lse": lse}
            dq, dk, dv = sdc.sdc_attention_grad(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], **how)
            return {"dq": dq, "dk": dk, "dv": dv}
        if s["op"] == "ffn":
            return {"h": sdc.sdc_gated_ffn(s["x"], s["w_gate"], s["w_up"], act=s["act"])}
        dx, dw_gate, dw_up = sdc.sdc_gated_ffn_grad(s["x"], s["w_gate"], s["w_up"], s["dh"], act=s["act"])
        return {"dx": dx, "dw_gate": dw_gate, "dw_up": dw_up}
    plain = {"attn": _plain_attn, "attn_grad": _plain_attn_grad, "ffn": _plain_ffn, "ffn_grad": _plain_ffn_grad}
    return plain[s["op"]](s)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_attn(case, seed):
    """Softmax attention and, by its chain rule, its gradient: one sequence and
    one head of queries at a time."""
    s = _prepare_attn(case, seed)
    grad, hq, group = case["op"] == "attn_grad", case["hq"], case["hq"] // case["hkv"]
    flat = {n: s[n].reshape(-1, *s[n].shape[-2:]) for n in ("q", "k", "v") + (("dout",) if grad else ())}
    made = {n: torch.zeros(flat[n[-1]].shape, dtype=torch.float64, device=DEV) for n in ("dq", "dk", "dv")}
    made["out"] = torch.zeros(flat["q"].shape, dtype=torch.float64, device=DEV)
    made["lse"] = torch.zeros(flat["q"].shape[:2], dtype=torch.float64, device=DEV)
    each = [(n, n) for n in _lengths(case)] if case["packed"] else [(case["lq"], case["lk"])] * case["batch"]
    q0 = k0 = 0
    for lq, lk in each:
        qs, ks = slice(q0, q0 + lq), slice(k0, k0 + lk)
        q0, k0 = q0 + lq, k0 + lk
        # how far each key lies behind the query, whose own place is lk - lq further on
        behind = torch.arange(lq, device=DEV).unsqueeze(1) + (lk - lq) - torch.arange(lk, device=DEV)
        out_of_sight = torch.zeros_like(behind, dtype=torch.bool)
        if case["causal"]:
            out_of_sight = behind < 0
            if case["window"] > 0:
                out_of_sight = out_of_sight | (behind >= case["window"])
        for h in range(hq):
            q, k, v = flat["q"][qs, h].double(), flat["k"][ks, h // group].double(), flat["v"][ks, h // group].double()
            z = torch.mm(q, k.t()) / math.sqrt(case["d"])
            z[out_of_sight] = NONE
            if not grad:
                made["lse"][qs, h] = torch.logsumexp(z, 1)
                made["out"][qs, h] = torch.mm(torch.softmax(z, 1), v)
                continue
            p, do = torch.softmax(z, 1), flat["dout"][qs, h].double()
            made["dv"][ks, h // group] += torch.mm(p.t(), do)
            dp = torch.mm(do, v.t())
            dz = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(case["d"])
            made["dq"][qs, h] = torch.mm(dz, k)
            made["dk"][ks, h // group] += torch.mm(dz.t(), q)
    if not grad:
        return {"out": made["out"].view(s["q"].shape), "lse": made["lse"].view(s["q"].shape[:-1])}
    return {"dq": made["dq"].view(s["q"].shape), "dk": made["dk"].view(s["k"].shape), "dv": made["dv"].view(s["v"].shape)}


def _exact_ffn(case, seed):
    s = _prepare_ffn(case, seed)
    x, wg, wu = s["x"].double(), s["w_gate"].double(), s["w_up"].double()
    g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    if case["act"] == "silu":
        half = torch.sigmoid(g)
        a, slope = g * half, half + g * half * (1 - half)
    else:
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (g + 0.044715 * g ** 3))
        a, slope = g * (1 + th) / 2, (1 + th) / 2 + g / 2 * (1 - th ** 2) * c * (1 + 3 * 0.044715 * g ** 2)
    if case["op"] == "ffn":
        return {"h": a * u}
    dh = s["dh"].double()
    dg, du = dh * u * slope, dh * a
    return {"dx": torch.mm(dg, wg) + torch.mm(du, wu), "dw_gate": torch.mm(dg.t(), x), "dw_up": torch.mm(du.t(), x)}


def exact(case, seed):
    return _exact_attn(case, seed) if case["op"] in ("attn", "attn_grad") else _exact_ffn(case, seed)
