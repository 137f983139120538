"""The optimizer step and the loss head, as measured cases: AdamW over a tensor
list (states in 32 or in 8 bits) and the softmax cross entropy of a linear head
whose logits are never kept, with its gradient.

Each case runs either in plain elementary torch operations (`own` false) or
through the library's entry points (`own` true).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1
STEP, SEED = 1000, 1234567
BLOCK = 128   # elements that share a scale of an 8-bit state


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one 1M-element fp32 tensor: the smallest step, where launches count
        dict(name="adamw32_one_1m", op="adamw", list="one", n=1 << 20, param="fp32", grad="fp32",
             master=False, state=32, clip=True),
        # a GPT-style 0.96B fp32 model (embedding, LayerNorm gains, biases): the whole step, clipped
        dict(name="adamw32_gpt_fp32", op="adamw", list="gpt", d=2048, layers=17, vocab=50304, param="fp32",
             grad="fp32", master=False, state=32, clip=True),
        # one layer of a 70B-shaped model: bf16 weights and gradients with fp32 master weights
        dict(name="adamw32_layer_master", op="adamw", list="layer", d=8192, kv=1024, ffn=28672,
             param="bf16", grad="bf16", master=True, state=32, clip=False),
        # thousands of small tensors of mixed types at odd offsets (adapters, norms, biases)
        dict(name="adamw32_small_mixed", op="adamw", list="small", n=20000, most=65536, param="mixed",
             grad="same", master=False, state=32, clip=True),
        # one 1M-element bf16 tensor with 8-bit states
        dict(name="adamw8_one_1m", op="adamw", list="one", n=1 << 20, param="bf16", grad="bf16",
             master=False, state=8, clip=True),
        # the GPT-style model in bf16 with 8-bit states
        dict(name="adamw8_gpt_bf16", op="adamw", list="gpt", d=2048, layers=17, vocab=50304, param="bf16",
             grad="bf16", master=False, state=8, clip=True),
        # small tensors whose last 128-element block is short, fp32 gradients of 16-bit weights
        dict(name="adamw8_small_ragged", op="adamw", list="small", n=4000, most=65536, param="mixed",
             grad="fp32", master=False, state=8, clip=False),
        # the loss of one token against a 128k vocabulary: bound by reading the head once
        dict(name="xent_one_token", op="xent", n=1, d=8192, vocab=128256, type="bf16", ignored=0.0),
        # two sequences of 2048 tokens through the GPT-style model's head
        dict(name="xent_gpt_4096", op="xent", n=4096, d=2048, vocab=50304, type="bf16", ignored=0.0),
        # odd sizes in fp16, a third of the rows without a target (padding, prompts)
        dict(name="xent_grad_ragged", op="xent_grad", n=1037, d=1000, vocab=32003, type="fp16", ignored=0.33),
        # the gradient for the GPT-style head
        dict(name="xent_grad_gpt_4096", op="xent_grad", n=4096, d=2048, vocab=50304, type="bf16", ignored=0.0),
        # the gradient for a 70B-shaped model's head, the largest vocabulary here
        dict(name="xent_grad_2048_128k", op="xent_grad", n=2048, d=8192, vocab=128256, type="bf16", ignored=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        state = rng.choice((32, 8))
        param = rng.choice(("fp32", "bf16", "fp16", "mixed"))
        grad = rng.choice(("same", "fp32"))
        master = param in ("bf16", "fp16") and rng.random() < 0.4
        c = dict(op="adamw", param=param, grad=grad, master=master, state=state, clip=state == 8 or rng.random() < 0.5)
        kind = rng.choice(("one", "gpt", "layer", "small"))
        if kind == "one":
            c.update(list="one", n=_log(rng, 1000, 1 << 27))
        elif kind == "gpt":
            c.update(list="gpt", d=64 * _log(rng, 1, 24), layers=_log(rng, 1, 12), vocab=_log(rng, 500, 40000))
        elif kind == "layer":
            d = 128 * _log(rng, 2, 48)
            c.update(list="layer", d=d, kv=max(64, d // 8), ffn=8 * _log(rng, d // 4, d // 2))
        else:
            c.update(list="small", n=_log(rng, 10, 10000), most=_log(rng, 100, 65536))
        return c
    op = rng.choice(("xent", "xent_grad"))
    n, d, vocab = _log(rng, 1, 4096), _log(rng, 64, 8192), _log(rng, 500, 128256)
    n = max(1, min(n, int(5e11 / (d * vocab))))
    return dict(op=op, n=n, d=d, vocab=vocab, type=rng.choice(("bf16", "fp16")),
                ignored=rng.choice((0.0, 0.05, 0.5)))


def _sizes(case):
    """[(numel, weight decay applies)] of the list's tensors."""
    kind = case["list"]
    if kind == "one":
        return [(case["n"], True)]
    if kind == "gpt":
        d = case["d"]
        out = [(case["vocab"] * d, True)]
        for _ in range(case["layers"]):
            out += [(d, False), (d, False), (3 * d * d, True), (3 * d, False), (d * d, True), (d, False),
                    (d, False), (d, False), (4 * d * d, True), (4 * d, False), (4 * d * d, True), (d, False)]
        return out + [(d, False), (d, False)]
    if kind == "layer":
        d, kv, f = case["d"], case["kv"], case["ffn"]
        return [(d * d, True), (kv * d, True), (kv * d, True), (d * d, True), (f * d, True), (f * d, True),
                (d * f, True), (d, False), (d, False)]
    # log-uniform sizes, the same list for every seed of the values
    g = torch.Generator().manual_seed(4)
    u = torch.rand(case["n"], generator=g, dtype=torch.float64) * math.log(case["most"] + 1)
    return [(max(1, min(case["most"], int(s))), k % 4 != 3) for k, s in enumerate(torch.exp(u).tolist())]


def _classes(case):
    """The list's tensors by element type and decay group, in list order:
    [(param type, grad type, group, [numels])].  Tensors of one class lie
    packed in one buffer, so odd sizes give odd offsets."""
    names = ("fp32", "bf16", "fp16") if case["param"] == "mixed" else (case["param"],)
    got = {}
    for k, (n, decays) in enumerate(_sizes(case)):
        got.setdefault((names[k % len(names)], 0 if decays else 1), []).append(n)
    return [(TYPES[p], TYPES["fp32"] if case["grad"] == "fp32" else TYPES[p], grp, sizes)
            for (p, grp), sizes in sorted(got.items())]


def work(case):
    if case["op"] == "adamw":
        nbytes, n_all = 0, 0
        for p, g, _, sizes in _classes(case):
            n = sum(sizes)
            es, eg = p.itemsize, g.itemsize
            nbytes += n * (2 * es + eg)
            if case["master"]:
                nbytes += n * (8 - es)        # the 16-bit weights are only written
            nbytes += n * 16 if case["state"] == 32 else n * 4 + 4 * sum(-(-s // BLOCK) for s in sizes)
            n_all += n
        return {"bytes": nbytes, "flops": 15 * n_all}
    n, d, v = case["n"], case["d"], case["vocab"]
    if case["op"] == "xent":
        return {"bytes": 2 * (n + v) * d + 16 * n, "flops": 2 * n * v * d}
    return {"bytes": 4 * (n + v) * d + 12 * n, "flops": 6 * n * v * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(n, std, dtype, g):
    return torch.empty(n, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _prepare_adamw(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    classes, total = [], torch.zeros((), dtype=torch.float64, device=DEV)
    for p, gt, grp, sizes in _classes(case):
        n = sum(sizes)
        c = {"group": grp, "sizes": sizes}
        w = _normal(n, 0.02, torch.float32, gen)
        c["param"] = w.to(p)
        c["master"] = w if case["master"] else None
        # magnitudes that differ from row to row, as those of real gradients do
        c["grad"] = _normal(n, 1e-3, torch.float32, gen)
        c["grad"] *= torch.rand(n, device=DEV, generator=gen)
        c["grad"] = c["grad"].to(gt)
        total += torch.linalg.vector_norm(c["grad"], dtype=torch.float64).square()
        if case["state"] == 32:
            c["m"] = _normal(n, 3e-4, torch.float32, gen)
            c["v"] = _normal(n, 1.0, torch.float32, gen).exp_().mul_(3e-7)
        else:
            # the blocks' largest values lie between the powers of two, where a last-bit
            # difference does not choose another scale
            nb = sum(-(-s // BLOCK) for s in sizes)
            c["m"] = _normal(n, 90.0, torch.float32, gen).clamp_(-240, 240).to(torch.float8_e4m3fn)
            c["v"] = _normal(n, 0.6, torch.float32, gen).exp_().mul_(50).clamp_(0.05, 240).to(torch.float8_e4m3fn)
            c["m_scale"] = torch.randint(107, 111, (nb,), dtype=torch.uint8, device=DEV, generator=gen)
            c["v_scale"] = torch.randint(109, 112, (nb,), dtype=torch.uint8, device=DEV, generator=gen)
        classes.append(c)
    s = {"op": "adamw", "state": case["state"], "classes": classes, "sq_total": total.reshape(1),
         # a clip that is at work: every gradient is scaled by about 1/e, so that sums of
         # 8-bit states and 16-bit gradients do not fall exactly on powers of two
         "max_norm": math.sqrt(float(total)) / math.e if case["clip"] else 0.0,
         "groups": torch.tensor([[LR, BETA1, BETA2, EPS, DECAY], [LR, BETA1, BETA2, EPS, 0.0]],
                                dtype=torch.float64, device=DEV)}
    if own:
        import silent_corruption_detection_amd as sdc
        lists = {k: [] for k in ("param", "grad", "m", "v", "master", "m_scale", "v_scale")}
        group = []
        for c in classes:
            group += [c["group"]] * len(c["sizes"])
            for k, into in lists.items():
                if c.get(k) is not None:
                    into += c[k].split([-(-x // BLOCK) for x in c["sizes"]] if "scale" in k else c["sizes"])
        s["plan"] = sdc.sdc_adamw_plan_build(
            lists["param"], lists["grad"], lists["m"], lists["v"], master=lists["master"] or None,
            exp_avg_scale=lists["m_scale"] or None, exp_avg_sq_scale=lists["v_scale"] or None,
            group=group, n_groups=2)
        s["control"] = sdc.sdc_adamw_control(DEV, step=STEP, seed=SEED)
    else:
        s["step"] = torch.full((), STEP, dtype=torch.int64, device=DEV)
    return s


def _prepare_xent(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n, d, v, t = case["n"], case["d"], case["vocab"], TYPES[case["type"]]
    s = {"op": case["op"],
         "x": _normal(n * d, 1.0, t, gen).view(n, d),
         "w": _normal(v * d, 1.0 / math.sqrt(d), t, gen).view(v, d),
         "target": torch.randint(0, v, (n,), device=DEV, generator=gen)}
    skip = torch.rand(n, device=DEV, generator=gen) < case["ignored"]
    s["target"] = torch.where(skip, torch.full_like(s["target"], -100), s["target"])
    if case["op"] == "xent_grad":
        # what the forward pass left: each row's log-sum-exp, and 1 / rows with a target
        s["lse"] = torch.logsumexp(s["x"].float() @ s["w"].float().t(), 1)
        s["coef"] = 1.0 / (~skip).sum().clamp(min=1).float().reshape(1)
    return s


def prepare(case, seed):
    return _prepare_adamw(case, seed) if case["op"] == "adamw" else _prepare_xent(case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _outputs(s):
    """The updated weights and states; an 8-bit state as the e4m3 values it
    holds and the powers of two that scale its blocks."""
    out = []
    for c in s["classes"]:
        o = {"param": c["param"], "m": c["m"], "v": c["v"]}
        if c["master"] is not None:
            o["master"] = c["master"]
        if s["state"] == 8:
            o["m_scale"] = c["m_scale"].view(torch.float8_e8m0fnu)
            o["v_scale"] = c["v_scale"].view(torch.float8_e8m0fnu)
        out.append(o)
    return out


def _random_bits(first, n, step):
    """The 32 random bits of each element: a hash of the seed, the step and
    the element's index over the whole list (two multiply-xorshift rounds)."""
    m32 = 0xFFFFFFFF
    k0 = ((SEED & m32) * 0x9E3779B1 + (step & m32) * 0x85157AF5) & m32
    k1 = ((SEED >> 32) * 0x9E3779B1 + (step >> 32) * 0x85157AF5 + 0x6C8E9CF5) & m32
    i = torch.arange(first, first + n, dtype=torch.int64, device=DEV)
    a = ((i & m32) + k0) & m32
    a = a ^ (a >> 16)
    a = (a * 0x7FEB352D) & m32
    a = a ^ ((k1 + (i >> 32) * 0x2C1B3C6D) & m32)
    a = a ^ (a >> 15)
    a = (a * 0x846CA68B) & m32
    return a ^ (a >> 16)


def _block_of(sizes):
    """Scale index of each element (blocks start anew with each tensor)."""
    if all(s % BLOCK == 0 for s in sizes):
        return None
    n = torch.tensor(sizes, device=DEV)
    nb = (n + BLOCK - 1) // BLOCK
    first = torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    base = torch.repeat_interleave(torch.cumsum(nb, 0) - nb, n)
    return base + (torch.arange(int(sum(sizes)), device=DEV) - first) // BLOCK


def _spread(per_block, block, n):
    """A value of each block at each of its elements."""
    if block is None:
        return per_block.unsqueeze(1).expand(-1, BLOCK).reshape(n)
    return per_block[block]


def _scale_byte(x, block, blocks):
    """max(exponent field of the block's largest value - 7, 1)."""
    if block is None:
        top = x.view(-1, BLOCK).amax(1)
    else:
        top = torch.zeros(blocks, device=DEV).scatter_reduce(0, block, x, "amax")
    return ((top.view(torch.int32) >> 23) - 7).clamp(min=1)


def _pow2(field):
    return (field << 23).view(torch.float32)


UP, DOWN = 2.0 ** 120, 2.0 ** -120   # e4m3's exponent offset within fp32's


def _held_m(m, block, blocks, bits):
    s = _scale_byte(m.abs(), block, blocks)
    y = m.abs() * _spread(_pow2(254 - s), block, m.numel()) * DOWN
    code = (y.view(torch.int32) + (((bits & 0xFFFF) << 4) + 8).int()) >> 20
    code = code.clamp(max=0x7F) | torch.where(m < 0, 0x80, 0)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), s.to(torch.uint8)


def _held_r(r, block, blocks, bits):
    """r = sqrt(v), rounded up or down so that the expected square is r^2; never to zero."""
    s = _scale_byte(r, block, blocks)
    t = r * _spread(_pow2(254 - s), block, r.numel())
    code = (t * DOWN).view(torch.int32) >> 20
    lo = (code << 20).view(torch.float32) * UP
    hi = ((code + 1) << 20).view(torch.float32) * UP
    u = ((bits >> 16).float() + 0.5) * 2.0 ** -16
    code = code + (u * (hi * hi - lo * lo) < t * t - lo * lo).int()
    code = torch.where(r > 0, code.clamp(min=1), code).clamp(max=0x7F)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), s.to(torch.uint8)


def _plain_adamw(s):
    s["step"] += 1
    t = s["step"].double()
    scale = torch.ones((), device=DEV)
    if s["max_norm"] > 0:
        scale = (s["max_norm"] / (s["sq_total"].sqrt() + 1e-6)).clamp(max=1.0).float()
    first = 0
    for c in s["classes"]:
        lr, b1, b2, eps, wd = LR, BETA1, BETA2, EPS, DECAY if c["group"] == 0 else 0.0
        size = (lr / (1.0 - b1 ** t)).float()
        rbc2 = (1.0 / (1.0 - b2 ** t).sqrt()).float()
        n = c["param"].numel()
        g = c["grad"].float() * scale
        if s["state"] == 32:
            m, v = c["m"], c["v"]
        else:
            block, blocks = _block_of(c["sizes"]), c["m_scale"].numel()
            m = c["m"].float() * _spread(_pow2(c["m_scale"].int()), block, n)
            v = (c["v"].float() * _spread(_pow2(c["v_scale"].int()), block, n)).square()
        m = m * b1 + g * (1.0 - b1)
        v = v * b2 + g * g * (1.0 - b2)
        r = v.sqrt()
        p = c["master"] if c["master"] is not None else c["param"].float()
        p = p * (1.0 - lr * wd) - size * (m / (r * rbc2 + eps))
        c["param"] = p.to(c["param"].dtype)
        if c["master"] is not None:
            c["master"] = p
        if s["state"] == 32:
            c["m"], c["v"] = m, v
        else:
            bits = _random_bits(first, n, s["step"])
            c["m"], c["m_scale"] = _held_m(m, block, blocks, bits)
            c["v"], c["v_scale"] = _held_r(r, block, blocks, bits)
        first += n
    return _outputs(s)


def _plain_xent(s):
    z = s["x"].float() @ s["w"].float().t()
    top = z.amax(1)
    lse = top + (z - top.unsqueeze(1)).exp().sum(1).log()
    counted = s["target"] >= 0
    at = z.gather(1, s["target"].clamp(min=0).unsqueeze(1)).squeeze(1)
    loss = torch.where(counted, lse - at, 0.0)
    return {"loss": loss, "lse": lse, "total": loss.double().sum().float().reshape(1)}


def _plain_xent_grad(s):
    x, w = s["x"].float(), s["w"].float()
    dz = (x @ w.t() - s["lse"].unsqueeze(1)).exp()
    counted = s["target"] >= 0
    dz.scatter_add_(1, s["target"].clamp(min=0).unsqueeze(1), torch.full_like(dz[:, :1], -1.0))
    dz = torch.where(counted.unsqueeze(1), dz * s["coef"], 0.0)
    return {"dx": (dz @ w).to(s["x"].dtype), "dw": (dz.t() @ x).to(s["w"].dtype)}


def run(state):
    if own:
        import silent_corruption_detection_amd as sdc
        if state["op"] == "adamw":
            sdc.sdc_adamw_step(state["plan"], state["groups"], state["control"],
                               sq_total=state["sq_total"], max_norm=state["max_norm"])
            return _outputs(state)
        if state["op"] == "xent":
            loss, lse, total = sdc.sdc_cross_entropy(state["x"], state["w"], state["target"])
            return {"loss": loss, "lse": lse, "total": total}
        dx, dw = sdc.sdc_cross_entropy_grad(state["x"], state["w"], state["target"], state["lse"],
                                            state["coef"])
        return {"dx": dx, "dw": dw}
    if state["op"] == "adamw":
        return _plain_adamw(state)
    return _plain_xent(state) if state["op"] == "xent" else _plain_xent_grad(state)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_codes(value, sizes, first, root):
    """Definition of the 8-bit states on one class: magnitudes in units of the
    block's power of two, the two neighbouring e4m3 values, and the one that
    the element's random bits choose.  root: `value` is v, held as sqrt(v)."""
    mag = value.sqrt() if root else value.abs()
    idx = torch.arange(value.numel(), device=DEV) + first
    h = (idx % 2 ** 32 + (SEED * 0x9E3779B1 + (STEP + 1) * 0x85157AF5)) % 2 ** 32
    h = ((h ^ (h >> 16)) * 0x7FEB352D) % 2 ** 32
    h = h ^ ((0x6C8E9CF5 + (idx // 2 ** 32) * 0x2C1B3C6D) % 2 ** 32)
    h = ((h ^ (h >> 15)) * 0x846CA68B) % 2 ** 32
    h = h ^ (h >> 16)
    runs = [sum(sizes)] if all(s % BLOCK == 0 for s in sizes) else sizes
    if len(runs) > 1:
        # pad every tensor to whole blocks
        width = -(-max(sizes) // BLOCK) * BLOCK
        n = torch.tensor(sizes, device=DEV)
        row = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), n)
        col = torch.arange(value.numel(), device=DEV) - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
        grid = torch.zeros(len(sizes), width, dtype=torch.float64, device=DEV)
        grid[row, col] = mag
        tops = grid.view(len(sizes), -1, BLOCK).amax(2)
        live = torch.arange(width // BLOCK, device=DEV).unsqueeze(0) * BLOCK < n.unsqueeze(1)
        pick = (row, col // BLOCK)
    else:
        pad = -(-mag.numel() // BLOCK) * BLOCK - mag.numel()
        tops = torch.nn.functional.pad(mag, (0, pad)).view(-1, BLOCK).amax(1)
        live, pick = torch.ones_like(tops, dtype=torch.bool), (torch.arange(mag.numel(), device=DEV) // BLOCK,)
    e = torch.frexp(tops)[1].to(torch.float64) - 1 - 7          # the largest value lands in [128, 256)
    e = torch.where(tops > 0, e, -126.0).clamp(min=-126.0)
    t = mag / torch.exp2(e[pick])
    step = torch.exp2((torch.frexp(t)[1] - 1).clamp(min=-6).double() - 3)
    step = torch.where(t > 0, step, 2.0 ** -9)
    lo = torch.floor(t / step) * step
    hi = lo + step
    if root:
        up = (((h >> 16).double() + 0.5) / 65536 * (hi * hi - lo * lo)) < t * t - lo * lo
        held = torch.where(up, hi, lo)
        held = torch.where(value > 0, held.clamp(min=2.0 ** -9), held)
    else:
        up = (t - lo) / step + (((h % 65536) * 16 + 8).double() / 2 ** 20) >= 1
        held = torch.where(up, hi, lo) * torch.sign(value)
    return held, torch.exp2(e)[live].reshape(-1)


def _exact_adamw(case, seed):
    s = _prepare_adamw(case, seed)
    clip = 1.0
    if case["clip"]:
        clip = min(1.0, s["max_norm"] / (math.sqrt(float(s["sq_total"])) + 1e-6))
    t, out, first = STEP + 1, [], 0
    for c in s["classes"]:
        sizes, n = c["sizes"], c["param"].numel()
        g = c["grad"].double() * clip
        m, v = c["m"].double(), c["v"].double()
        if case["state"] == 8:
            nb = torch.tensor([-(-x // BLOCK) for x in sizes], device=DEV)
            length = torch.full((int(nb.sum()),), BLOCK, device=DEV)
            length[torch.cumsum(nb, 0) - 1] = torch.tensor([x - (-(-x // BLOCK) - 1) * BLOCK for x in sizes], device=DEV)
            m = m * torch.repeat_interleave(torch.exp2(c["m_scale"].double() - 127), length)
            v = (v * torch.repeat_interleave(torch.exp2(c["v_scale"].double() - 127), length)) ** 2
        m += (g - m) * (1 - BETA1)
        v += (g * g - v) * (1 - BETA2)
        p = (c["param"] if c["master"] is None else c["master"]).double()
        p = p - LR * (DECAY if c["group"] == 0 else 0.0) * p
        p -= LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
        del g
        o = {"param": p, "m": m, "v": v}
        if case["master"]:
            o["master"] = p
        if case["state"] == 8:
            o["m"], o["m_scale"] = _exact_codes(m, sizes, first, False)
            o["v"], o["v_scale"] = _exact_codes(v, sizes, first, True)
        out.append(o)
        first += n
    return out


def exact(case, seed):
    if case["op"] == "adamw":
        return _exact_adamw(case, seed)
    s = _prepare_xent(case, seed)
    x, w, rows = s["x"].double(), s["w"].double(), torch.arange(case["n"], device=DEV)
    z = torch.mm(x, w.t())
    has = s["target"] != -100
    hit = torch.where(has, s["target"], 0)
    if case["op"] == "xent":
        lse = torch.logsumexp(z, 1)
        loss = (lse - z[rows, hit]) * has
        return {"loss": loss, "lse": lse, "total": loss.sum().reshape(1)}
    q = torch.softmax(z, 1)
    q[rows, hit] -= 1.0
    q *= (has / has.sum().clamp(min=1)).unsqueeze(1)
    return {"dx": torch.mm(q, w), "dw": torch.mm(q.t(), x)}
