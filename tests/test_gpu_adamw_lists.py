"""GPU tests of the memory of an AdamW plan: what the step writes shares none, what
it only reads may, and the plan's own lives as long as a step that uses it."""
import pytest
import torch

import silent_corruption_detection_amd as sdc

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_overlapping_views_are_refused():
    flat = lambda n=400: torch.zeros(n, device=DEV)  # noqa: E731
    build = sdc.sdc_adamw_plan_build
    p, m, v = flat(), flat(), flat()
    g = [flat(200), flat(200)]
    sides = lambda t, step=200: [t[:200], t[step:step + 200]]  # noqa: E731
    build(sides(p), g, sides(m), sides(v))
    for columns in ((sides(p, 199), sides(m), sides(v)), (sides(p), sides(m, 1), sides(v)), (sides(p), sides(m), sides(v, 100))):
        with pytest.raises(ValueError, match=r"\[0\] and .*\[1\] overlap"):
            build(columns[0], g, *columns[1:])
    with pytest.raises(ValueError, match="listed twice"):
        build(sides(p, 0), g, sides(m), sides(v))
    with pytest.raises(ValueError, match=r"param\[0\] and grad\[1\] overlap"):
        build(sides(p), [g[0], p[100:300]], sides(m), sides(v))
    # 16-bit weights behind masters; the masters overlap
    with pytest.raises(ValueError, match=r"master\[0\] and master\[1\] overlap"):
        build([t.half() for t in sides(p)], g, sides(m), sides(v), master=sides(flat(), 199))
    # 8-bit states: the scale bytes of 200 elements are two
    code = lambda: torch.zeros(400, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # noqa: E731
    s = torch.zeros(8, dtype=torch.uint8, device=DEV)
    kw = dict(exp_avg_sq_scale=[s[4:6], s[6:8]])
    build(sides(p), g, sides(code()), sides(code()), exp_avg_scale=[s[0:2], s[2:4]], **kw)
    with pytest.raises(ValueError, match=r"exp_avg_scale\[0\] and exp_avg_scale\[1\] overlap"):
        build(sides(p), g, sides(code()), sides(code()), exp_avg_scale=[s[0:2], s[1:3]], **kw)


def test_what_is_only_read_may_be_shared():
    g = torch.Generator(device=DEV).manual_seed(1)
    p = [torch.empty(300, device=DEV).normal_(generator=g) for _ in range(3)]
    grad = torch.empty(300, device=DEV).normal_(generator=g)
    m, v = ([torch.zeros(300, device=DEV) for _ in range(3)] for _ in range(2))
    frozen = torch.ones(300, device=DEV)
    start = [t.clone() for t in p]
    plan = sdc.sdc_adamw_plan_build([p[0], p[1], frozen, frozen], [grad, grad, None, None],
                                    [m[0], m[1], m[2], m[2]], [v[0], v[1], v[2], v[2]])
    groups = torch.tensor([[1e-2, 0.9, 0.99, 1e-8, 0.0]], dtype=torch.float64, device=DEV)
    rows = torch.zeros(4, 4, dtype=torch.int64, device=DEV)
    sdc.sdc_adamw_step(plan, groups, sdc.sdc_adamw_control(DEV), rows=rows)
    for k in range(2):   # the first step is lr times the gradient's sign, up to eps and 20 roundings of 2^-24
        want = start[k].double() - 1e-2 * grad.sign().double()
        assert ((p[k].double() - want).abs() <= 20 * 2.0 ** -24 * (start[k].double().abs() + 1e-2)
                + 1e-2 * 1e-8 / grad.double().abs()).all()
    assert torch.equal(m[0], m[1]) and torch.equal(rows[2], rows[3]) and (frozen == 1).all()
    # weights that a step writes are not those of a tensor without a gradient
    with pytest.raises(ValueError, match=r"param\[0\] and param\[1\]"):
        sdc.sdc_adamw_plan_build([p[0], p[0]], [grad, None], [m[0], m[1]], [v[0], v[1]])


@pytest.mark.parametrize("current", [False, True])
def test_a_plan_dropped_behind_a_step_on_another_stream(current):
    """The plan holds the step's scratch, so its memory is not handed out before the
    step has run, also where that is on another stream than the plan was made on."""
    p, g, m, v = (torch.zeros(5_000_000, device=DEV) for _ in range(4))
    plan = sdc.sdc_adamw_plan_build([p], [g], [m], [v])
    groups = torch.tensor([[1e-2, 0.9, 0.99, 1e-8, 0.0]], dtype=torch.float64, device=DEV)
    control = sdc.sdc_adamw_control(DEV)
    at, size = plan.buf.data_ptr(), plan.buf.numel()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    if current:
        with torch.cuda.stream(s):
            sdc.sdc_adamw_step(plan, groups, control)
    else:
        sdc.sdc_adamw_step(plan, groups, control, stream=s)
    del plan
    again = torch.empty(size, dtype=torch.uint8, device=DEV)
    running = not s.query()
    torch.cuda.synchronize()
    assert running and again.data_ptr() != at
    assert control.tolist()[0] == 1


@pytest.mark.parametrize("eps", [1e-46, 1e-40, 2.0 ** -127, 1e-30, 1e-8])
@pytest.mark.parametrize("state", [32, 8])
def test_elements_that_never_had_a_gradient_stay(state, eps):
    """m = v = 0 moves nothing, however small eps is: eps above 0 but below fp32's normal
    numbers has no reciprocal in fp32.  Elements with a gradient move by lr."""
    n = 1000
    g = torch.Generator(device=DEV).manual_seed(2)
    p = torch.empty(n, device=DEV).normal_(generator=g)
    grad = torch.empty(n, device=DEV).normal_(generator=g).sign()
    grad[100:400] = 0
    start = p.clone()
    z = lambda k, t: torch.zeros(k, dtype=t, device=DEV)  # noqa: E731
    if state == 32:
        m, v, kw = z(n, torch.float32), z(n, torch.float32), {}
    else:
        m, v = (z(n, torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
        kw = dict(exp_avg_scale=[z(8, torch.uint8)], exp_avg_sq_scale=[z(8, torch.uint8)])
    plan = sdc.sdc_adamw_plan_build([p], [grad], [m], [v], **kw)
    groups = torch.tensor([[1e-2, 0.9, 0.99, eps, 0.0]], dtype=torch.float64, device=DEV)
    sdc.sdc_adamw_step(plan, groups, sdc.sdc_adamw_control(DEV))
    assert torch.equal(p[100:400], start[100:400])
    # the update is lr, up to 20 roundings and eps
    want = start.double() - 1e-2 * grad.double()
    assert ((p.double() - want).abs() <= 20 * 2.0 ** -24 * (start.double().abs() + 1e-2) + 1e-2 * eps).all()
