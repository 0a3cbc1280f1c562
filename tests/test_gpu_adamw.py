"""The AdamW step over many tensors against its formula in 64 bits, and the 8-bit states against their format.

Tolerances: m and v are two products and a sum, each rounded to 2^-24: 2e-7 of the sizes added.  The parameter's new
value has a few fp32 roundings of p and of the step lr m_hat / (sqrt(v_hat) + eps), whose division and root add 2^-22:
3e-7 |p| + 2e-6 |step|, and 2^-8 |p| more where it is stored in bf16 (half a unit in the last place of 8 bits).  The 8-bit states
are exactly those that the same fp32 operations give in the format's definition, here in torch on the host.
"""
import math

import pytest

from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from lora_fine_tuning_gb300 import api, native  # noqa: E402

B1, B2 = 0.9, 0.999
SIZES = [1, 7, 8, 9, 255, 256, 257, 1000, 2048, 4095, 4096, 4097, 12289]


def tensor(n, pdtype, gdtype, bits, master, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = torch.randn(n, device="cuda", generator=g) * 0.05
    grad = (torch.randn(n, device="cuda", generator=g) * torch.exp(2 * torch.randn(n, device="cuda", generator=g)) * 1e-3)
    t = api.adamw_tensor(full.to(pdtype), grad.to(gdtype), bits=bits, master=master)
    if master:
        t.master.copy_(full)
    return t


def state(t):
    return {k: (v.clone() if v is not None else None) for k, v in vars(t).items()}


def expected(s, lr, wd, eps, step, gs=1.0):
    """The step in 64 bits from the tensors of `s` (fp32 states)."""
    g = s["grad"].double().cpu() * gs
    m = s["m"].double().cpu().view(-1) * B1 + (1 - B1) * g
    v = s["v"].double().cpu().view(-1) * B2 + (1 - B2) * g * g
    p0 = (s["master"] if s["master"] is not None else s["param"]).double().cpu()
    upd = lr * (m / (1 - B1 ** step)) / ((v / (1 - B2 ** step)).sqrt() + eps)
    return p0 * (1 - lr * wd) - upd, m, v, upd


def check_param(t, want, upd):
    tol = 3e-7 * want.abs() + 2e-6 * upd.abs() + 1e-12
    if t.master is not None:
        assert bool(((t.master.double().cpu() - want).abs() <= tol).all())
        assert torch.equal(t.param, t.master.bfloat16())
        return
    if t.param.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    assert bool(((t.param.double().cpu() - want).abs() <= tol).all())


@pytest.mark.parametrize("pdtype,gdtype,master", [(torch.bfloat16, torch.bfloat16, False), (torch.bfloat16, torch.float32, False),
                                                  (torch.float32, torch.float32, False), (torch.float32, torch.bfloat16, False),
                                                  (torch.bfloat16, torch.bfloat16, True)])
def test_fp32_states(pdtype, gdtype, master):
    ts = [tensor(n, pdtype, gdtype, 32, master, n) for n in SIZES]
    table = api.adamw_tensors(ts)
    for step in (1, 2, 3):
        before = [state(t) for t in ts]
        api.adamw_step(table, lr=1e-3, weight_decay=0.1, step=step)
        for t, s in zip(ts, before):
            p, m, v, upd = expected(s, 1e-3, 0.1, 1e-8, step)
            g = s["grad"].double().cpu()
            assert bool(((t.m.double().cpu() - m).abs() <= 2e-7 * (s["m"].double().cpu().abs() + g.abs())).all())
            assert bool(((t.v.double().cpu() - v).abs() <= 3e-7 * v + 1e-44).all())
            check_param(t, p, upd)
            assert torch.equal(t.grad, s["grad"])


def encode(x, positive):
    """256 values a block -> e4m3 codes and scales, in fp32 on the host."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256)
    top = b.abs().amax(1, keepdim=True)
    top = torch.where(top >= 2.0 ** -100, top, torch.zeros_like(top))
    y = b * torch.where(top > 0, top.reciprocal() * 448.0, torch.zeros_like(top))
    if positive:
        y = torch.where((b > 0) & (top > 0), y.clamp(min=2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn).view(-1)[:n].view(torch.uint8), (top * (1.0 / 448.0)).view(-1)


def decode(codes, scale):
    x = codes.view(torch.float8_e4m3fn).float()
    return x * scale.repeat_interleave(256)[:x.numel()]


@pytest.mark.parametrize("pdtype,master", [(torch.bfloat16, False), (torch.float32, False), (torch.bfloat16, True)])
def test_8_bit_states(pdtype, master):
    ts = [tensor(n, pdtype, torch.bfloat16, 8, master, n) for n in SIZES]
    f32 = torch.float32
    for step in (1, 2, 3, 4):
        before = [state(t) for t in ts]
        api.adamw_step(ts, lr=1e-3, weight_decay=0.01, step=step)
        for t, s in zip(ts, before):
            g = s["grad"].float().cpu()
            root = decode(s["v"].cpu(), s["v_scale"].cpu())
            m = decode(s["m"].cpu(), s["m_scale"].cpu()) * B1 + g * (1 - B1)
            v = (root * root) * B2 + (g * g) * (1 - B2)
            assert m.dtype == f32 and v.dtype == f32
            for got, scale, want in ((t.m, t.m_scale, encode(m, False)), (t.v, t.v_scale, encode(v.sqrt(), True))):
                assert torch.equal(got.cpu(), want[0]) and torch.equal(scale.cpu(), want[1])
            s["m"], s["v"] = decode(s["m"].cpu(), s["m_scale"].cpu()), root * root
            p, _, _, upd = expected(s, 1e-3, 0.01, 1e-8, step)
            check_param(t, p, upd)


def test_8_bit_extremes():
    """Blocks of zeros, of values near fp32's ends, one large among tiny ones (none of the roots becomes zero), and
    gradients of infinity and NaN (they stay visible)."""
    n = 256 * 6
    t = api.adamw_tensor(torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), bits=8)
    g = t.grad.view(6, 256)
    g[1] = 1e-41
    g[2] = 1e18
    g[3] = 1e-6
    g[3, 5] = 10.0
    g[4, 7] = math.inf
    g[5, 9] = math.nan
    api.adamw_step([t], lr=1e-3, step=1)
    p = t.param.view(6, 256).cpu()
    assert not p[0].count_nonzero() and torch.isfinite(p[:4]).all()
    assert not t.m.view(6, 256)[:2].count_nonzero() and not t.v_scale[:2].count_nonzero()
    assert bool((t.v.view(6, 256)[3] > 0).all())
    assert bool((p[3].abs() <= 1.01e-3).all())
    assert math.isnan(float(p[5, 9])) and torch.isfinite(p[5, :9]).all()
    assert not math.isfinite(float(p[4, 7]))
    # the next step, without gradients: the tiny entries' step stays bounded by the smallest code
    t.grad.zero_()
    before = t.param.clone()
    api.adamw_step([t], lr=1e-3, step=2)
    d = (t.param - before).view(6, 256)[3].cpu()
    assert torch.isfinite(d).all() and float(d.abs().max()) <= 1.1e-3


def test_zero_gradients_leave_zero_states():
    t = api.adamw_tensor(torch.ones(300, device="cuda").bfloat16(), torch.zeros(300, device="cuda").bfloat16())
    api.adamw_step([t], lr=0.5, step=1)
    assert bool((t.param == 1).all()) and not t.m.count_nonzero() and not t.v.count_nonzero()


def test_grad_scale_and_many_tensors():
    """More tensors than a launch's table holds, of both state widths and all types, with a device-side factor."""
    kinds = [(torch.bfloat16, torch.bfloat16, 32, False), (torch.float32, torch.float32, 8, False),
             (torch.bfloat16, torch.float32, 8, True), (torch.float32, torch.bfloat16, 32, False)]
    ts = [tensor(1 + 37 * i % 911, *kinds[i % 4], seed=i) for i in range(900)]
    ts.insert(3, api.adamw_tensor(torch.zeros(0, device="cuda"), torch.zeros(0, device="cuda")))
    before = [state(t) for t in ts]
    api.adamw_step(ts, lr=1e-3, step=1, grad_scale=torch.tensor(0.25, device="cuda"))
    for t, s in zip(ts, before):
        if t.m.dtype == torch.float32 and t.param.numel():
            p, m, v, upd = expected(s, 1e-3, 0.0, 1e-8, 1, 0.25)
            assert bool(((t.m.double().cpu() - m).abs() <= 2e-7 * m.abs() + 1e-44).all())
            check_param(t, p, upd)
        elif t.param.numel():
            s["m"], s["v"] = torch.zeros(t.param.numel()), torch.zeros(t.param.numel())
            p, _, _, upd = expected(s, 1e-3, 0.0, 1e-8, 1, 0.25)
            check_param(t, p, upd)


def test_repeated_and_captured_steps():
    """The same bits from the same state, on another stream and in a graph."""
    ref = None
    for how in ("plain", "stream", "graph"):
        ts = [tensor(n, torch.bfloat16, torch.bfloat16, b, False, n) for n in (5000, 300) for b in (8, 32)]
        table = api.adamw_tensors(ts)
        torch.cuda.synchronize()
        if how == "stream":
            side = torch.cuda.Stream()
            for step in (1, 2):
                api.adamw_step(table, lr=1e-3, step=step, stream=side)
        elif how == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                for step in (1, 2):
                    api.adamw_step(table, lr=1e-3, step=step)
            graph.replay()
        else:
            for step in (1, 2):
                api.adamw_step(table, lr=1e-3, step=step)
        torch.cuda.synchronize()
        got = [x.clone() for t in ts for x in (t.param, t.m, t.v)]
        ref = ref or got
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_training_follows_the_64_bit_optimiser():
    """300 steps on |x - a|^2 / 2 from zero: fp32 states follow AdamW in 64 bits (300 steps of 2e-2 at most, each
    within 1e-5 of its size), and 8-bit states end with a loss within a tenth of the distance covered (their codes
    carry 2^-4 of each value; the errors of successive steps are not aligned)."""
    a = torch.randn(3000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    y, m, v = (torch.zeros(3000, dtype=torch.float64, device="cuda") for _ in range(3))
    for step in range(1, 301):
        g = y - a.double()
        m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
        y = y - 2e-2 * (1 - step / 320) * (m / (1 - B1 ** step)) / ((v / (1 - B2 ** step)).sqrt() + 1e-8)
    first, last = float((a.double() ** 2).sum()), float(((y - a) ** 2).sum())
    for bits in (32, 8):
        x = torch.zeros(3000, device="cuda")
        t = api.adamw_tensor(x, torch.zeros_like(x), bits=bits)
        table = api.adamw_tensors([t])
        for step in range(1, 301):
            t.grad.copy_(x - a)
            api.adamw_step(table, lr=2e-2 * (1 - step / 320), step=step)
        if bits == 32:
            assert float((x - y).abs().max()) < 300 * 2e-2 * 1e-5
        else:
            assert float(((x.double() - a) ** 2).sum()) < last + 0.1 * (first - last)


def test_refusals():
    t = tensor(100, torch.bfloat16, torch.bfloat16, 32, False, 0)

    def refused(status, *args, **kw):
        with pytest.raises(native.LoraError) as e:
            api.adamw_step(*args, **{"lr": 1e-3, "step": 1, **kw})
        assert e.value.status == status

    refused(1, [t], step=0)
    refused(1, [t], beta1=1.0)
    refused(1, [t], beta2=-0.1)
    refused(1, [t], eps=0.0)
    refused(1, [t], lr=math.nan)
    odd = torch.zeros(101, dtype=torch.bfloat16, device="cuda")[1:]
    refused(2, [api.AdamWTensor(odd, t.grad, t.m, t.v)])
    f = tensor(100, torch.float32, torch.float32, 32, False, 0)
    refused(1, [api.AdamWTensor(f.param, f.grad, f.m, f.v, master=torch.zeros(100, device="cuda"))])
    with pytest.raises(ValueError):
        api.adamw_tensors([api.AdamWTensor(t.param, t.grad, t.m.half(), t.v.half())])
    with pytest.raises(ValueError):
        api.adamw_tensors([api.AdamWTensor(t.param, t.grad[:50], t.m, t.v)])
    eight = tensor(600, torch.bfloat16, torch.bfloat16, 8, False, 0)
    with pytest.raises(ValueError):
        api.adamw_tensors([api.AdamWTensor(eight.param, eight.grad, eight.m, eight.v, None, eight.m_scale[:2], eight.v_scale)])
    before = [x.clone() for x in (t.param, t.m, t.v)]
    refused(1, [t, api.AdamWTensor(f.param, f.grad, f.m, f.v, master=torch.zeros(100, device="cuda"))])
    assert all(torch.equal(a, b) for a, b in zip(before, (t.param, t.m, t.v)))   # nothing of a refused call runs


@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_past_32_bits(bits):
    """A tensor of more than 2^31 values: its ends are updated as the same values in a small tensor."""
    n, k = 2 ** 31 + 4096 + 17, 4096 + 17
    g = torch.Generator(device="cuda").manual_seed(4)
    small = [api.adamw_tensor(torch.randn(k, device="cuda", generator=g).bfloat16(),
                              torch.randn(k, device="cuda", generator=g).bfloat16(), bits=bits) for _ in range(2)]
    p, gr = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x, name in ((p, "param"), (gr, "grad")):
        x[:k], x[n - k:] = getattr(small[0], name), getattr(small[1], name)
    big = api.adamw_tensor(p, gr, bits=bits)
    assert (n - k) % 256 == 0
    for step in (1, 2):
        api.adamw_step([big], lr=1e-3, step=step)
        api.adamw_step(small, lr=1e-3, step=step)
    for name in ("param", "m", "v"):
        x = getattr(big, name)
        # the first block after the small tensor's end shares its scale with zeros: the last whole block is compared
        assert torch.equal(x[:4096], getattr(small[0], name)[:4096]) and torch.equal(x[n - k:], getattr(small[1], name))
        assert not x[k:n - k].count_nonzero()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("pdtype,gdtype,master", [(torch.float32, torch.float32, False), (torch.bfloat16, torch.bfloat16, True)])
def test_8_bit_states_beside_a_value_that_is_not_finite(bad, pdtype, gdtype, master):
    """A gradient that is infinite or NaN spoils its own value, as with fp32 states: the others of its block keep the
    states and parameters, bit by bit, that they have where that gradient is zero."""
    n, at = 256 + 256 + 100, (9, 300, 600)
    g = (torch.randn(4, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)) * 1e-3).to(gdtype)
    g[:, at] = 0
    good, spoiled = (api.adamw_tensor(torch.ones(n, device="cuda").to(pdtype), torch.zeros(n, device="cuda").to(gdtype), bits=8,
                                      master=master) for _ in range(2))
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[list(at)] = False
    for step in range(4):
        for t in (good, spoiled):
            t.grad.copy_(g[step])
        if step == 1:
            spoiled.grad[list(at)] = bad
        for t in (good, spoiled):
            api.adamw_step([t], lr=1e-3, step=step + 1)
        for name in ("param", "m", "v", "master"):
            a, b = getattr(good, name), getattr(spoiled, name)
            assert a is None or torch.equal(a[others], b[others]), (name, step)
        assert torch.equal(good.m_scale, spoiled.m_scale) and torch.equal(good.v_scale, spoiled.v_scale)
        if step:
            assert bool(torch.isnan(spoiled.param[~others]).all())
            for codes in (spoiled.m, spoiled.v):
                assert bool(torch.isnan(codes.view(torch.float8_e4m3fn).float()[~others]).all())


def test_8_bit_block_without_a_finite_value():
    t = api.adamw_tensor(torch.ones(512, device="cuda"), torch.full((512,), 1e-3, device="cuda"), bits=8)
    t.grad[:256] = math.nan
    for step in (1, 2):
        api.adamw_step([t], lr=1e-3, step=step)
    assert bool(torch.isnan(t.param[:256]).all()) and bool(torch.isfinite(t.param[256:]).all())
    assert bool(torch.isnan(t.m[:256].view(torch.float8_e4m3fn).float()).all()) and t.m_scale[:1].count_nonzero() == 0
