"""GPU parity of the optimizer step against float64 and, for the codes of the
8-bit states, bit for bit against integer arithmetic on the CPU.

Tolerances in eps = 2^-24, operation by operation: m = b1 m + c1 (c g) rounds the two
constants, three products and the sum: 4 eps (|b1 m| + |c1 c g|).  v = b2 v + c2 x^2:
7 eps v.  p: p (1 - lr wd) rounds twice; the update u = s m / (r d + eps) carries m's
error times s / (r d + eps), r's (v's half, the root's 2 eps), and about 8 roundings and
1-ulp operations: 16 eps |u|; the last rounding eps |p|.
"""
import math

import numpy as np
import pytest
import torch

import boolean_weight_amd as bw
import step_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

F64 = torch.float64
EPS = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
B = bw.MBOK_ADAMW_BLOCK


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def cpu_tensor(count, seed, grad="f32", eight=False):
    """Values and states of very different sizes on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    size = torch.exp(2 * torch.randn(count, generator=gen))
    t = dict(param=torch.randn(count, generator=gen),
             grad=(1e-3 * size * torch.randn(count, generator=gen)).to(TYPES[grad]))
    m, r = 1e-3 * size * torch.randn(count, generator=gen), \
        1e-3 * size * torch.rand(count, generator=gen)
    if not eight:
        return dict(t, m=m, v=r * r)
    blocks = (count + B - 1) // B
    for name, x in (("m", m), ("v", r)):
        pad = torch.nn.functional.pad(x, (0, blocks * B - count)).view(blocks, B)
        scale = torch.exp2(torch.floor(torch.log2(pad.abs().amax(-1).clamp_min(1e-30))) - 7)
        t[name] = (pad / scale[:, None]).view(-1)[:count].to(F8)
        t[name + "_scale"] = scale
    return t


def to_dev(t, off=0):
    """The tensors on the device, `off` elements into buffers of their own."""
    out = {}
    for k, x in t.items():
        if k in ("layer", "weight_decay"):
            out[k] = x
            continue
        bytes_ = x.contiguous().view(torch.uint8)
        buf = torch.zeros(bytes_.numel() + 64, dtype=torch.uint8, device=DEV)
        at = off * x.element_size()
        buf[at:at + bytes_.numel()] = bytes_.to(DEV)
        out[k] = buf[at:at + bytes_.numel()].view(x.dtype)
    return out


def values(code, scale):
    """What codes and scales stand for, in float64 on the CPU."""
    x = code.cpu().to(torch.float32).to(F64)
    return x * scale.cpu().to(F64).repeat_interleave(B)[:len(x)]


def check32(before, after, t, lr, wd=0.0, c=1.0, b1=0.9, b2=0.999, eps=1e-8):
    f = {k: before[k].to(F64) for k in ("param", "grad", "m", "v")}
    p, m, v = ref.adamw(f["param"], f["grad"], f["m"], f["v"], t, lr, b1, b2, eps, wd, c)
    tol_m = 4 * EPS * ((b1 * f["m"]).abs() + ((1 - b1) * c * f["grad"]).abs())
    got = {k: after[k].cpu().to(F64) for k in ("param", "m", "v")}
    assert ((got["m"] - m).abs() <= tol_m + 2.0 ** -140).all()
    assert ((got["v"] - v).abs() <= 7 * EPS * v + 2.0 ** -140).all()
    check_p(got["param"], f["param"], p, m, v, tol_m, t, lr, b1, b2, eps)


def check_p(got, before, p, m, v, tol_m, t, lr, b1, b2, eps):
    step, den = lr / (1 - b1 ** t), (v / (1 - b2 ** t)).sqrt() + eps
    tol = EPS * (4 * before.abs() + p.abs() + 16 * step * (m / den).abs()) + step / den * tol_m
    assert ((got - p).abs() <= tol + 2.0 ** -140).all(), ((got - p).abs() - tol).max()


COUNTS = [1, 3, 4, 255, 256, 257, 1000, 1024, 1025, 4096, 5000, 70001]


@pytest.mark.parametrize("grad", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
def test_many_tensors_32bit(grad, off):
    say(f"adamw 32-bit {grad} offset {off}")
    cpu, outs = [], [None, "f32", "f16", "bf16"]
    for i, c in enumerate(COUNTS):
        t = cpu_tensor(c, 10 + i, grad)
        if outs[i % 4]:
            t["out"] = torch.full((c,), -5.0, dtype=TYPES[outs[i % 4]])
        if i % 3 == 0:
            t["weight_decay"] = 0.05
        cpu.append(t)
    gpu = [to_dev(t, off) for t in cpu]
    plan = bw.mbok_adamw_plan_init(gpu)
    bw.mbok_adamw(plan, lr=1e-3, step=3, grad_scale=0.25)
    for before, after in zip(cpu, gpu):
        check32(before, after, 3, 1e-3, before.get("weight_decay", 0.0), 0.25)
        assert torch.equal(after["grad"].cpu(), before["grad"])
        if "out" in after:
            assert torch.equal(after["out"], after["param"].to(after["out"].dtype))


@pytest.mark.parametrize("t", [1, 2, 1000, 1 << 40])
@pytest.mark.parametrize("b1,b2", [(0.9, 0.999), (0.0, 0.5), (0.95, 0.0)])
def test_steps_and_constants(t, b1, b2):
    say(f"adamw step {t} betas {b1} {b2}")
    before = cpu_tensor(3000, 5)
    if t == 1:
        before["m"].zero_(), before["v"].zero_()
    after = to_dev(before)
    bw.mbok_adamw(bw.mbok_adamw_plan_init([after]), lr=2e-3, step=t, beta1=b1, beta2=b2, eps=1e-6)
    check32(before, after, t, 2e-3, b1=b1, b2=b2, eps=1e-6)


def check8(before, after, place, t, seed, lr, wd=0.0, c=1.0, b1=0.9, b2=0.999, eps=1e-8):
    m0, r0 = values(before["m"], before["m_scale"]), values(before["v"], before["v_scale"])
    p0, g = before["param"].to(F64), before["grad"].to(F64)
    p, m, v = ref.adamw(p0, g, m0, r0 * r0, t, lr, b1, b2, eps, wd, c)
    tol_m = 4 * EPS * ((b1 * m0).abs() + ((1 - b1) * c * g).abs())
    check_p(after["param"].cpu().to(F64), p0, p, m, v, tol_m, t, lr, b1, b2, eps)
    # the states: within one step of a code (2^-3 of the value, 2^-9 of the scale), and
    # no root that is not 0 lost
    for name, want in (("m", m), ("v", v.sqrt())):
        scale = after[name + "_scale"].cpu().to(F64).repeat_interleave(B)[:len(want)]
        got = values(after[name], after[name + "_scale"])
        step = torch.maximum(want.abs() / 8, scale * 2.0 ** -9)
        assert ((got - want).abs() <= step * (1 + 2.0 ** -10)).all()
    assert (values(after["v"], after["v_scale"])[v > 1e-40] > 0).all()
    # bit for bit: the moments by the same float32 operations, one at a time
    f = np.float32
    m32, r32 = m0.numpy().astype(f), r0.numpy().astype(f)
    x = before["grad"].float().numpy() * f(c)
    m32 = m32 * f(b1) + x * f(1 - b1)
    r32 = np.sqrt((r32 * r32) * f(b2) + (x * x) * f(1 - b2))
    low, high = ref.random_bits(len(x), place, t, seed)
    for name, val, rnd, least in (("m", m32, low, 0), ("v", r32, high, 1)):
        codes, scales = ref.encode(val, rnd, least)
        assert np.array_equal(after[name + "_scale"].cpu().numpy(), scales)
        assert np.array_equal(after[name].cpu().view(torch.uint8).numpy(), codes)


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
def test_many_tensors_8bit(grad, off):
    say(f"adamw 8-bit {grad} offset {off}")
    cpu = [cpu_tensor(c, 40 + i, grad, eight=True) for i, c in enumerate(COUNTS[:-1])]
    cpu.insert(3, cpu_tensor(777, 2, grad))  # one with 32-bit states among them
    gpu = [to_dev(t, off) for t in cpu]
    bw.mbok_adamw(bw.mbok_adamw_plan_init(gpu), lr=1e-3, step=7, seed=99, grad_scale=0.5)
    for i, (before, after) in enumerate(zip(cpu, gpu)):
        if i == 3:
            check32(before, after, 7, 1e-3, c=0.5)
        else:
            check8(before, after, i, 7, 99, 1e-3, c=0.5)


def test_8bit_ranges():
    """Blocks of zeros, of one size, of sizes 2^40 apart, of subnormals; a value that is
    not finite makes its block's scale NaN and no other's."""
    say("adamw 8-bit ranges")
    n = 8 * B
    before = cpu_tensor(n, 3, eight=True)
    g = torch.zeros(8, B)
    g[1] = 1e-3
    g[2] = torch.exp2(-torch.arange(B) * 40.0 / B)
    g[3] = 1e-30
    g[4] = 1e-42
    g[5] = 1e18
    g[6, 7] = math.inf
    g[7, 9] = math.nan
    before["grad"] = g.view(-1)
    for k in ("m", "v"):
        before[k] = torch.zeros(n).to(F8)
        before[k + "_scale"] = torch.ones(8)
    after = to_dev(before)
    bw.mbok_adamw(bw.mbok_adamw_plan_init([after]), lr=1e-3, step=1, seed=4)
    low, high = ref.random_bits(n, 0, 1, 4)
    f = np.float32
    x = g.view(-1).numpy()
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        m32, r32 = x * f(1 - 0.9), np.sqrt((x * x) * f(1 - 0.999))
    for name, val, rnd, least in (("m", m32, low, 0), ("v", r32, high, 1)):
        codes, scales = ref.encode(val, rnd, least)
        got = after[name + "_scale"].cpu().numpy()
        assert np.array_equal(got, scales, equal_nan=True)
        assert np.isnan(got[6:]).all() and np.isfinite(got[:6]).all()
        got = after[name].cpu().view(torch.uint8).numpy()
        assert np.array_equal(got[:6 * B], codes[:6 * B])
    p = after["param"].cpu()
    bad = ~torch.isfinite(p)
    assert bad[7 * B + 9] and int(bad.sum()) <= 2
    assert torch.equal(p[:B], before["param"][:B])  # no gradient, no decay
    # the next step: a NaN scale is its whole block's state, and no other block's
    bw.mbok_adamw(bw.mbok_adamw_plan_init([after]), lr=1e-3, step=2, seed=4)
    bad = ~torch.isfinite(after["param"].cpu()).view(8, B)
    assert bad[6:].all() and not bad[:6].any()


def test_8bit_second_moment_moves():
    """With gradients that shrink a hundredfold the second moment follows, as nearest
    rounding of an update of a thousandth never would.  Without a gradient a step takes r
    to sqrt(b2) r, a distance of at most d = (1 - sqrt(b2)) r < 0.00051 r below a code,
    whose step s is r / 16 to r / 8; stochastic rounding keeps the mean and adds a variance
    f (1 - f) s^2 with f = d / s, at most d s <= 0.00051 / 8 r^2.  So the mean of v = r^2
    falls by a factor of 0.999 to 0.999 + 6.4e-5 per step: after 3000 steps it is 1 to
    exp(0.192) = 1.22 times 0.999^3000 of the start (and the small gradient's part).  The
    mean over 4096 values of a relative deviation below 1: 5 / 64 either way."""
    say("adamw 8-bit second moment")
    n = 4096
    t = cpu_tensor(n, 6, eight=True)
    t["grad"] = torch.full((n,), 1e-4)
    t["v"], t["v_scale"] = torch.full((n,), 128.0).to(F8), torch.full((n // B,), 2.0 ** -14)
    t["m"] = torch.zeros(n).to(F8)
    after = to_dev(t)
    plan = bw.mbok_adamw_plan_init([after])
    for step in range(1, 3001):
        bw.mbok_adamw(plan, lr=0.0, step=step, seed=1)
    got = float((values(after["v"], after["v_scale"]) ** 2).mean())
    start = (128 * 2.0 ** -14) ** 2
    want = start * 0.999 ** 3000 + 1e-8 * (1 - 0.999 ** 3000)
    assert want * (1 - 5 / 64) <= got <= 1.22 * want * (1 + 5 / 64), (got, want)


LAYERS = [(1, 128, 1, "f16"), (64, 256, 2, "f32"), (65, 128, 3, "f16"), (100, 4096, 2, "f16"),
          (1000, 11008, 1, "f32"), (37, 1 << 18, 1, "f16"), (3, 1 << 20, 2, "f16"),
          (5000, 640, 4, "f16"), (129, 128, 4, "f32")]


@pytest.mark.parametrize("eight", [False, True])
def test_layers(eight):
    """Scales go into the packed buffers, rounded once; signs and padding stay."""
    cpu, descs = [], []
    for i, (m, n, K, dt) in enumerate(LAYERS):
        say(f"adamw layer {m}x{n} K={K} {dt} eight={eight}")
        d = bw.mbok_desc_init(m, n, K, bw.MBOK_F16 if dt == "f16" else bw.MBOK_F32)
        t = cpu_tensor(K * m * (n // 128), 70 + i, eight=eight)
        t["weight_decay"] = 0.01
        if n < 1 << 18:
            t["out"] = torch.randint(0, 256, (bw.mbok_packed_bytes(d),), dtype=torch.uint8,
                                     generator=torch.Generator().manual_seed(i))
        else:
            t["out"] = torch.full((bw.mbok_packed_bytes(d),), 0x5A, dtype=torch.uint8)
        cpu.append(t)
        descs.append(d)
    gpu = [dict(to_dev(t), layer=d) for t, d in zip(cpu, descs)]
    bw.mbok_adamw(bw.mbok_adamw_plan_init(gpu), lr=1e-2, step=5, seed=3)
    for i, (before, after, d) in enumerate(zip(cpu, gpu, descs)):
        if eight:
            check8(before, after, i, 5, 3, 1e-2, 0.01)
        else:
            check32(before, after, 5, 1e-2, 0.01)
        at = torch.float16 if d.alpha_dtype == bw.MBOK_F16 else torch.float32
        bits = d.K * ((d.m + 63) // 64 * 64) * d.n // 8
        got, was = after["out"].cpu(), before["out"]
        assert torch.equal(got[:bits], was[:bits])
        want = ref.packed_scales(after["param"].cpu().to(at), d).view(-1)
        padding = torch.isnan(want)
        want[padding] = was[bits:].view(at)[padding]
        assert torch.equal(got[bits:], want.view(torch.uint8))


def test_live_constants_and_skipped_steps():
    say("adamw live")
    before = cpu_tensor(5000, 8)
    eight = cpu_tensor(2000, 9, eight=True)
    runs = []
    for live in (None, torch.tensor([0.5 ** 10, 0.5, 12.0, 0.0], device=DEV)):
        a, b = to_dev(before), to_dev(eight)
        kw = dict(lr=0.5 ** 10, step=12, grad_scale=0.5) if live is None else \
            dict(lr=7.0, step=3, grad_scale=9.0, live=live)
        bw.mbok_adamw(bw.mbok_adamw_plan_init([a, b]), seed=5, **kw)
        runs.append((a, b))
    check32(before, runs[1][0], 12, 0.5 ** 10, c=0.5)
    check8(eight, runs[1][1], 1, 12, 5, 0.5 ** 10, c=0.5)
    for x, y in zip(*runs):
        for k in x:
            assert torch.equal(x[k].view(torch.uint8), y[k].view(torch.uint8))
    skip = to_dev(before)
    plan = bw.mbok_adamw_plan_init([skip])
    bw.mbok_adamw(plan, lr=1.0, step=1, live=torch.tensor([1.0, 1.0, 1.0, 1.0], device=DEV))
    for k in ("param", "m", "v"):
        assert torch.equal(skip[k].cpu(), before[k])


def test_binding_refusals():
    t = to_dev(cpu_tensor(300, 1))
    e = to_dev(cpu_tensor(300, 1, eight=True))
    good = dict(t)
    for kw in (dict(param=t["param"].half()), dict(grad=t["grad"][:-1]), dict(m=t["m"][:-1]),
               dict(grad=t["grad"].double()), dict(m=e["m"]), dict(m_scale=e["m_scale"]),
               dict(out=t["param"].double().clone()), dict(out=torch.empty(299, device=DEV)),
               dict(param=torch.empty(600, device=DEV)[::2]), dict(more=1),
               dict(layer=bw.mbok_desc_init(64, 128, 1))):
        with pytest.raises((ValueError, TypeError)):
            bw.mbok_adamw_plan_init([dict(good, **kw)])
    for kw in (dict(m_scale=e["m_scale"][:1]), dict(v=t["v"]), dict(v_scale=None)):
        with pytest.raises(ValueError):
            bw.mbok_adamw_plan_init([dict(e, **kw)])
    with pytest.raises(bw.MbokError) as err:
        bw.mbok_adamw_plan_init([good, good])
    assert err.value.status == -1
