"""The operators of a fine-tuning step together, as a program calls them: a
Boolean-kernel layer with bias, activation and residual, a Boolean-kernel output
layer, the policy or preference loss, the backward pass, scale gradients and the
optimizer, whose step writes the scales into the packed layers.  Each stage is
checked against float64 on the stage's own inputs; the whole step captured into a
graph, and two steps on two streams, give the bits of the eager one."""
import pytest
import torch

import boolean_weight_amd as bw
import finetune_ref
import step_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

F64, BF = torch.float64, torch.bfloat16
U, EPS = 2.0 ** -8, 2.0 ** -24
GELU = bw.MBOK_ACT_GELU


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


class Model:
    """h = x + gelu(W1 x + b1); logits = W2 h.  W1 [n, n], W2 [V, n]."""

    def __init__(self, T, n, V, K, seed, eight=False):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.T, self.n, self.V = T, n, V
        self.layers = []
        for m in (n, V):
            d = bw.mbok_desc_init(m, n, K, bw.MBOK_F16)
            signs = torch.randint(0, 2, (K, m, n), generator=gen, device=DEV,
                                  dtype=torch.int8) * 2 - 1
            alpha = (0.01 + 0.03 * torch.rand((K, m, n // 128), generator=gen, device=DEV)).half()
            packed = torch.empty(bw.mbok_packed_bytes(d), dtype=torch.uint8, device=DEV)
            bw.mbok_pack(d, signs, alpha, packed)
            self.layers.append(dict(d=d, signs=signs, packed=packed, param=alpha.float(),
                                    grad=torch.zeros_like(alpha, dtype=torch.float32)))
        bf = dict(dtype=BF, device=DEV)
        self.bias = 0.1 * torch.randn(n, generator=gen, device=DEV)
        self.dbias = torch.empty(n, device=DEV)
        self.x = torch.randn(T, n, generator=gen, device=DEV).to(BF)
        self.h, self.pre, self.dpre = (torch.empty(T, n, **bf) for _ in range(3))
        self.Z, self.dZ = torch.empty(T, V, **bf), torch.empty(T, V, **bf)
        self.dh, self.dx = torch.empty(T, n, **bf), torch.empty(T, n, **bf)
        self.label = torch.randint(-1, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
        self.adv = torch.randn(T, generator=gen, device=DEV)
        self.old = -6 + 0.3 * torch.randn(T, generator=gen, device=DEV)
        self.loss, self.logp = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        self.policy = bw.mbok_policy_desc_init(V, kl=0.1)
        tensors = [dict(param=L["param"], grad=L["grad"], out=L["packed"], layer=L["d"],
                        weight_decay=0.01, **self.states(L["param"].numel(), eight))
                   for L in self.layers]
        tensors.append(dict(param=self.bias, grad=self.dbias, **self.states(n, False)))
        self.plan = bw.mbok_adamw_plan_init(tensors)

    @staticmethod
    def states(count, eight):
        if not eight:
            return dict(m=torch.zeros(count, device=DEV), v=torch.zeros(count, device=DEV))
        blocks = (count + bw.MBOK_ADAMW_BLOCK - 1) // bw.MBOK_ADAMW_BLOCK
        f8 = dict(dtype=torch.float8_e4m3fn, device=DEV)
        return dict(m=torch.zeros(count, **f8), v=torch.zeros(count, **f8),
                    m_scale=torch.zeros(blocks, device=DEV), v_scale=torch.zeros(blocks, device=DEV))

    def forward(self, **kw):
        a, b = self.layers
        bw.mbok_linear(a["d"], a["packed"], self.x, self.h, bias=self.bias, act=GELU,
                       residual=self.x, pre=self.pre, **kw)
        bw.mbok_linear(b["d"], b["packed"], self.h, self.Z, **kw)

    def losses(self, **kw):
        bw.mbok_policy(self.policy, self.Z, self.label, self.adv, self.loss, old_logp=self.old,
                       ref_logp=self.old, logp=self.logp, dZ=self.dZ, **kw)

    def backward(self, **kw):
        a, b = self.layers
        bw.mbok_linear_backward(b["d"], b["packed"], self.dZ, dX=self.dh, **kw)
        bw.mbok_scale_grad(b["d"], b["packed"], self.dZ, self.h, b["grad"], **kw)
        bw.mbok_linear_backward(a["d"], a["packed"], self.dh, pre=self.pre, dpre=self.dpre,
                                dbias=self.dbias, dX=self.dx, act=GELU, **kw)
        bw.mbok_scale_grad(a["d"], a["packed"], self.dpre, self.x, a["grad"], **kw)

    def step(self, t=1, live=None, **kw):
        self.forward(**kw)
        self.losses(**kw)
        self.backward(**kw)
        bw.mbok_adamw(self.plan, lr=1e-3, step=t, live=live, seed=3, **kw)

    def state(self):
        out = [self.loss, self.logp, self.dx, self.bias, self.dbias]
        for t in self.plan.tensors:
            out += [v for k, v in t.items() if isinstance(v, torch.Tensor)]
        return [x.clone().view(torch.uint8) for x in out]


def dense(L):
    """The layer as its packed buffer holds it, from the masters."""
    return finetune_ref.dense(L["signs"].cpu(), L["param"].half().cpu())


def f64(x):
    return x.cpu().to(F64)


@pytest.mark.parametrize("T,n,V", [(5, 256, 700), (48, 384, 1001)])
def test_every_stage_of_a_step(T, n, V):
    say(f"training step T={T} n={n} V={V}")
    M = Model(T, n, V, 2, T)
    a, b = M.layers
    for t in (1, 2):  # the second step runs on the scales that the first one wrote
        W1, W2 = dense(a), dense(b)
        bias, masters = f64(M.bias), [L["param"].clone() for L in M.layers]
        M.step(t)
        x, h, Z, dZ = f64(M.x), f64(M.h), f64(M.Z), f64(M.dZ)
        per_weight = U if T > 16 else 2.0 ** -16
        want, z = ref.linear(W1, x, bias, "gelu", x)
        D = (per_weight + n * EPS) * (x.abs() @ W1.abs().t())
        assert ((f64(M.pre) - z).abs() <= D + U * z.abs()).all()
        assert ((h - want).abs() <= 1.13 * D + U * want.abs() + 16 * EPS * z.abs()).all()
        want = h @ W2.t()
        D = (per_weight + n * EPS) * (h.abs() @ W2.abs().t())
        assert ((Z - want).abs() <= D + U * want.abs()).all()
        lp, q = ref.logp(Z, M.label.cpu(), 1.0)
        d = M.policy
        loss, slope, size = ref.policy(lp, M.label.cpu(), V, M.adv.cpu(), M.old.cpu(),
                                       M.old.cpu(), None, float(d.clip_low), float(d.clip_high),
                                       float(d.kl))
        E = 2.0 ** -15 + 2.0 ** -21 * lp.abs()
        assert ((f64(M.loss) - loss).abs() <= E * size + 2.0 ** -22 * loss.abs()).all()
        want = ref.logp_grad(Z, M.label.cpu(), 1.0, slope)
        near = (ref.onehot(M.label.cpu(), V) - q).abs()
        assert ((dZ - want).abs() <= (2.0 ** -16 * q * slope.abs()[:, None] +
                                      (E * size)[:, None] * near + U * want.abs() + 1e-37)).all()
        dh, want = f64(M.dh), dZ @ W2
        assert ((dh - want).abs() <= (U + V * EPS) * (dZ.abs() @ W2.abs()) + U * want.abs()).all()
        dpre, want = f64(M.dpre), dh * ref.act_slope("gelu", f64(M.pre))
        off = 16 * EPS * dh.abs() * (1 + f64(M.pre).abs())
        assert ((dpre - want).abs() <= off + U * want.abs()).all()
        assert ((f64(M.dbias) - want.sum(0)).abs() <=
                (off + (T + 8) * EPS * want.abs()).sum(0)).all()
        want = dpre @ W1
        assert ((f64(M.dx) - want).abs() <= (U + n * EPS) * (dpre.abs() @ W1.abs()) +
                U * want.abs()).all()
        for L, dy, inp, before in ((a, dpre, x, masters[0]), (b, dZ, h, masters[1])):
            want = finetune_ref.scale_grad(L["signs"].cpu(), dy, inp)
            bound = (dy.abs().t() @ inp.abs()).view(L["d"].m, n // 128, 128).sum(-1)
            assert ((f64(L["grad"]) - want).abs() <= (T + 256) * EPS * bound).all()
            # the optimizer moved the masters and the packed scales with them
            assert not torch.equal(L["param"], before)
            bits = L["d"].K * ((L["d"].m + 63) // 64 * 64) * n // 8
            got = L["packed"][bits:].view(torch.float16).cpu()
            want = ref.packed_scales(L["param"].half().cpu(), L["d"]).view(-1)
            inside = ~torch.isnan(want)
            assert torch.equal(got[inside], want[inside])


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T", [1, 12, 200])
def test_step_captured_into_a_graph(T, eight):
    """Replayed four times with eager work between: every replay is the eager step, by
    the constants that are live when it runs."""
    say(f"captured step T={T} eight={eight}")
    eager, held = (Model(T, 256, 513, 3, 7, eight) for _ in range(2))
    live = torch.zeros(4, device=DEV)
    side = torch.cuda.Stream()
    start = held.state()
    tensors = [v for t in held.plan.tensors for v in t.values() if isinstance(v, torch.Tensor)]
    keep = [x.clone() for x in tensors]
    with torch.cuda.stream(side):
        held.step(live=live.fill_(0.0))  # warm
    torch.cuda.synchronize()
    for x, k in zip(tensors, keep):
        x.copy_(k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.step(live=live)
    assert all(torch.equal(x, y) for x, y in zip(start[3:4], held.state()[3:4]))
    for t in (1, 2, 3, 4):
        constants = torch.tensor([1e-3 * t, 0.5, t, 1.0 if t == 3 else 0.0])
        live.copy_(constants)
        graph.replay()
        eager.step(live=constants.to(DEV))
        junk = torch.randn(1 << 20, device=DEV).sum()  # the program's own work
        torch.cuda.synchronize()
        for x, y in zip(eager.state(), held.state()):
            assert torch.equal(x, y), t
        del junk


def test_two_steps_at_once():
    """Two models on two streams, interleaved call by call."""
    say("two streams")
    alone = [Model(40, 256, 513, 2, s) for s in (1, 2)]
    both = [Model(40, 256, 513, 2, s) for s in (1, 2)]
    for M in alone:
        for t in (1, 2, 3):
            M.step(t)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for t in (1, 2, 3):
        for part in ("forward", "losses", "backward"):
            for M, s in zip(both, streams):
                getattr(M, part)(stream=s)
        for M, s in zip(both, streams):
            bw.mbok_adamw(M.plan, lr=1e-3, step=t, seed=3, stream=s)
    torch.cuda.synchronize()
    for A, B in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(A.state(), B.state()))


def test_preference_step_captured():
    say("captured preference step")
    T, V, pairs = 30, 900, 4
    gen = torch.Generator(device=DEV).manual_seed(4)
    Z = torch.randn(T, V, generator=gen, device=DEV).to(BF)
    label = torch.randint(-1, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
    off = torch.tensor([0, 3, 9, 9, 14, 20, 25, 28, 30], dtype=torch.int32, device=DEV)
    d, dp = bw.mbok_logp_desc_init(V), bw.mbok_preference_desc_init(0.2, 0.1, mean=True)
    logp, dlogp, loss = (torch.zeros(k, device=DEV) for k in (T, T, pairs))
    stats, dZ = torch.empty(T, bw.MBOK_LOGP_STATS, device=DEV), torch.empty_like(Z)

    def step():
        bw.mbok_logp(d, Z, label, logp, stats=stats)
        bw.mbok_preference(dp, off, logp, loss, label=label, dlogp=dlogp)
        bw.mbok_logp_backward(d, Z, label, stats, dlogp, dZ)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        Z.copy_(torch.randn(T, V, generator=gen, device=DEV).to(BF))
        graph.replay()
        got = [x.clone() for x in (loss, logp, dlogp, dZ)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (loss, logp, dlogp, dZ))), i
