"""GPU parity of the distillation loss and its gradient (mbok_distill,
mbok_distill_backward) against the float64 reference, through the C ABI.

Tolerances, derived (eps = 2^-24, the fp32 half step):
  loss   The exponentials of a row are summed in fp32 per thread (at most 128
         terms before float64) and each carries the hardware exponential's 1
         ulp = 2 eps; log2(e) / tau in fp32 moves log S by at most eps / 2 log V: log S is off by at most
         ~ 130 eps in the worst case, the listed p by ~ 8 eps relative.  So
         |loss - ref| <= w tau^2 (2^-16 + 2^-20 (|kl| + spread)), where spread
         bounds |log p - log q| over the listed entries with p > 0.
  dZ     q and p carry at most 2^-16 relative (the argument (z - max) / tau,
         below 2^7 where q > 2^-126 q_max, rounds to 2^-24 2^7 = 2^-17, plus
         log S), then one rounding to the gradient's type, eps_t / 2 of the
         value, or half its smallest step near zero.
"""
import math

import pytest
import torch

import boolean_weight_amd as bw
import finetune_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

F64 = torch.float64
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def inputs(T, V, top, z, seed, scale=2.5):
    """Student and teacher logits; distinct listed tokens (top <= V)."""
    gen = torch.Generator().manual_seed(seed)
    teacher = torch.randn(T, V, generator=gen) * scale
    Z = (teacher + torch.randn(T, V, generator=gen)).to(TYPES[z])
    l, idx = teacher.topk(top, -1)
    return Z, l.contiguous(), idx.to(torch.int32).contiguous(), teacher


def dev(x):
    return None if x is None else x.to(DEV)


def check(got_loss, got_dz, Z, l, idx, tau, lse=None, w=None, dloss=None):
    loss, dZ = ref.distill(Z, l, idx, tau, lse, w)
    got = got_loss.cpu().to(F64)
    wt = torch.ones(Z.shape[0], dtype=F64) if w is None else w.to(F64)
    spread = (l.to(F64)[l > -math.inf].abs().max() * 2 + Z.to(F64)[Z > -math.inf].abs().max() * 2) \
        / tau + math.log(Z.shape[1])
    finite = torch.isfinite(loss)
    assert torch.equal(torch.isnan(loss), torch.isnan(got))
    assert torch.equal(loss[torch.isinf(loss)], got[torch.isinf(loss)])
    tol = wt.abs() * tau * tau * (2.0 ** -16 + 2.0 ** -20 * spread) + 2.0 ** -20 * loss.abs()
    assert (((got - loss).abs() <= tol) | ~finite).all(), (got - loss).abs().max()
    if got_dz is None:
        return
    if dloss is not None:
        dZ = dZ * dloss.to(F64)[:, None]
        wt = wt * dloss.to(F64)
    g = got_dz.cpu().to(F64)
    assert torch.equal(torch.isnan(dZ), torch.isnan(g))
    info = torch.finfo(got_dz.dtype)
    # q and p are at most 1: what cancels in q - p is off by 2^-16 of them
    q = torch.softmax(Z.to(F64) / tau, -1)
    pq = (wt * tau).abs()[:, None] * (q + torch.zeros_like(q).scatter_add(
        1, idx.long().clamp(0, Z.shape[1] - 1),
        torch.where((idx >= 0) & (idx < Z.shape[1]), listed_p(l, idx, tau, lse, Z.shape[1]), 0.0)))
    tol = 2.0 ** -16 * torch.maximum(pq, dZ.abs()) + info.eps / 2 * dZ.abs() + info.smallest_normal
    if info.dtype == "float16":
        tol = tol + 2.0 ** -25
    ok = ((g - dZ).abs() <= tol) | ~torch.isfinite(dZ)
    assert ok.all(), ((g - dZ).abs() - tol).max()


def listed_p(l, idx, tau, lse, V):
    x = torch.where((idx >= 0) & (idx < V), l.to(F64) / tau, -math.inf)
    if lse is None:
        top = x.max(-1, keepdim=True).values
        x = x - torch.where(top > -math.inf, torch.logsumexp(x, -1, keepdim=True), 0.0)
    else:
        x = x - lse.to(F64)[:, None]
    return x.exp()


def run(Z, l, idx, tau, lse=None, w=None, grad="same", mode="step", dloss=None):
    T, V = Z.shape
    d = bw.mbok_distill_desc_init(V, l.shape[1], tau)
    Zd, ld, idxd = dev(Z), dev(l), dev(idx)
    loss = torch.full((T,), -5.0, device=DEV)
    dt = Z.dtype if grad == "same" else torch.bfloat16
    dZ = torch.full((T, V), -7.0, dtype=dt, device=DEV)
    kw = dict(t_lse=dev(lse), weight=dev(w))
    if mode == "step":
        bw.mbok_distill(d, Zd, ld, idxd, loss, dZ=dZ, **kw)
        return loss, dZ
    stats = torch.full((T, bw.MBOK_DISTILL_STATS), float("nan"), device=DEV)
    bw.mbok_distill(d, Zd, ld, idxd, loss, stats=stats, **kw)
    dl = torch.ones(T, device=DEV) if dloss is None else dev(dloss)
    bw.mbok_distill_backward(d, Zd, ld, idxd, stats, dl, dZ, **kw)
    return loss, dZ


# vocabularies around the vector width, a wavefront's share, each number of
# vectors per thread, and past what the registers hold (read again)
SHAPES = [(1, 1, 1), (3, 7, 3), (2, 8, 8), (5, 63, 5), (4, 512, 16), (3, 513, 64), (2, 2049, 20),
          (2, 4100, 33), (3, 8200, 7), (2, 17000, 64), (2, 33001, 128), (1, 70001, 1024),
          (1, 140003, 50), (1, bw.MBOK_MAX_VOCAB, 3)]


@pytest.mark.parametrize("T,V,top", SHAPES)
@pytest.mark.parametrize("rest", [False, True])
def test_distill_shapes(T, V, top, rest):
    for z, grad, tau in (("f32", "same", 1.0), ("bf16", "same", 2.0), ("f16", "bf16", 4.0)):
        say(f"distill T={T} V={V} top={top} rest={rest} {z}->{grad} tau={tau}")
        Z, l, idx, teacher = inputs(T, V, top, z, 3 * V + top)
        lse = torch.logsumexp(teacher / tau, -1) if rest else None
        dl = torch.linspace(0.5, 2.0, T)
        check(*run(Z, l, idx, tau, lse, grad=grad), Z, l, idx, tau, lse)
        check(*run(Z, l, idx, tau, lse, grad=grad, mode="pair", dloss=dl), Z, l, idx, tau, lse,
              dloss=dl)


@pytest.mark.parametrize("z,grad", [("f32", "same"), ("f32", "bf16"), ("f16", "same"),
                                    ("f16", "bf16"), ("bf16", "same")])
@pytest.mark.parametrize("td", ["f32", "f16", "bf16"])
def test_distill_types(z, grad, td):
    say(f"distill types {z}->{grad} teacher {td}")
    Z, l, idx, teacher = inputs(6, 1000, 20, z, 77)
    l = l.to(TYPES[td])
    for lse in (None, torch.logsumexp(teacher, -1)):
        check(*run(Z, l, idx, 1.0, lse, grad=grad), Z, l, idx, 1.0, lse)
        check(*run(Z, l, idx, 1.0, lse, grad=grad, mode="pair"), Z, l, idx, 1.0, lse)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_missing_repeated_and_weightless(rest):
    """Short lists, an empty list, indices past V, an index listed twice and
    three times, a list of -inf, rows of weight 0."""
    say(f"distill lists rest={rest}")
    T, V, top = 9, 300, 6
    Z, l, idx, teacher = inputs(T, V, top, "f32", 21)
    idx[1, 3:] = -1
    idx[2, :] = -1
    idx[3, 2] = V
    idx[3, 4] = 1 << 30
    idx[4, 5] = idx[4, 0]
    idx[5, 1] = idx[5, 2] = idx[5, 3]
    l[6, :] = -math.inf
    l[7, 2] = -math.inf
    idx[7, 0] = -(1 << 31)
    lse = torch.logsumexp(teacher, -1) if rest else None
    w = torch.tensor([1.0, 0.5, 1.0, 1.0, 2.0, 1.0, 1.0, 1.0, 0.0])
    for mode in ("step", "pair"):
        loss, dZ = run(Z, l, idx, 1.0, lse, w, mode=mode)
        check(loss, dZ, Z, l, idx, 1.0, lse, w)
        assert float(loss[8]) == 0.0 and not dZ[8].any()
        if not rest:
            for t in (2, 6):
                assert float(loss[t]) == 0.0 and not dZ[t].any()


def test_distill_every_token_listed():
    """Nothing is left for the rest: the two forms agree."""
    say("distill all listed")
    V = 24
    Z, l, idx, teacher = inputs(3, V, V, "f32", 5)
    lse = torch.logsumexp(teacher, -1)
    check(*run(Z, l, idx, 1.0, lse), Z, l, idx, 1.0, lse)
    check(*run(Z, l, idx, 1.0), Z, l, idx, 1.0)


def test_distill_masked_vocabulary_and_bad_rows():
    """-inf masks (as the type's lowest value too), a listed token the student
    rules out (+inf), rows of NaN, +inf and only -inf: NaN, and only there."""
    say("distill masks")
    T, V, top = 8, 777, 9
    Z, l, idx, _ = inputs(T, V, top, "f32", 31)
    free = [v for v in range(V) if v not in set(idx[0].tolist()) | set(idx[1].tolist())]
    Z[0, free[:500]] = -math.inf
    Z[1, free[:500]] = torch.finfo(torch.float32).min
    Z[2, int(idx[2, 3])] = -math.inf
    Z[3, 400] = math.nan
    Z[4, 5] = math.inf
    Z[5, :] = -math.inf
    Z[6, V - 1] = math.nan
    for mode in ("step", "pair"):
        loss, dZ = run(Z, l, idx, 1.0, mode=mode)
        loss, dZ = loss.cpu(), dZ.cpu()
        keep = [0, 1, 7]
        check(loss[keep], dZ[keep], Z[keep], l[keep], idx[keep], 1.0)
        assert math.isinf(float(loss[2])) and float(loss[2]) > 0
        assert torch.isnan(loss[[3, 4, 5, 6]]).all()
        assert torch.isfinite(dZ[2]).all()
        assert torch.isnan(dZ[[3, 4, 5, 6]]).all()


@pytest.mark.parametrize("shift", [-3000.0, 300.0, 3.0e4])
def test_distill_large_logits(shift):
    """Logits far from zero: only differences count (as far as the type keeps
    them: the reference takes the rounded logits)."""
    for z in ("f32", "f16", "bf16"):
        say(f"distill shift {shift} {z}")
        Z, l, idx, teacher = inputs(3, 900, 12, "f32", 19)
        Z = (Z + shift).to(TYPES[z])
        lse = torch.logsumexp(teacher, -1)
        for t_lse in (None, lse):
            check(*run(Z, l, idx, 1.0, t_lse), Z, l, idx, 1.0, t_lse)
            check(*run(Z, l, idx, 1.0, t_lse, mode="pair"), Z, l, idx, 1.0, t_lse)


def test_distill_largest_values():
    """The type's largest finite logits: the row's mass is on them."""
    say("distill largest values")
    for z in ("f32", "bf16", "f16"):
        big = torch.finfo(TYPES[z]).max
        Z = torch.zeros(2, 100, dtype=TYPES[z])
        Z[0, 7], Z[1, 3], Z[1, 50] = big, big, big
        l, idx = torch.zeros(2, 2), torch.tensor([[7, 9], [3, 50]], dtype=torch.int32)
        loss, dZ = run(Z, l, idx, 1.0)
        want = torch.zeros(2, 100)
        want[0, 7], want[0, 9] = 0.5, -0.5
        assert torch.equal(dZ.cpu().float(), want)


def test_distill_longest_list_of_the_largest_vocabulary():
    say("distill largest")
    V, top = bw.MBOK_MAX_VOCAB, bw.MBOK_MAX_TOP
    Z, l, idx, teacher = inputs(1, V, top, "bf16", 3)
    idx[0, 5] = idx[0, 900]
    lse = torch.logsumexp(teacher, -1)
    check(*run(Z, l, idx, 1.0, lse), Z, l, idx, 1.0, lse)


def test_distill_strides_and_neighbours():
    """Rows at odd elements inside wider buffers: nothing outside is written."""
    say("distill strides")
    for z in ("f32", "bf16"):
        T, V, top = 4, 1001, 12
        Z, l, idx, _ = inputs(T, V, top, z, 41)
        wide = torch.full((T, 1030), 3.0, dtype=Z.dtype)
        wide[:, 3:3 + V] = Z
        lw, iw = torch.zeros(T, 17), torch.zeros(T, 17, dtype=torch.int32)
        lw[:, 2:2 + top], iw[:, 2:2 + top] = l, idx
        d = bw.mbok_distill_desc_init(V, top, 1.0)
        out = torch.full((T, 1040), -9.0, dtype=Z.dtype, device=DEV)
        loss = torch.empty(T, device=DEV)
        bw.mbok_distill(d, dev(wide)[:, 3:3 + V], dev(lw)[:, 2:2 + top], dev(iw)[:, 2:2 + top],
                        loss, dZ=out[:, 5:5 + V])
        check(loss, out[:, 5:5 + V], Z, l, idx, 1.0)
        assert (out[:, :5] == -9).all() and (out[:, 5 + V:] == -9).all()


@pytest.mark.parametrize("V", [900, 33001, 140003])
def test_distill_in_place(V):
    """dZ may be Z: the same bits as into another buffer."""
    say(f"distill in place V={V}")
    Z, l, idx, teacher = inputs(3, V, 10, "bf16", V)
    lse = dev(torch.logsumexp(teacher, -1))
    d = bw.mbok_distill_desc_init(V, 10, 1.0)
    loss, other = run(Z, l, idx, 1.0, lse.cpu())
    Zd, loss2 = dev(Z), torch.empty(3, device=DEV)
    bw.mbok_distill(d, Zd, dev(l), dev(idx), loss2, dZ=Zd, t_lse=lse)
    assert torch.equal(loss, loss2) and torch.equal(other, Zd)
    stats = torch.empty(3, bw.MBOK_DISTILL_STATS, device=DEV)
    Zd = dev(Z)
    bw.mbok_distill(d, Zd, dev(l), dev(idx), loss2, stats=stats, t_lse=lse)
    bw.mbok_distill_backward(d, Zd, dev(l), dev(idx), stats, torch.ones(3, device=DEV), Zd,
                             t_lse=lse)
    assert torch.equal(other, Zd)


def test_distill_differences():
    """The gradient against central differences of the call's own loss.  With
    h = 2^-5 the third derivative (below 1 for q (1 - q) ..) leaves h^2 / 6 <
    2e-4, and the fp32 loss (below 8, off by 2^-18) adds 2^-18 / h = 2^-13."""
    say("distill differences")
    V, top, h = 40, 5, 2.0 ** -5
    Z, l, idx, teacher = inputs(1, V, top, "f32", 9, scale=1.0)
    lse = torch.logsumexp(teacher, -1)
    for t_lse in (None, lse):
        many = Z.repeat(2 * V, 1)
        for v in range(V):
            many[2 * v, v] += h
            many[2 * v + 1, v] -= h
        rep = lambda x: None if x is None else x.repeat(2 * V, *[1] * (x.dim() - 1))  # noqa: E731
        loss, _ = run(many, rep(l), rep(idx), 1.0, rep(t_lse))
        loss = loss.cpu().to(F64).view(V, 2)
        _, dZ = run(Z, l, idx, 1.0, t_lse)
        diff = (loss[:, 0] - loss[:, 1]) / (2 * h)
        assert (diff - dZ[0].cpu()).abs().max() < 4e-4


def test_distill_many_rows_graph_and_streams():
    """Captured and replayed with other work between, on two streams at once,
    and twice in a row: the eager bits every time."""
    say("distill graph and streams")
    T, V, top = 700, 2000, 32
    Z, l, idx, _ = inputs(T, V, top, "bf16", 55)
    d = bw.mbok_distill_desc_init(V, top, 2.0)
    Zd, ld, idxd = dev(Z), dev(l), dev(idx)
    w = torch.full((T,), 1.0 / T, device=DEV)
    loss, dZ = torch.empty(T, device=DEV), torch.empty_like(Zd)

    def go(loss=loss, dZ=dZ, z=Zd):
        bw.mbok_distill(d, z, ld, idxd, loss, dZ=dZ, weight=w)

    go()
    want = loss.clone(), dZ.clone()
    check(loss, dZ, Z, l, idx, 2.0, w=w.cpu())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    other = torch.empty(T, device=DEV), torch.empty_like(Zd)
    for _ in range(4):
        loss.fill_(-1), dZ.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(dZ, want[1])
        go(*other, z=Zd.flip(0))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [(torch.empty(T, device=DEV), torch.empty_like(Zd)) for _ in streams]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        bw.mbok_distill(d, Zd, ld, idxd, o[0], dZ=o[1], weight=w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


def test_distill_most_rows():
    """The most rows a call takes, of 8 tokens each: every row against the same
    formulas in float64."""
    T, V = bw.MBOK_MAX_DISTILL_ROWS, 8
    say(f"distill T={T} V={V}")
    gen = torch.Generator(device=DEV).manual_seed(5)
    Z = torch.randn(T, V, generator=gen, device=DEV, dtype=torch.float32)
    l = torch.zeros(T, 1, device=DEV)
    idx = torch.randint(0, V, (T, 1), generator=gen, device=DEV, dtype=torch.int32)
    d = bw.mbok_distill_desc_init(V, 1, 1.0)
    loss = torch.full((T,), -5.0, device=DEV)
    stats = torch.empty(T, bw.MBOK_DISTILL_STATS, device=DEV)
    dZ, dZ2 = torch.empty_like(Z), torch.empty_like(Z)
    bw.mbok_distill(d, Z, l, idx, loss, stats=stats, dZ=dZ)
    bw.mbok_distill_backward(d, Z, l, idx, stats, torch.ones(T, device=DEV), dZ2)
    logq = torch.log_softmax(Z.to(F64), -1)
    want = -logq.gather(1, idx.long())[:, 0]
    # |log q| < 16: 2^-16 and 2^-20 of it, as above
    assert ((loss.to(F64) - want).abs() <= 2.0 ** -15).all()
    grad = logq.exp()
    grad.scatter_add_(1, idx.long(), torch.full((T, 1), -1.0, dtype=F64, device=DEV))
    for g in (dZ, dZ2):
        assert ((g.to(F64) - grad).abs() <= 2.0 ** -15).all()
