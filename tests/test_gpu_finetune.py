"""GPU parity of the gated feed-forward block (forward, backward), the
transposed product for several tokens and the scale gradients, through the C
ABI, against float64.

Exact regime (integer activations in [-8, 8], scales 2^-e with e in 4..8):
every W_hat level has at most 8 significant bits and every partial sum is a
multiple of 2^-8 below 2^16, so all products and sums are exact and a result
differs from the float64 one by its single rounding alone (none for fp32).

Otherwise, with u = 2^-8 the relative half step of bf16: a W_hat level and an
output each round by at most u relative, and fp32 sums of c terms by c 2^-24
of the absolute sum, so |y - ref| <= (u + c 2^-24) sum |W_hat| |x| + u |y|.
"""
import numpy as np
import pytest
import torch

import boolean_weight_amd as bw
import finetune_ref as ref
import mbok_synth as syn
from gpu_util import DEV, alpha_enum, np_alpha, pack_on_gpu, say, to_dev

pytestmark = pytest.mark.gpu

F64, BF = torch.float64, torch.bfloat16
U = 2.0 ** -8
ACTS = {"silu": bw.MBOK_ACT_SILU, "gelu": bw.MBOK_ACT_GELU}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def exact_layer(m, n, K, dt, seed):
    S = syn.random_signs(K, m, n, seed=seed)
    return S, syn.exact_alpha(K, m, n // 128, seed=seed + 1).astype(np_alpha(dt))


def gauss_layer(m, n, K, dt, seed):
    """Scales with full significands, of both signs now and then (a refit)."""
    rng = np.random.default_rng(seed)
    A = rng.normal(0.01, 0.006, size=(K, m, n // 128))
    return syn.random_signs(K, m, n, seed=seed), A.astype(np_alpha(dt))


def ints(T, n, seed):
    return torch.from_numpy(syn.exact_activations(T, n, seed=seed))


def gauss(T, n, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(T, n, generator=gen) * scale).to(BF).float()


def wide(x, ld, fill=float("nan"), off=0):
    """x as bf16 rows of a [T, ld] device buffer full of `fill`."""
    buf = torch.full((x.shape[0], ld), fill, dtype=BF, device=DEV)
    buf[:, off:off + x.shape[1]] = x.to(BF).to(DEV)
    return buf[:, off:off + x.shape[1]]


def bf16_of(x):
    return x.to(F64).float().to(BF).to(F64)  # exact in fp32 by construction, one rounding


def garbage(nbytes):
    return torch.full((max(nbytes, 256) // 4 + 64,), float("nan"), device=DEV)


def gated_layer(a, b, dt):
    K, m, n = a[0].shape
    d = bw.mbok_desc_init(m, n, K, alpha_enum(dt))
    packed = torch.full((bw.mbok_packed_bytes(bw.mbok_gated_stack(d)),), 0xA5, dtype=torch.uint8,
                        device=DEV)
    bw.mbok_gated_pack(d, to_dev(a[0]), to_dev(a[1]), to_dev(b[0]), to_dev(b[1]), packed)
    return d, packed


# ------------------------------------------------------- transposed product

GEMMT = [(1, 1, 128), (2, 7, 128), (5, 63, 256), (16, 64, 384), (32, 65, 512), (33, 130, 640),
         (64, 200, 256), (65, 1000, 128), (128, 129, 1152), (129, 64, 256), (257, 300, 768),
         (300, 128, 384), (40, 4096, 256), (513, 70, 11008), (2049, 520, 7680),
         (1025, 300, 13312)]


@pytest.mark.parametrize("T,m,n", GEMMT)
@pytest.mark.parametrize("ws", [True, None])
def test_gemmt_exact(T, m, n, ws):
    for K, dt in ((1, "f16"), (2, "f32"), (3, "f16"), (4, "f32")):
        say(f"gemmt exact T={T} m={m} n={n} K={K} {dt} workspace={ws}")
        S, A = exact_layer(m, n, K, dt, 7 * m + n + K)
        d, packed = pack_on_gpu(S, A, dt)
        dY = ints(T, m, 3 * T + m)
        # odd strides, NaN around the rows, guarded output rows
        out = torch.full((T, n + 24), -5.0, dtype=BF, device=DEV)
        w = garbage(bw.mbok_gemmt_workspace_bytes(d, T)) if ws else None
        bw.mbok_gemmt(d, packed, wide(dY, m + 5, off=2), out[:, 8:8 + n], workspace=w)
        want = dY.to(F64) @ ref.dense(S, A)
        assert torch.equal(out[:, 8:8 + n].cpu().to(F64), bf16_of(want))
        assert (out[:, :8] == -5).all() and (out[:, 8 + n:] == -5).all()


def test_gemmt_one_hot_rows():
    """Unit rows of dY return rows of W_hat rounded to bf16."""
    say("gemmt one-hot")
    m, n, K = 200, 384, 3
    S, A = gauss_layer(m, n, K, "f16", 4)
    d, packed = pack_on_gpu(S, A, "f16")
    out = torch.empty(m, n, dtype=BF, device=DEV)
    bw.mbok_gemmt(d, packed, wide(torch.eye(m), m), out)
    assert torch.equal(out.cpu().to(F64), ref.dense(S, A).float().to(BF).to(F64))


@pytest.mark.parametrize("T,m,n,K", [(2048, 1000, 640, 3), (17, 5120, 1280, 3), (100, 2050, 512, 4),
                                     (1, 4096, 4096, 2)])
def test_gemmt_gaussian(T, m, n, K):
    say(f"gemmt gaussian T={T} m={m} n={n} K={K}")
    S, A = gauss_layer(m, n, K, "f16", m + n)
    d, packed = pack_on_gpu(S, A, "f16")
    dY = gauss(T, m, T + m, 0.01)
    out = [torch.empty(T, n, dtype=BF, device=DEV) for _ in range(3)]
    bw.mbok_gemmt(d, packed, wide(dY, m), out[0])
    bw.mbok_gemmt(d, packed, wide(dY, m), out[1])
    bw.mbok_gemmt(d, packed, wide(dY, m), out[2], workspace=None)
    assert torch.equal(out[0], out[1])
    W, y = ref.dense(S, A).to(DEV), dY.to(F64).to(DEV)
    want, bound = y @ W, y.abs() @ W.abs()
    for o in (out[0], out[2]):
        assert ((o.to(F64) - want).abs() <= (U + m * 2.0 ** -24) * bound + U * want.abs()).all()


def test_gemmt_matches_one_row_form():
    """T = 1 within the two roundings of mbok_gemvt's fp32 result."""
    say("gemmt against gemvt")
    m, n, K = 777, 512, 2
    S, A = exact_layer(m, n, K, "f16", 6)
    d, packed = pack_on_gpu(S, A, "f16")
    g = wide(ints(1, m, 9), m)
    dx, dX = torch.empty(n, device=DEV), torch.empty(1, n, dtype=BF, device=DEV)
    bw.mbok_gemvt(d, packed, g.view(-1).contiguous(), dx)
    bw.mbok_gemmt(d, packed, g, dX)
    assert torch.equal(dX[0], dx.to(BF))


# ---------------------------------------------------------- scale gradients

GRAD = [(1, 1, 128), (2, 9, 256), (63, 64, 128), (64, 65, 384), (65, 200, 256), (128, 256, 512),
        (300, 130, 640), (1000, 300, 256), (17, 1030, 1152)]


@pytest.mark.parametrize("T,m,n", GRAD)
def test_scale_grad_exact(T, m, n):
    for K, dt in ((1, "f32"), (2, "f16"), (3, "f16"), (4, "f32")):
        say(f"scale_grad exact T={T} m={m} n={n} K={K}")
        S, A = exact_layer(m, n, K, dt, 5 * m + n + K)
        d, packed = pack_on_gpu(S, A, dt)
        dY, X = ints(T, m, T + m), ints(T, n, T + n + 1)
        want = ref.scale_grad(S, dY, X)
        count = want.numel()
        buf = torch.full((count + 8,), -3.0, device=DEV)
        w = garbage(bw.mbok_scale_grad_workspace_bytes(d, T))
        y, x = wide(dY, m + 3, off=1), wide(X, n + 16, off=8)
        bw.mbok_scale_grad(d, packed, y, x, buf[4:4 + count], workspace=w)
        assert torch.equal(buf[4:4 + count].cpu().to(F64).view_as(want), want)
        assert (buf[:4] == -3).all() and (buf[4 + count:] == -3).all()
        # without a workspace, and added to what is there
        bw.mbok_scale_grad(d, packed, y, x, buf[4:4 + count], accumulate=True, workspace=None)
        assert torch.equal(buf[4:4 + count].cpu().to(F64).view_as(want), 2 * want)
        bw.mbok_scale_grad(d, packed, y, x, buf[4:4 + count], accumulate=True, workspace=w)
        assert torch.equal(buf[4:4 + count].cpu().to(F64).view_as(want), 3 * want)


@pytest.mark.parametrize("T,m,n,K", [(2048, 700, 640, 3), (5000, 128, 256, 2)])
def test_scale_grad_gaussian(T, m, n, K):
    """Products of bf16 values are exact in fp32: the sums' rounding alone."""
    say(f"scale_grad gaussian T={T} m={m} n={n} K={K}")
    S, A = gauss_layer(m, n, K, "f16", m + n)
    d, packed = pack_on_gpu(S, A, "f16")
    dY, X = gauss(T, m, T + m, 0.01), gauss(T, n, T + n)
    out = [torch.empty(K, m, n // 128, device=DEV) for _ in range(2)]
    for o in out:
        bw.mbok_scale_grad(d, packed, wide(dY, m), wide(X, n), o)
    assert torch.equal(*out)
    want = ref.scale_grad(S, dY, X)
    bound = (dY.to(F64).abs().t() @ X.to(F64).abs()).view(m, n // 128, 128).sum(-1)
    assert ((out[0].cpu().to(F64) - want).abs() <= (T + 256) * 2.0 ** -24 * bound).all()


def test_scale_grad_nonfinite_stays_in_its_scales():
    say("scale_grad non-finite")
    T, m, n, K = 70, 100, 384, 2
    S, A = exact_layer(m, n, K, "f16", 3)
    d, packed = pack_on_gpu(S, A, "f16")
    dY, X = ints(T, m, 1), ints(T, n, 2)
    dY[69, 40] = float("nan")
    X[3, 200] = float("inf")
    out = torch.empty(K, m, 3, device=DEV)
    bw.mbok_scale_grad(d, packed, wide(dY, m), wide(X, n), out)
    bad = torch.zeros(K, m, 3, dtype=torch.bool)
    bad[:, 40] = True
    nz = dY[3] != 0
    bad[:, nz, 1] = True
    got = out.cpu()
    assert not torch.isfinite(got[:, 40]).any() and not torch.isfinite(got[:, nz, 1]).any()
    keep = ~bad
    keep[:, ~nz, 1] = False  # 0 times infinity
    dY[69, 40], X[3, 200] = 0, 0
    assert torch.equal(got[keep].to(F64), ref.scale_grad(S, dY, X)[keep])


# -------------------------------------------------------- the gated block

# one token, a pair, few tokens (each form), token tiles; row counts around
# the 8-row interleaving, the 64-row blocks and the 128-output tiles
GATED = [(1, 1, 128), (1, 200, 1280), (2, 8, 256), (2, 73, 640), (3, 9, 128), (7, 100, 512),
         (16, 65, 384), (16, 4100, 256), (17, 31, 128), (64, 130, 256), (255, 64, 384),
         (257, 129, 256), (300, 250, 1152), (300, 8500, 128), (257, 5600, 128)]


def gated_want(a, b, X, kind):
    g, u = X.to(F64) @ ref.dense(*a).t(), X.to(F64) @ ref.dense(*b).t()
    return g, u, ref.act(kind, g) * u


def run_gated(d, packed, X, kind, pad=3):
    """H and pre inside guarded buffers."""
    T, m, m2 = X.shape[0], d.m, ref.stacked_rows(d.m)
    H = torch.full((T, m + 2 * pad), -5.0, dtype=BF, device=DEV)
    pre = torch.full((T, m2 + 16), -6.0, dtype=BF, device=DEV)
    x = wide(X, X.shape[1] + 8)
    bw.mbok_gated(d, packed, x, H[:, pad:pad + m], pre=pre[:, 8:8 + m2], act=ACTS[kind])
    only = torch.full((T, m), -5.0, dtype=BF, device=DEV)
    bw.mbok_gated(d, packed, x, only, act=ACTS[kind])
    assert torch.equal(only.view(torch.int16), H[:, pad:pad + m].view(torch.int16))
    assert (H[:, :pad] == -5).all() and (H[:, pad + m:] == -5).all()
    assert (pre[:, :8] == -6).all() and (pre[:, 8 + m2:] == -6).all()
    return only.cpu().to(F64), pre[:, 8:8 + m2].cpu().to(F64)


@pytest.mark.parametrize("T,m,n", GATED)
def test_gated_exact(T, m, n):
    """g and u exact; the activation in fp32: exp's argument is off by
    |g| 2^-24 at most and the base-2 exponential, the reciprocal and the two
    products by 2^-23 each, together below 2^-14 for |g| < 2^9; values below
    2^-100 may be flushed."""
    for K, dt, kind in ((1, "f32", "silu"), (2, "f16", "gelu"), (3, "f16", "silu"),
                        (4, "f32", "gelu")):
        say(f"gated exact T={T} m={m} n={n} K={K} {dt} {kind}")
        a, b = exact_layer(m, n, K, dt, m + n + K), exact_layer(m, n, K, dt, 3 * m + n + K)
        d, packed = gated_layer(a, b, dt)
        X = ints(T, n, T + n)
        X[X.abs() > 2] = 0  # keeps most |g| small enough to matter
        g, u, h = gated_want(a, b, X, kind)
        H, pre = run_gated(d, packed, X, kind)
        assert torch.equal(pre, bf16_of(ref.stack(g, u)))
        assert ((H - h).abs() <= (U + 2.0 ** -14) * h.abs() + 2.0 ** -100).all(), \
            ((H - h).abs() / h.abs()).max()


@pytest.mark.parametrize("variant", ["f4g", "stream", "blocks"])
def test_gated_few_token_forms(variant, monkeypatch):
    """Every few-token kernel, whatever the layer's size would choose."""
    monkeypatch.setenv("MBOK_SKINNY_VARIANT", variant)
    for T, m, n, K in ((2, 70, 384, 3), (5, 1030, 640, 2), (8, 200, 5120, 1), (13, 90, 256, 4),
                       (6, 9000, 256, 3)):
        say(f"gated {variant} T={T} m={m} n={n} K={K}")
        a, b = exact_layer(m, n, K, "f16", m + K), exact_layer(m, n, K, "f16", m + K + 50)
        d, packed = gated_layer(a, b, "f16")
        X = ints(T, n, T)
        X[X.abs() > 2] = 0
        g, u, h = gated_want(a, b, X, "silu")
        H, pre = run_gated(d, packed, X, "silu")
        assert torch.equal(pre, bf16_of(ref.stack(g, u)))
        assert ((H - h).abs() <= (U + 2.0 ** -14) * h.abs() + 2.0 ** -100).all()


def test_gated_octet_rule(monkeypatch):
    """7 and 8 tokens of a large layer take the per-group form: its bits."""
    m, n, K = 6000, 4096, 3
    a, b = gauss_layer(m, n, K, "f16", 3), gauss_layer(m, n, K, "f16", 4)
    d, packed = gated_layer(a, b, "f16")
    for T in (7, 8):
        say(f"gated octet T={T}")
        X = wide(gauss(T, n, T), n)
        H = [torch.empty(T, m, dtype=BF, device=DEV) for _ in range(2)]
        monkeypatch.delenv("MBOK_SKINNY_VARIANT", raising=False)
        bw.mbok_gated(d, packed, X, H[0])
        monkeypatch.setenv("MBOK_SKINNY_VARIANT", "f4g")
        bw.mbok_gated(d, packed, X, H[1])
        assert torch.equal(*H)


@pytest.mark.parametrize("T", [1, 2, 4, 16, 100, 600])
def test_gated_gaussian(T):
    """|H - ref| <= the activation's slope (at most 1.13) times g's error times
    |u|, plus |act(g)| times u's, plus their product, plus the rounding."""
    m, n, K = 1000, 2048, 3
    say(f"gated gaussian T={T}")
    a, b = gauss_layer(m, n, K, "f16", 1), gauss_layer(m, n, K, "f16", 2)
    d, packed = gated_layer(a, b, "f16")
    X = gauss(T, n, T)
    for kind in ACTS:
        g, u, h = gated_want(a, b, X, kind)
        H, pre = run_gated(d, packed, X, kind)
        e = U + n * 2.0 ** -24
        eg = e * (X.to(F64).abs() @ ref.dense(*a).abs().t())
        eu = e * (X.to(F64).abs() @ ref.dense(*b).abs().t())
        want = ref.stack(g, u)
        assert ((pre - want).abs() <= ref.stack(eg, eu) + U * want.abs()).all()
        tol = 1.13 * eg * (u.abs() + eu) + ref.act(kind, g).abs() * eu + 2 * U * h.abs()
        assert ((H - h).abs() <= tol + 2.0 ** -100).all()


def test_gated_large_and_small_gates():
    """The activation's tails: |g| from 2^-20 to 2^12 of both signs, u = 1."""
    say("gated tails")
    n = 128
    S = np.ones((1, 8, n), dtype=np.int8)
    A = np.full((1, 8, 1), 1.0, dtype=np.float32)
    d, packed = gated_layer((S, A), (S, A), "f32")
    vals = [s * 2.0 ** e for e in range(-20, 13) for s in (1, -1)] + [0.0, 88.0, -88.0, -103.0]
    X = torch.zeros(len(vals), n)
    X[:, 5] = torch.tensor(vals)
    for kind in ACTS:
        H, pre = run_gated(d, packed, X, kind)
        g = X[:, 5:6].to(F64).expand(-1, 8)
        h = ref.act(kind, g) * g
        # the argument's rounding: |g| 2^-23 (1 + g^2 for the cubic) relative, while
        # the value is above 2^-100
        rel = U + 2.0 ** -14 + 2.0 ** -22 * g.abs().clamp_max(128.0) * \
            (1 if kind == "silu" else 1 + g.clamp(-8, 8) ** 2)
        assert ((H - h).abs() <= rel * h.abs() + 2.0 ** -100).all()


def test_gated_nonfinite_tokens():
    """A bad activation reaches its own token only (one token: everything)."""
    m, n, K = 100, 256, 2
    a, b = exact_layer(m, n, K, "f16", 1), exact_layer(m, n, K, "f16", 2)
    d, packed = gated_layer(a, b, "f16")
    for T in (1, 2, 9, 40):
        say(f"gated non-finite T={T}")
        X = ints(T, n, T)
        X[X.abs() > 2] = 0
        good = X.clone()
        X[T - 1, 77] = float("nan")
        H, pre = run_gated(d, packed, X, "silu")
        assert torch.isnan(H[T - 1]).all()
        _, _, h = gated_want(a, b, good, "silu")
        assert ((H - h).abs() <= (U + 2.0 ** -14) * h.abs() + 2.0 ** -100)[:T - 1].all()


def test_gated_pack_is_the_interleaved_layer():
    """The stacked buffer equals mbok_pack of the interleaved signs and scales."""
    for m, dt in ((1, "f16"), (9, "f32"), (64, "f16"), (101, "f16")):
        say(f"gated pack m={m}")
        n, K = 256, 3
        a, b = gauss_layer(m, n, K, dt, 1), gauss_layer(m, n, K, dt, 2)
        d, packed = gated_layer(a, b, dt)
        m2 = ref.stacked_rows(m)
        S, A = np.full((K, m2, n), -1, np.int8), np.zeros((K, m2, 2), np_alpha(dt))
        ig, iu = (x.numpy() for x in ref.stack_index(m))
        S[:, ig], S[:, iu], A[:, ig], A[:, iu] = a[0], b[0], a[1], b[1]
        assert torch.equal(packed, pack_on_gpu(S, A, dt)[1])


BACK = [(1, 1, 128), (3, 9, 256), (40, 130, 384), (100, 64, 256), (300, 200, 512)]


@pytest.mark.parametrize("T,m,n", BACK)
def test_gated_backward(T, m, n):
    """dpre: slope and activation in fp32 are off by 2^-14 of s u (1 + |g|) at
    most (the sum 1 + g (1 - s) cancels near the slope's zero), then one
    rounding.  dX: the transposed product of the dpre that was written."""
    for K, dt, kind in ((2, "f16", "silu"), (3, "f32", "gelu")):
        say(f"gated_backward T={T} m={m} n={n} K={K} {kind}")
        a, b = exact_layer(m, n, K, dt, m + K), exact_layer(m, n, K, dt, m + K + 9)
        d, packed = gated_layer(a, b, dt)
        m2 = ref.stacked_rows(m)
        g, u, s = gauss(T, m, 1, 2.0), gauss(T, m, 2, 2.0), gauss(T, m, 3, 0.1)
        pre = ref.stack(g, u)
        if m % 8:  # the padding columns are not read
            pad = torch.ones(m2, dtype=torch.bool)
            pad[torch.cat(ref.stack_index(m))] = False
            pre[:, pad] = float("nan")
        pre, dH = wide(pre, m2 + 8), wide(s, m + 1, off=1)
        dpre = torch.full((T, m2 + 8), -4.0, dtype=BF, device=DEV)
        dX = torch.full((T, n + 8), -4.0, dtype=BF, device=DEV)
        w = garbage(bw.mbok_gemmt_workspace_bytes(bw.mbok_gated_stack(d), T))
        bw.mbok_gated_backward(d, packed, pre, dH, dpre[:, :m2], dX[:, :n], act=ACTS[kind],
                               workspace=w)
        G, Uu, s = g.to(F64), u.to(F64), s.to(F64)
        want = ref.stack(s * Uu * ref.act_slope(kind, G), s * ref.act(kind, G))
        scale = ref.stack((s * Uu).abs() * (1 + G.abs()), (s * G).abs())
        got = dpre[:, :m2].cpu().to(F64)
        assert ((got - want).abs() <= U * want.abs() + 2.0 ** -14 * scale).all()
        W = torch.zeros(m2, n, dtype=F64)
        ig, iu = ref.stack_index(m)
        W[ig], W[iu] = ref.dense(*a), ref.dense(*b)
        x, bound = got @ W, got.abs() @ W.abs()
        assert ((dX[:, :n].cpu().to(F64) - x).abs() <=
                m2 * 2.0 ** -24 * bound + U * x.abs()).all()
        assert (dpre[:, m2:] == -4).all() and (dX[:, n:] == -4).all()
        # dpre alone, in place of pre: the same bits
        again = pre.clone() if pre.is_contiguous() else pre
        bw.mbok_gated_backward(d, packed, again, dH, again, act=ACTS[kind])
        assert torch.equal(again, dpre[:, :m2])


# ------------------------------------------------------------- together

def test_finetuning_step_of_a_block():
    """One step as a program runs it: gated block, down projection, head, loss
    from the teacher's top logits, and back to the block's input and scales.
    Every call's output is checked against float64 of its own inputs; the
    whole chain's gradient direction against the float64 chain: each of its
    five roundings to bf16 and three products with bf16 levels is at most
    2^-8 relative per element and independent, so the relative distance stays
    below 8 2^-8, far from what a wrong operand would give (about 1)."""
    say("fine-tuning step")
    T, n, m, V, top, K, tau = 96, 256, 520, 640, 12, 2, 2.0
    a, b = gauss_layer(m, n, K, "f16", 1), gauss_layer(m, n, K, "f16", 2)
    D, Hd = gauss_layer(n, m // 128 * 128 + 128, K, "f16", 3), gauss_layer(V, n, K, "f16", 4)
    mp = D[0].shape[2]  # the down projection's columns, H zero-padded to them
    d, packed = gated_layer(a, b, "f16")
    dd, dpacked = pack_on_gpu(D[0], D[1], "f16")
    dh, hpacked = pack_on_gpu(Hd[0], Hd[1], "f16")
    X = gauss(T, n, 5)
    teacher = torch.randn(T, V, generator=torch.Generator().manual_seed(6)) * 2
    l, idx = teacher.topk(top, -1)
    x = wide(X, n)
    m2 = ref.stacked_rows(m)
    H = torch.zeros(T, mp, dtype=BF, device=DEV)
    pre = torch.empty(T, m2, dtype=BF, device=DEV)
    y, z = torch.empty(T, n, device=DEV), torch.empty(T, V, device=DEV)
    bw.mbok_gated(d, packed, x, H[:, :m], pre=pre)
    bw.mbok_gemm(dd, dpacked, H, y)
    bw.mbok_gemm(dh, hpacked, y.to(BF), z)
    loss = torch.empty(T, device=DEV)
    dz = torch.empty(T, V, dtype=BF, device=DEV)
    ds = bw.mbok_distill_desc_init(V, top, tau)
    bw.mbok_distill(ds, z, l.to(DEV), idx.to(torch.int32).to(DEV), loss, dZ=dz)
    dy = torch.empty(T, n, dtype=BF, device=DEV)
    bw.mbok_gemmt(dh, hpacked, dz, dy)
    dHg = torch.empty(T, mp, dtype=BF, device=DEV)
    bw.mbok_gemmt(dd, dpacked, dy, dHg)
    dpre, dX = torch.empty_like(pre), torch.empty(T, n, dtype=BF, device=DEV)
    bw.mbok_gated_backward(d, packed, pre, dHg[:, :m], dpre, dX)
    d2 = bw.mbok_gated_stack(d)
    da = torch.empty(K, m2, n // 128, device=DEV)
    bw.mbok_scale_grad(d2, packed, dpre, x, da)

    # the float64 chain by autograd
    leaves = [torch.as_tensor(v[1]).to(F64).requires_grad_() for v in (a, b)]
    Xr = X.to(F64).requires_grad_()
    Wg, Wu = ref.dense(a[0], leaves[0]), ref.dense(b[0], leaves[1])
    g, u = Xr @ Wg.t(), Xr @ Wu.t()
    h = ref.act("silu", g) * u
    zr = (h @ ref.dense(*D)[:, :m].t()) @ ref.dense(*Hd).t()
    logq, logp = torch.log_softmax(zr / tau, -1), torch.log_softmax(l.to(F64) / tau, -1)
    want = tau * tau * (logp.exp() * (logp - logq.gather(1, idx))).sum(-1)
    want.sum().backward()

    def near(got, ref_value, most=8 * U):
        got = got.cpu().to(F64)
        assert float((got - ref_value).norm() / ref_value.norm()) < most

    near(z, zr.detach())
    near(loss, want.detach())
    near(dX, Xr.grad)
    ig, iu = ref.stack_index(m)
    near(da[:, ig.to(DEV)], leaves[0].grad)
    near(da[:, iu.to(DEV)], leaves[1].grad)


def test_graphs_and_streams():
    """Each call captured and replayed with eager work of other sizes between
    (which grows the kept workspace), and on two streams at once: the eager
    bits every time."""
    say("graphs and streams")
    T, m, n, K = 40, 300, 512, 3
    a, b = gauss_layer(m, n, K, "f16", 1), gauss_layer(m, n, K, "f16", 2)
    d, packed = gated_layer(a, b, "f16")
    d2 = bw.mbok_gated_stack(d)
    x, dH = wide(gauss(T, n, 1), n), wide(gauss(T, m, 2), m)
    big, bpacked = pack_on_gpu(*gauss_layer(3000, 512, 3, "f16", 9), "f16")
    bigY = wide(gauss(128, 3000, 3), 3000)
    bigX = wide(gauss(128, 512, 3), 512)

    def outputs():
        return [torch.empty(T, m, dtype=BF, device=DEV), torch.empty(T, d2.m, dtype=BF, device=DEV),
                torch.empty(T, d2.m, dtype=BF, device=DEV), torch.empty(T, n, dtype=BF, device=DEV),
                torch.empty(K, d2.m, n // 128, device=DEV)]

    def step(o, stream=None):
        bw.mbok_gated(d, packed, x, o[0], pre=o[1], stream=stream)
        bw.mbok_gated_backward(d, packed, o[1], dH, o[2], o[3], stream=stream)
        bw.mbok_scale_grad(d2, packed, o[2], x, o[4], stream=stream)

    def other():
        bw.mbok_gemmt(big, bpacked, bigY, torch.empty(128, 512, dtype=BF, device=DEV))
        bw.mbok_scale_grad(big, bpacked, bigY, bigX, torch.empty(3, 3000, 4, device=DEV))

    out = outputs()
    step(out)
    want = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g, o = torch.cuda.CUDAGraph(), outputs()
        with torch.cuda.graph(g):
            step(o)
        graphs.append((g, o))
    for _ in range(3):
        for g, o in graphs:
            for v in o:
                v.fill_(-1)
            g.replay()
        other()
        torch.cuda.synchronize()
        for _, o in graphs:
            assert all(torch.equal(v, w) for v, w in zip(o, want))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [outputs(), outputs()]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        step(o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(v, w) for v, w in zip(o, want))
