"""GPU parity of the layer with bias, activation and residual (mbok_linear) and
of its backward, through the C ABI, against float64.

Exact regime, roundings and the bound of a product: see test_gpu_finetune.py.
With z off by D (the product's bound, and 2^-24 (|W x| + |z|) for the sums and
the bias), an activation of slope at most 1.13 and two more fp32 operations, y =
R + act(z) is off by 1.13 D + 2^-22 (|z| + |R| + |y|) (the activation's
exponential and reciprocal carry a few 2^-24 relative) before its rounding to
Y's type, half a step of the value.
"""
import pytest
import torch

import boolean_weight_amd as bw
import finetune_ref
import step_ref as ref
from gpu_util import DEV, pack_on_gpu, say
from test_gpu_finetune import bf16_of, exact_layer, garbage, gauss, gauss_layer, ints, wide

pytestmark = pytest.mark.gpu

F64, BF = torch.float64, torch.bfloat16
U, EPS = 2.0 ** -8, 2.0 ** -24
ACTS = {"none": bw.MBOK_ACT_NONE, "silu": bw.MBOK_ACT_SILU, "gelu": bw.MBOK_ACT_GELU}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def rows(x, ld, off, dtype=BF, fill=float("nan")):
    """x as rows of a [T, ld] device buffer full of `fill`."""
    buf = torch.full((x.shape[0], ld), fill, dtype=dtype, device=DEV)
    buf[:, off:off + x.shape[1]] = x.to(dtype).to(DEV)
    return buf, buf[:, off:off + x.shape[1]]


def guards_hold(buf, off, n, fill=-5.0):
    return bool((buf[:, :off] == fill).all() and (buf[:, off + n:] == fill).all())


# every form: one token, two, the octet and the few-token kernels (some streaming),
# and each tile of the many-token kernel, whole rounds with halves of the rest among
# them; widths of one row up, no multiples of a tile
SHAPES = [(1, 1, 128), (1, 4096, 640), (2, 130, 384), (3, 65, 256), (5, 1000, 512), (9, 15, 128),
          (12, 8200, 256), (16, 77, 1152), (16, 4096, 256), (17, 1, 128), (17, 300, 256),
          (64, 129, 384), (65, 1000, 128), (129, 513, 256), (200, 4100, 256), (1300, 4099, 128),
          (4000, 4400, 128), (1000, 5000, 256)]


@pytest.mark.parametrize("T,m,n", SHAPES)
def test_linear_exact(T, m, n):
    """Integers plus a bias and a residual that keep every sum a multiple of 2^-8
    below 2^16: Y without an activation differs by its one rounding, none in fp32."""
    for K, dt, yt in ((1, "f16", BF), (2, "f32", torch.float32), (3, "f16", BF), (4, "f32", BF)):
        say(f"linear exact T={T} m={m} n={n} K={K} {dt} {yt}")
        S, A = exact_layer(m, n, K, dt, 7 * m + n + K)
        d, packed = pack_on_gpu(S, A, dt)
        X, R = ints(T, n, 3 * T + n), ints(T, m, T + m + 1)
        bias = ints(1, m, 5)[0] / 4
        x = wide(X, n + 16, off=8)
        _, r = rows(R, m + 3, 2, yt)
        buf = torch.full((T, m + 9), -5.0, dtype=yt, device=DEV)
        pbuf = torch.full((T, m + 7), -5.0, dtype=BF, device=DEV)
        y, pre = buf[:, 4:4 + m], pbuf[:, 3:3 + m]
        bw.mbok_linear(d, packed, x, y, bias=bias.to(DEV), residual=r, pre=pre)
        want, z = ref.linear(finetune_ref.dense(S, A), X, bias, "none", R)
        assert torch.equal(y.cpu().to(F64), want if yt == torch.float32 else bf16_of(want))
        assert torch.equal(pre.cpu().to(F64), bf16_of(z))
        assert guards_hold(buf, 4, m) and guards_hold(pbuf, 3, m)
        # nothing but the product; the residual updated in place
        bw.mbok_linear(d, packed, x, y)
        want0 = ref.linear(finetune_ref.dense(S, A), X)[0]
        assert torch.equal(y.cpu().to(F64), want0 if yt == torch.float32 else bf16_of(want0))
        bw.mbok_linear(d, packed, x, r, residual=r, bias=bias.to(torch.float16).to(DEV))
        assert torch.equal(r.cpu().to(F64), want if yt == torch.float32 else bf16_of(want))


# each shape of the few-token products for more than 16 tokens (tiles and chunks of a
# workgroup: 1 x 1, 2 x 1, 2 x 2, 4 x 2), ragged tokens and rows, tall contractions
@pytest.mark.parametrize("T,m,n", [(17, 30, 2048), (100, 9, 5120), (33, 2500, 2048),
                                   (64, 2490, 2048), (100, 2497, 2048), (33, 4096, 2176),
                                   (250, 1000, 2048)])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
def test_linear_small_layers_exact(T, m, n, K):
    say(f"linear small layer T={T} m={m} n={n} K={K}")
    dt = "f16" if K % 2 else "f32"
    S, A = exact_layer(m, n, K, dt, m + n + K)
    d, packed = pack_on_gpu(S, A, dt)
    X, R = ints(T, n, T + n), ints(T, m, T + m)
    buf = torch.full((T, m + 9), -5.0, device=DEV)
    pbuf = torch.full((T, m + 7), -5.0, dtype=BF, device=DEV)
    y, pre = buf[:, 4:4 + m], pbuf[:, 3:3 + m]
    x = wide(X, n + 8, off=0)
    bw.mbok_linear(d, packed, x, y, residual=R.to(DEV), pre=pre)
    want, z = ref.linear(finetune_ref.dense(S, A), X, None, "none", R)
    assert torch.equal(y.cpu().to(F64), want)
    assert torch.equal(pre.cpu().to(F64), bf16_of(z))
    assert guards_hold(buf, 4, m) and guards_hold(pbuf, 3, m)
    again = torch.empty(T, m, device=DEV)
    bw.mbok_linear_precise(d, packed, x, again, residual=R.to(DEV))
    assert torch.equal(again, y)


# the many-token forms: 64 x 64 tiles in 4 and in 2 shares of the contraction (groups
# that do not divide by them, fewer groups than shares), 128 x 128 in 2, and tiles of 64
# and 128 whole
@pytest.mark.parametrize("T,m,n", [(100, 300, 640), (65, 9, 896), (250, 1030, 1408), (40, 70, 384),
                                   (260, 4100, 512), (1000, 2300, 384), (129, 9000, 256),
                                   (300, 300, 128), (50, 33000, 128), (2048, 2300, 128)])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
def test_linear_few_tiles_exact(T, m, n, K):
    say(f"linear few tiles T={T} m={m} n={n} K={K}")
    dt = "f32" if K % 2 else "f16"
    S, A = exact_layer(m, n, K, dt, m + n + K)
    d, packed = pack_on_gpu(S, A, dt)
    X, R = ints(T, n, T + n), ints(T, m, T + m)
    buf = torch.full((T, m + 9), -5.0, device=DEV)
    pbuf = torch.full((T, m + 7), -5.0, dtype=BF, device=DEV)
    y, pre = buf[:, 4:4 + m], pbuf[:, 3:3 + m]
    x = wide(X, n + 8, off=0)
    bw.mbok_linear(d, packed, x, y, residual=R.to(DEV), pre=pre)
    want, z = ref.linear(finetune_ref.dense(S, A), X, None, "none", R)
    assert torch.equal(y.cpu().to(F64), want)
    assert torch.equal(pre.cpu().to(F64), bf16_of(z))
    assert guards_hold(buf, 4, m) and guards_hold(pbuf, 3, m)
    again = torch.empty(T, m, dtype=BF, device=DEV)
    bw.mbok_linear_precise(d, packed, x, again, residual=R.to(DEV, BF))
    assert torch.equal(again.cpu().to(F64), bf16_of(want))


def bound_of(T, W, X, z):
    few = T <= 16
    # T <= 16: every scale exact in fp32, activations to 2^-16 at worst (f4 forms)
    per_weight = 2.0 ** -16 if few else U
    return (per_weight + W.shape[1] * EPS) * (X.abs() @ W.abs().t()) + 2 * EPS * z.abs()


@pytest.mark.parametrize("T,m,n,K", [(1, 4096, 1024, 3), (2, 513, 640, 2), (6, 8192, 4096, 2),
                                     (8, 11008, 4096, 3), (16, 700, 1280, 3), (33, 300, 640, 4),
                                     (300, 1030, 512, 3), (2048, 520, 384, 3),
                                     (1024, 5120, 256, 1)])
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_linear_gaussian(T, m, n, K, kind):
    say(f"linear gaussian T={T} m={m} n={n} K={K} {kind}")
    S, A = gauss_layer(m, n, K, "f16", m + n)
    d, packed = pack_on_gpu(S, A, "f16")
    X, R = gauss(T, n, T + n), gauss(T, m, T + m + 9)
    bias = gauss(1, m, 4, 0.3)[0]
    W, Xd, Rd = finetune_ref.dense(S, A).to(DEV), X.to(F64).to(DEV), R.to(F64).to(DEV)
    want, z = ref.linear(W, Xd, bias.to(DEV), kind, Rd)
    for yt, name in ((BF, "mbok_linear"), (torch.float32, "mbok_linear"),
                     (torch.float32, "mbok_linear_precise")):
        out = [torch.empty(T, m, dtype=yt, device=DEV) for _ in range(2)]
        pre = torch.empty(T, m, dtype=BF, device=DEV)
        for o in out:
            getattr(bw, name)(d, packed, wide(X, n), o, bias=bias.to(BF).to(DEV), act=ACTS[kind],
                              residual=R.to(yt).to(DEV), pre=pre)
        assert torch.equal(*out)
        D = bound_of(16 if name.endswith("precise") else T, W, Xd, z)
        half = U if yt == BF else EPS
        tol = 1.13 * D + 4 * EPS * (z.abs() + Rd.abs() + want.abs()) + half * want.abs()
        assert ((out[0].to(F64) - want).abs() <= tol).all()
        assert ((pre.to(F64) - z).abs() <= D + U * z.abs()).all()


@pytest.mark.parametrize("T", [1, 2, 7, 16, 40, 300])
def test_linear_is_the_product_with_its_epilogue(T):
    """A long activation range through silu and gelu: no overflow, limits exact."""
    say(f"linear limits T={T}")
    m, n, K = 70, 128, 1
    S, A = exact_layer(m, n, K, "f32", 3)
    d, packed = pack_on_gpu(S, A, "f32")
    X = torch.zeros(T, n)
    bias = torch.tensor([0.0, -0.0, 3e38, -3e38, 100.0, -100.0, 1e-30, -1e4] * 9)[:m]
    for kind in ("silu", "gelu"):
        y = torch.empty(T, m, device=DEV)
        bw.mbok_linear(d, packed, wide(X, n), y, bias=bias.to(DEV), act=ACTS[kind])
        want = ref.act(kind, bias.to(F64)).expand(T, m)
        got = y.cpu().to(F64)
        assert torch.isfinite(got).all()
        assert ((got - want).abs() <= 8 * EPS * want.abs() + 1e-37).all()


@pytest.mark.parametrize("T", [1, 2, 6, 16, 40, 400])
def test_linear_nonfinite_rows_stay_alone(T):
    say(f"linear non-finite T={T}")
    m, n, K = 300, 384, 2
    S, A = exact_layer(m, n, K, "f16", 8)
    d, packed = pack_on_gpu(S, A, "f16")
    X, R = ints(T, n, 1), ints(T, m, 2)
    X[T - 1, 5] = float("nan")
    R[0, 3] = float("inf")
    y = torch.empty(T, m, dtype=BF, device=DEV)
    bw.mbok_linear(d, packed, wide(X, n), y, residual=wide(R, m))
    got = y.cpu()
    assert torch.isnan(got[T - 1]).all()
    if T > 1:
        assert got[0, 3] == float("inf")
        keep = torch.ones(T, m, dtype=torch.bool)
        keep[T - 1], keep[0, 3] = False, False
        assert torch.isfinite(got[keep]).all()


BACKWARD = [(1, 1, 128), (7, 9, 256), (16, 1001, 128), (63, 256, 384), (128, 257, 128),
            (300, 130, 640), (1000, 2050, 128), (2049, 520, 256)]


@pytest.mark.parametrize("T,m,n", BACKWARD)
@pytest.mark.parametrize("ws", [True, None])
def test_backward_without_activation_exact(T, m, n, ws):
    for K, dt in ((1, "f16"), (3, "f32")):
        say(f"linear backward exact T={T} m={m} n={n} K={K} workspace={ws}")
        S, A = exact_layer(m, n, K, dt, 5 * m + n + K)
        d, packed = pack_on_gpu(S, A, dt)
        dY = ints(T, m, 2 * T + m)
        y = wide(dY, m + 5, off=3)
        w = garbage(bw.mbok_linear_backward_workspace_bytes(d, T)) if ws else None
        buf = torch.full((m + 8,), -3.0, device=DEV)
        db = buf[4:4 + m]
        out = torch.full((T, n + 16), -5.0, dtype=BF, device=DEV)
        bw.mbok_linear_backward(d, packed, y, dbias=db, dX=out[:, 8:8 + n], workspace=w)
        want = dY.to(F64) @ finetune_ref.dense(S, A)
        assert torch.equal(out[:, 8:8 + n].cpu().to(F64), bf16_of(want))
        assert guards_hold(out, 8, n)
        sums = dY.to(F64).sum(0)  # integers below 2^24: exact
        assert torch.equal(db.cpu().to(F64), sums)
        bw.mbok_linear_backward(d, packed, y, dbias=db, accumulate=True, workspace=w)
        assert torch.equal(db.cpu().to(F64), 2 * sums)
        assert (buf[:4] == -3).all() and (buf[4 + m:] == -3).all()
        only = torch.empty(T, n, dtype=BF, device=DEV)
        bw.mbok_linear_backward(d, packed, y, dX=only, workspace=w)
        assert torch.equal(only, out[:, 8:8 + n])


def test_backward_bias_of_more_columns_than_a_grid_has_rows():
    """One token, 2.2 million outputs: the bias sums do not fit beside the product's
    joining kernel."""
    say("linear backward, many columns")
    m, n = 2200000, 128
    S, A = exact_layer(m, n, 1, "f16", 3)
    d, packed = pack_on_gpu(S, A, "f16")
    dY = ints(1, m, 4)
    db, dX = torch.empty(m, device=DEV), torch.empty(1, n, dtype=BF, device=DEV)
    bw.mbok_linear_backward(d, packed, wide(dY, m), dbias=db, dX=dX)
    assert torch.equal(db.cpu().to(F64), dY[0].to(F64))
    want = torch.empty(1, n, dtype=BF, device=DEV)
    bw.mbok_gemmt(d, packed, wide(dY, m), want)
    assert torch.equal(dX, want)


@pytest.mark.parametrize("T,m,n,K", [(1, 300, 128, 2), (5, 9, 128, 1), (37, 1001, 640, 2),
                                     (200, 4096, 256, 3), (2048, 1000, 384, 3), (129, 7, 256, 4)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_gaussian(T, m, n, K, kind):
    """dpre: the slope to a few 2^-24 of its terms (at most 1.13 (1 + |z|)), one
    rounding; dbias: T fp32 sums of those; dX: of the rounded dpre."""
    say(f"linear backward T={T} m={m} n={n} K={K} {kind}")
    S, A = gauss_layer(m, n, K, "f16", m + n)
    d, packed = pack_on_gpu(S, A, "f16")
    dY, z = gauss(T, m, T + m, 0.02), gauss(T, m, T + m + 1, 2.0)
    y, p = wide(dY, m + 2, off=1), wide(z, m + 3, off=2)
    db, dX = torch.empty(m, device=DEV), torch.empty(T, n, dtype=BF, device=DEV)
    dbuf = torch.full((T, m + 6), -5.0, dtype=BF, device=DEV)
    dpre = dbuf[:, 5:5 + m]
    bw.mbok_linear_backward(d, packed, y, pre=p, dpre=dpre, dbias=db, dX=dX, act=ACTS[kind])
    dYd, zd = dY.to(F64), z.to(F64)
    slope = ref.act_slope(kind, zd)
    want = dYd * slope
    # near 0 a slope is the difference of terms of up to 1.13 (1 + |z|)
    off = 16 * EPS * dYd.abs() * (1 + zd.abs())
    got = dpre.cpu().to(F64)
    assert ((got - want).abs() <= off + U * want.abs()).all()
    assert guards_hold(dbuf, 5, m)
    assert ((db.cpu().to(F64) - want.sum(0)).abs() <=
            (off + (T + 8) * EPS * want.abs()).sum(0)).all()
    W = finetune_ref.dense(S, A)
    dx = got @ W
    tol = (U + m * EPS) * (got.abs() @ W.abs()) + U * dx.abs()
    assert ((dX.cpu().to(F64) - dx).abs() <= tol).all()
    precise = torch.empty_like(dX)
    # in place of dY and of pre, the two-term form, no workspace
    bw.mbok_linear_backward_precise(d, packed, y, pre=p, dpre=y, dX=precise, act=ACTS[kind],
                                    workspace=None)
    assert torch.equal(y, dpre)
    tol = (2.0 ** -16 + m * EPS) * (got.abs() @ W.abs()) + U * dx.abs()
    assert ((precise.cpu().to(F64) - dx).abs() <= tol).all()
    again = wide(dY, m)
    db2 = torch.empty_like(db)
    bw.mbok_linear_backward(d, packed, again, pre=p, dpre=p, dbias=db2, act=ACTS[kind])
    assert torch.equal(p, dpre) and torch.equal(db2, db)


def test_backward_gradient_by_differences():
    """dX and dbias against differences of the kernel's own forward (fp32 Y, T <= 16:
    exact per scale).  h = 0.125 on unit activations: the difference's own error is
    h^2 / 6 times the third derivative (below 1.3 |w|^3 sums), the fp32 outputs' 2^-21 /
    h; dX itself rounds twice to bf16."""
    say("linear backward by differences")
    T, m, n, K = 4, 24, 128, 2
    S, A = gauss_layer(m, n, K, "f16", 2)
    d, packed = pack_on_gpu(S, A, "f16")
    X, up = gauss(T, n, 3), gauss(T, m, 4)
    W = finetune_ref.dense(S, A)
    act = dict(act=bw.MBOK_ACT_GELU)

    def loss(x):
        y = torch.empty(T, m, device=DEV)
        bw.mbok_linear(d, packed, wide(x, n), y, **act)
        return float((y.cpu().to(F64) * up.to(F64)).sum())

    pre, y = torch.empty(T, m, dtype=BF, device=DEV), torch.empty(T, m, device=DEV)
    bw.mbok_linear(d, packed, wide(X, n), y, pre=pre, **act)
    dX, dpre = torch.empty(T, n, dtype=BF, device=DEV), torch.empty_like(pre)
    bw.mbok_linear_backward(d, packed, wide(up, m), pre=pre, dpre=dpre, dX=dX, **act)
    for t, j in ((0, 0), (1, 17), (2, 64), (3, 127)):
        hi, lo = X.clone(), X.clone()
        hi[t, j] += 0.125
        lo[t, j] -= 0.125
        hi, lo = hi.to(BF).float(), lo.to(BF).float()
        h = float(hi[t, j] - lo[t, j])
        slope = (loss(hi) - loss(lo)) / h
        terms = float((up[t].to(F64).abs() * W[:, j].abs()).sum())
        third = float((up[t].to(F64).abs() * W[:, j].abs() ** 3).sum()) * 1.3 * 0.14 ** 2 / 6
        # pre is rounded to bf16 (slope changes by at most 1.2 2^-8 |z|), dpre and the
        # levels round once each, dX once
        z = pre[t].cpu().to(F64).abs()
        rounding = float((up[t].to(F64).abs() * W[:, j].abs() * (1.2 * U * z + 2.3 * U)).sum())
        tol = rounding + third + U * abs(slope) + 2.0 ** -19 * terms / 0.125 + 2.0 ** -14
        assert abs(float(dX[t, j]) - slope) <= tol
