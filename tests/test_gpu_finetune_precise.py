"""The two-term forms (mbok_gemmt_precise, mbok_gated_precise,
mbok_gated_backward_precise) against float64.

Exact regime: power-of-two scales spread over 2^-2 .. 2^-14, so that a level
has up to 14 significant bits, more than one bf16 term and fewer than two;
integer activations in [-2, 2], every partial sum a multiple of 2^-14 below
2^10: products and sums are exact, a result is the float64 one after its single
rounding, and the one-term form differs.

Otherwise a weight is off by at most 2^-16 of itself and fp32 sums of 2 c terms
by 2 c 2^-24 of the absolute sum: |y - ref| <= (2^-16 + 2 c 2^-24) sum |W| |x| +
2^-8 |y|.
"""
import numpy as np
import pytest
import torch

import boolean_weight_amd as bw
import finetune_ref as ref
import mbok_synth as syn
from gpu_util import DEV, np_alpha, pack_on_gpu, say
from test_gpu_finetune import (ACTS, BF, F64, U, bf16_of, garbage, gated_layer, gauss,
                               gauss_layer, wide)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def spread_layer(m, n, K, dt, seed):
    rng = np.random.default_rng(seed)
    A = 2.0 ** -rng.integers(2, 15, size=(K, m, n // 128)).astype(np.float64)
    return syn.random_signs(K, m, n, seed=seed), A.astype(np_alpha(dt))


def small_ints(T, n, seed, most):
    """Integers in [-2, 2], at most `most` of a row not 0 (its sums stay exact)."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randint(-2, 3, (T, n), generator=gen).float()
    keep = torch.rand(T, n, generator=gen) < min(1.0, most / n)
    return x * keep


# token tiles of 32, 64, 128 and 256, rows that fill the last block and rows
# that do not, whole tiles beside sliced ones
GEMMT = [(1, 7, 128), (16, 64, 384), (20, 2048, 4096), (33, 130, 640), (64, 1928, 4096),
         (100, 2050, 2048), (129, 64, 256), (300, 1024, 4096), (513, 70, 11008), (1025, 300, 13312),
         (4096, 192, 4096)]


@pytest.mark.parametrize("T,m,n", GEMMT)
@pytest.mark.parametrize("aligned", [True, False])
def test_gemmt_precise_exact(T, m, n, aligned):
    differs = False
    for K, dt in ((1, "f16"), (2, "f32"), (3, "f16"), (4, "f32")):
        say(f"gemmt precise T={T} m={m} n={n} K={K} {dt} aligned={aligned}")
        S, A = spread_layer(m, n, K, dt, 7 * m + n + K)
        d, packed = pack_on_gpu(S, A, dt)
        dY = small_ints(T, m, T + m, 400)
        y = wide(dY, (m + 15) // 8 * 8, off=8 if m % 8 == 0 else 0) if aligned else \
            wide(dY, m + 5, off=3)
        exact = (dY.to(F64).to(DEV) @ ref.dense(S, A).to(DEV)).cpu()
        assert float(exact.abs().max()) < 2.0 ** 10
        want = bf16_of(exact)
        for ws in (garbage(bw.mbok_gemmt_workspace_bytes(d, T)), None):
            out = torch.full((T, n + 24), -5.0, dtype=BF, device=DEV)
            bw.mbok_gemmt_precise(d, packed, y, out[:, 8:8 + n], workspace=ws)
            assert torch.equal(out[:, 8:8 + n].cpu().to(F64), want)
            assert (out[:, :8] == -5).all() and (out[:, 8 + n:] == -5).all()
        bw.mbok_gemmt(d, packed, y, out[:, 8:8 + n])
        differs |= not torch.equal(out[:, 8:8 + n].cpu().to(F64), want)
    assert differs  # the input needs the second term


@pytest.mark.parametrize("T,m,n,K", [(2048, 1000, 640, 3), (17, 5120, 1280, 3), (100, 2050, 512, 4),
                                     (1, 4096, 4096, 2)])
def test_gemmt_precise_gaussian(T, m, n, K):
    say(f"gemmt precise gaussian T={T} m={m} n={n} K={K}")
    S, A = gauss_layer(m, n, K, "f16", m + n)
    d, packed = pack_on_gpu(S, A, "f16")
    dY = gauss(T, m, T + m, 0.01)
    out = [torch.empty(T, n, dtype=BF, device=DEV) for _ in range(3)]
    for o, ws in zip(out, (True, True, None)):
        bw.mbok_gemmt_precise(d, packed, wide(dY, m), o, workspace=ws)
    assert torch.equal(out[0], out[1])
    W, y = ref.dense(S, A).to(DEV), dY.to(F64).to(DEV)
    want, bound = y @ W, y.abs() @ W.abs()
    for o in (out[0], out[2]):
        tol = (2.0 ** -16 + 2 * m * 2.0 ** -24) * bound + U * want.abs()
        assert ((o.to(F64) - want).abs() <= tol).all()


def run_gated(fn, d, packed, X, kind):
    T, m, m2 = X.shape[0], d.m, ref.stacked_rows(d.m)
    H = torch.full((T, m + 6), -5.0, dtype=BF, device=DEV)
    pre = torch.full((T, m2 + 16), -6.0, dtype=BF, device=DEV)
    fn(d, packed, wide(X, X.shape[1] + 8), H[:, 3:3 + m], pre=pre[:, 8:8 + m2], act=ACTS[kind])
    assert (H[:, :3] == -5).all() and (H[:, 3 + m:] == -5).all()
    assert (pre[:, :8] == -6).all() and (pre[:, 8 + m2:] == -6).all()
    return H[:, 3:3 + m].cpu().to(F64), pre[:, 8:8 + m2].cpu().to(F64)


# 64 x 64, 128 x 128 and 256 x 256 tiles
@pytest.mark.parametrize("T,m,n", [(17, 31, 128), (64, 130, 256), (255, 64, 384), (257, 129, 1152),
                                   (300, 8500, 128), (257, 5600, 256)])
def test_gated_precise_exact(T, m, n):
    differs = False
    for K, dt, kind in ((1, "f32", "silu"), (2, "f16", "gelu"), (3, "f16", "silu"),
                        (4, "f32", "gelu")):
        say(f"gated precise T={T} m={m} n={n} K={K} {dt} {kind}")
        a, b = spread_layer(m, n, K, dt, m + n + K), spread_layer(m, n, K, dt, 3 * m + n + K)
        d, packed = gated_layer(a, b, dt)
        X = small_ints(T, n, T + n, 100)
        g, u = X.to(F64) @ ref.dense(*a).t(), X.to(F64) @ ref.dense(*b).t()
        h = ref.act(kind, g) * u
        H, pre = run_gated(bw.mbok_gated_precise, d, packed, X, kind)
        assert torch.equal(pre, bf16_of(ref.stack(g, u)))
        assert ((H - h).abs() <= (U + 2.0 ** -14) * h.abs() + 2.0 ** -100).all()
        differs |= not torch.equal(run_gated(bw.mbok_gated, d, packed, X, kind)[1], pre)
    assert differs


@pytest.mark.parametrize("T", [17, 100, 600])
def test_gated_precise_gaussian(T):
    m, n, K = 1000, 2048, 3
    say(f"gated precise gaussian T={T}")
    a, b = gauss_layer(m, n, K, "f16", 1), gauss_layer(m, n, K, "f16", 2)
    d, packed = gated_layer(a, b, "f16")
    X = gauss(T, n, T)
    g, u = X.to(F64) @ ref.dense(*a).t(), X.to(F64) @ ref.dense(*b).t()
    e = 2.0 ** -16 + 2 * n * 2.0 ** -24
    eg = e * (X.to(F64).abs() @ ref.dense(*a).abs().t())
    eu = e * (X.to(F64).abs() @ ref.dense(*b).abs().t())
    for kind in ACTS:
        h = ref.act(kind, g) * u
        H, pre = run_gated(bw.mbok_gated_precise, d, packed, X, kind)
        want = ref.stack(g, u)
        assert ((pre - want).abs() <= ref.stack(eg, eu) + U * want.abs()).all()
        tol = 1.13 * eg * (u.abs() + eu) + ref.act(kind, g).abs() * eu + (U + 2.0 ** -14) * h.abs()
        assert ((H - h).abs() <= tol + 2.0 ** -100).all()


@pytest.mark.parametrize("T", [1, 2, 5, 16])
def test_gated_precise_few_tokens_is_the_same(T):
    say(f"gated precise T={T}")
    a, b = gauss_layer(200, 640, 3, "f16", 1), gauss_layer(200, 640, 3, "f16", 2)
    d, packed = gated_layer(a, b, "f16")
    X = gauss(T, 640, T)
    one, two = (run_gated(f, d, packed, X, "silu") for f in (bw.mbok_gated, bw.mbok_gated_precise))
    assert all(torch.equal(x, y) for x, y in zip(one, two))


@pytest.mark.parametrize("T,m,n", [(3, 9, 256), (40, 130, 384), (300, 200, 512)])
def test_gated_backward_precise(T, m, n):
    """dpre's bits are the one-term form's; dX is the product of that dpre."""
    for K, dt, kind in ((2, "f16", "silu"), (3, "f32", "gelu")):
        say(f"gated_backward precise T={T} m={m} n={n} K={K} {kind}")
        a, b = gauss_layer(m, n, K, dt, 3), gauss_layer(m, n, K, dt, 4)
        d, packed = gated_layer(a, b, dt)
        m2 = ref.stacked_rows(m)
        pre, dH = wide(gauss(T, m2, 1, 1.3), m2), wide(gauss(T, m, 3, 0.1), m + 1, off=1)
        dpre = [torch.empty(T, m2, dtype=BF, device=DEV) for _ in range(3)]
        dX = torch.full((T, n + 8), -4.0, dtype=BF, device=DEV)
        bw.mbok_gated_backward(d, packed, pre, dH, dpre[0], act=ACTS[kind])
        bw.mbok_gated_backward_precise(d, packed, pre, dH, dpre[1], act=ACTS[kind])
        bw.mbok_gated_backward_precise(d, packed, pre, dH, dpre[2], dX[:, :n], act=ACTS[kind])
        assert torch.equal(dpre[0], dpre[1]) and torch.equal(dpre[0], dpre[2])
        W = torch.zeros(m2, n, dtype=F64)
        ig, iu = ref.stack_index(m)
        W[ig], W[iu] = ref.dense(*a), ref.dense(*b)
        got = dpre[0].cpu().to(F64)
        x, bound = got @ W, got.abs() @ W.abs()
        tol = (2.0 ** -16 + 2 * m2 * 2.0 ** -24) * bound + U * x.abs()
        assert ((dX[:, :n].cpu().to(F64) - x).abs() <= tol).all()
        assert (dX[:, n:] == -4).all()


def test_precise_forms_in_a_graph():
    say("precise graph")
    T, m, n = 70, 300, 512
    a, b = gauss_layer(m, n, 3, "f16", 1), gauss_layer(m, n, 3, "f16", 2)
    d, packed = gated_layer(a, b, "f16")
    m2 = ref.stacked_rows(m)
    x, dH = wide(gauss(T, n, 1), n), wide(gauss(T, m, 2), m)
    out = [torch.empty(T, c, dtype=BF, device=DEV) for c in (m, m2, m2, n)]

    def step():
        bw.mbok_gated_precise(d, packed, x, out[0], pre=out[1])
        bw.mbok_gated_backward_precise(d, packed, out[1], dH, out[2], out[3])

    step()
    want = [o.clone() for o in out]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for o in out:
            o.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(out, want))
        bw.mbok_gemmt_precise(bw.mbok_gated_stack(d), packed, out[2], torch.empty_like(out[3]))
