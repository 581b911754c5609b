"""Paths of the fine-tuning operators that training and decoding take: 16-byte
aligned rows copied straight to LDS over several steps, every token tile, whole
tiles beside sliced ones, every count of tiles per workgroup of the decode
forms, several column slabs.  Exact regime: a result is the float64 one after
its single rounding.  And float16 gradients of the distillation at their own
smallest step."""
import math

import pytest
import torch

import boolean_weight_amd as bw
import distill_ref
import finetune_ref as ref
from gpu_util import DEV, pack_on_gpu, say
from test_gpu_finetune import (BF, F64, U, bf16_of, exact_layer, garbage, gated_layer, gated_want,
                               ints, run_gated, wide)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------- transposed product

def check_gemmt(T, m, n, K, dt):
    S, A = exact_layer(m, n, K, dt, 11 * m + n + K)
    d, packed = pack_on_gpu(S, A, dt)
    dY = ints(T, m, T + 2 * m)
    y = wide(dY, (m + 15) // 8 * 8, off=8 if m % 8 == 0 else 0)
    assert y.data_ptr() % 16 == 0 and y.stride(0) % 8 == 0
    want = bf16_of((dY.to(F64).to(DEV) @ ref.dense(S, A).to(DEV)).cpu())
    for ws in (garbage(bw.mbok_gemmt_workspace_bytes(d, T)), None):
        out = torch.full((T, n + 16), -5.0, dtype=BF, device=DEV)
        bw.mbok_gemmt(d, packed, y, out[:, 8:8 + n], workspace=ws)
        assert torch.equal(out[:, 8:8 + n].cpu().to(F64), want)
        assert (out[:, :8] == -5).all() and (out[:, 8 + n:] == -5).all()


# token tiles of 32, 64, 128 and 256 (few columns or rows lower them), each with
# rows that fill the last 64-row block and rows that do not
@pytest.mark.parametrize("T,m,n", [(20, 2048, 4096), (32, 1000, 2048), (50, 2048, 4096),
                                   (64, 1928, 4096), (100, 4096, 2048), (128, 2056, 3968),
                                   (200, 4096, 1408), (300, 1024, 4096), (513, 712, 4224),
                                   (96, 64, 128), (40, 200, 640)])
def test_gemmt_aligned(T, m, n):
    for K, dt in ((1, "f16"), (2, "f32"), (3, "f16"), (4, "f16")):
        say(f"gemmt aligned T={T} m={m} n={n} K={K} {dt}")
        check_gemmt(T, m, n, K, dt)


@pytest.mark.parametrize("T,m,n", [(2049, 520, 7680), (1025, 320, 13312), (4096, 192, 4096),
                                   (4100, 200, 4096)])
@pytest.mark.parametrize("K,dt", [(1, "f32"), (2, "f16"), (3, "f16"), (4, "f32")])
def test_gemmt_aligned_whole_and_sliced(T, m, n, K, dt):
    """More than 256 tiles: 256 or 512 whole, the others in slices (or none)."""
    say(f"gemmt whole and sliced T={T} m={m} n={n} K={K} {dt}")
    check_gemmt(T, m, n, K, dt)


# ---------------------------------------------------------- scale gradients

@pytest.mark.parametrize("m", [256, 520, 1032])
@pytest.mark.parametrize("T", [128, 192, 257, 1000])
def test_scale_grad_aligned(T, m):
    """Whole tiles of aligned rows, of two to fifteen steps; the tile across the
    last row goes by way of registers."""
    n = 384
    for K, dt in ((1, "f32"), (2, "f16"), (3, "f16"), (4, "f32")):
        say(f"scale_grad aligned T={T} m={m} K={K}")
        S, A = exact_layer(m, n, K, dt, 5 * m + T + K)
        d, packed = pack_on_gpu(S, A, dt)
        dY, X = ints(T, m, T + m), ints(T, n, T + n + 1)
        y, x = wide(dY, m + 16, off=8), wide(X, n + 8, off=8)
        assert y.data_ptr() % 16 == 0 and y.stride(0) % 8 == 0
        want = ref.scale_grad(S, dY, X)
        for ws in (garbage(bw.mbok_scale_grad_workspace_bytes(d, T)), None):
            out = torch.full((want.numel() + 8,), -3.0, device=DEV)
            bw.mbok_scale_grad(d, packed, y, x, out[4:-4], workspace=ws)
            assert torch.equal(out[4:-4].cpu().to(F64).view_as(want), want)
            assert (out[:4] == -3).all() and (out[-4:] == -3).all()


def test_scale_grad_aligned_many_tiles():
    """More tiles than compute units, no slices."""
    T, m, n, K = 320, 4360, 4224, 2
    say(f"scale_grad aligned T={T} m={m} n={n}")
    S, A = exact_layer(m, n, K, "f16", 8)
    d, packed = pack_on_gpu(S, A, "f16")
    dY, X = ints(T, m, 1), ints(T, n, 2)
    out = torch.empty(K, m, n // 128, device=DEV)
    bw.mbok_scale_grad(d, packed, wide(dY, m), wide(X, n), out)
    dW = dY.to(F64).to(DEV).t() @ X.to(F64).to(DEV)
    for k in range(K):
        sign = torch.as_tensor(S[k]).to(DEV)
        assert torch.equal(out[k].to(F64), (dW * sign).view(m, -1, 128).sum(-1))


# ---------------------------------------------------------- the gated block

def check_gated(T, m, n, K, dt, kind):
    a, b = exact_layer(m, n, K, dt, m + n + K), exact_layer(m, n, K, dt, 3 * m + n + K)
    d, packed = gated_layer(a, b, dt)
    X = ints(T, n, T + n)
    X[X.abs() > 2] = 0
    g, u, h = gated_want(a, b, X, kind)
    H, pre = run_gated(d, packed, X, kind)
    assert torch.equal(pre, bf16_of(ref.stack(g, u)))
    assert ((H - h).abs() <= (U + 2.0 ** -14) * h.abs() + 2.0 ** -100).all()


@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("m", [2041, 2100, 3500, 5000, 8100, 11000, 16000, 17000])
def test_gated_tiles_per_workgroup(T, m):
    """One to eight 16-row tiles per workgroup, most with some workgroups a tile
    short, and more workgroups than compute units (17000 rows)."""
    for K, dt, kind in ((1, "f32", "gelu"), (3, "f16", "silu")):
        say(f"gated T={T} m={m} K={K} {dt} {kind}")
        check_gated(T, m, 256, K, dt, kind)


@pytest.mark.parametrize("T", [1, 2, 5, 8])
@pytest.mark.parametrize("m,n", [(300, 8192), (2500, 8192), (700, 13056)])
def test_gated_column_slabs(T, m, n):
    """Inputs wider than a workgroup's wavefronts hold at once."""
    for K, dt, kind in ((2, "f16", "silu"), (4, "f32", "gelu")):
        say(f"gated T={T} m={m} n={n} K={K} {dt}")
        check_gated(T, m, n, K, dt, kind)


@pytest.mark.parametrize("T", [3, 6, 7, 8, 9])
def test_gated_large_layer_few_tokens(T):
    """A layer large enough for the per-group form at 3 to 8 tokens."""
    say(f"gated large layer T={T}")
    check_gated(T, 6000, 4096, 3, "f16", "silu")


# ------------------------------------------------------------- distillation

@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("V,top", [(900, 12), (33001, 64)])
def test_distill_float16_gradients(V, top, rest):
    """Mean over the rows under a loss scale of 4096, and weight 1: unlisted
    gradients far below float16's smallest normal value are kept to half its
    smallest step, 2^-25."""
    T = 6
    for scale in (4096.0 / T, 1.0):
        say(f"distill f16 V={V} rest={rest} weight={scale}")
        gen = torch.Generator().manual_seed(V)
        teacher = torch.randn(T, V, generator=gen) * 2.5
        Z = (teacher + torch.randn(T, V, generator=gen)).half()
        l, idx = teacher.topk(top, -1)
        lse = torch.logsumexp(teacher, -1) if rest else None
        w = torch.full((T,), scale)
        d = bw.mbok_distill_desc_init(V, top, 1.0)
        dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        loss, dZ = torch.empty(T, device=DEV), torch.empty(T, V, dtype=torch.float16, device=DEV)
        args = [dev(Z), dev(l.contiguous()), dev(idx.to(torch.int32))]
        stats = torch.empty(T, bw.MBOK_DISTILL_STATS, device=DEV)
        for two in (False, True):
            dZ.fill_(math.nan)
            bw.mbok_distill(d, *args, loss, stats=stats if two else None,
                            dZ=None if two else dZ, t_lse=dev(lse), weight=dev(w))
            if two:
                bw.mbok_distill_backward(d, *args, stats, torch.ones(T, device=DEV), dZ,
                                         t_lse=dev(lse), weight=dev(w))
            _, want, size = distill_ref.distill(Z, l, idx, 1.0, lse, w)
            got = dZ.cpu().to(F64)
            tol = 2.0 ** -16 * size + 2.0 ** -11 * want.abs() + 2.0 ** -25
            assert ((got - want).abs() <= tol).all(), ((got - want).abs() - tol).max()
            small = (want.abs() < 2.0 ** -14) & (want.abs() > 2.0 ** -23)
            assert small.any() and (got[small] != 0).all()
