"""GPU tests of mbok_linear's many-token kernels at the shapes that reach them, which
each test checks by the kernels' names: tiles in shares of the contraction whose groups
do not divide between them, in one term and in two, and contractions of many steps.

Exact regime, bounds: see test_gpu_finetune.py, test_gpu_finetune_precise.py and
test_gpu_linear.py.  The float64 products run on the GPU."""
import pytest
import torch

import boolean_weight_amd as bw
import finetune_ref
import step_ref as ref
from gpu_util import DEV, pack_on_gpu, say
from test_gpu_finetune import bf16_of, exact_layer, gauss, gauss_layer, ints, wide
from test_gpu_finetune_precise import small_ints, spread_layer
from test_gpu_linear import ACTS, bound_of, guards_hold

pytestmark = pytest.mark.gpu

F64, BF = torch.float64, torch.bfloat16
U, EPS = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bw.load_library()
    yield
    torch.cuda.synchronize()


def launches(call, *parts):
    """Checks that a call launches a kernel whose name holds the parts (where a tracer is
    there to say)."""
    torch.cuda.synchronize()
    kinds = [torch.profiler.ProfilerActivity.CUDA]
    with torch.profiler.profile(activities=kinds) as p:
        call()
        torch.cuda.synchronize()
    names = [e.name for e in p.events() if "mbok" in e.name]
    assert not names or any(all(x in n for x in parts) for n in names), names


def exact_case(T, m, n, K, layer, X):
    """Inputs of an exact call, guarded outputs, and what they have to be."""
    dt = "f16" if K % 2 else "f32"
    S, A = layer(m, n, K, dt, m + n + K)
    d, packed = pack_on_gpu(S, A, dt)
    W, R = finetune_ref.dense(S, A).to(DEV), ints(T, m, T + m)
    want, z = ref.linear(W, X.to(DEV), None, "none", R.to(DEV))
    buf = torch.full((T, m + 9), -5.0, device=DEV)
    pbuf = torch.full((T, m + 7), -5.0, dtype=BF, device=DEV)
    args = dict(residual=R.to(DEV), pre=pbuf[:, 3:3 + m])

    def check(call):
        call(d, packed, wide(X, n + 8, off=0), buf[:, 4:4 + m], **args)
        assert torch.equal(buf[:, 4:4 + m].to(F64), want)
        assert torch.equal(pbuf[:, 3:3 + m].to(F64), bf16_of(z))
        assert guards_hold(buf, 4, m) and guards_hold(pbuf, 3, m)
    return check


# groups of 5, 7 and 13 in four shares, and one each; 3 and 5 in two; ragged tokens and
# rows (the tiles' sizes, shares: 64 x 64, 4; 64 x 64, 2; 128 x 128, 2)
SHARES = [("Tile<2, 1, 1>, 4", 130, 4500, 640), ("Tile<2, 1, 1>, 4", 65, 8000, 896),
          ("Tile<2, 1, 1>, 4", 129, 5400, 512), ("Tile<2, 1, 1>, 4", 200, 4090, 1664),
          ("Tile<2, 1, 1>, 2", 300, 6100, 384), ("Tile<2, 1, 1>, 2", 260, 4200, 640),
          ("Tile<2, 2, 2>, 2", 700, 4000, 640), ("Tile<2, 2, 2>, 2", 1000, 4096, 512)]


@pytest.mark.parametrize("form,T,m,n", SHARES)
@pytest.mark.parametrize("K", [1, 2, 3, 4])
def test_shares_exact(form, T, m, n, K):
    say(f"linear shares T={T} m={m} n={n} K={K}")
    check = exact_case(T, m, n, K, exact_layer, ints(T, n, T + n))
    launches(lambda: check(bw.mbok_linear), "linear_shares_kernel", f"{form}, false")
    check(bw.mbok_linear)


@pytest.mark.parametrize("form,T,m,n", [
    ("Tile<2, 1, 1>, 4", 130, 4500, 640), ("Tile<2, 1, 1>, 4", 129, 5400, 512),
    ("Tile<2, 1, 1>, 2", 300, 6100, 640), ("Tile<2, 2, 2>, 2", 700, 4000, 640),
    ("Tile<2, 2, 2>, 2", 1000, 4096, 512)])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
def test_shares_two_terms_exact(form, T, m, n, K):
    say(f"linear shares, two terms T={T} m={m} n={n} K={K}")
    check = exact_case(T, m, n, K, spread_layer, small_ints(T, n, T + n, 100))
    launches(lambda: check(bw.mbok_linear_precise), "linear_shares_kernel", f"{form}, true")


# whole rounds and halves of what is left, halves alone, whole tiles, tiles of 128 and of
# 64: 17 to 66 steps of 64 columns, where the kernel's buffers turn over many times
LONG = [("Tile<2, 4, 4>", 4096, 4400, 1152), ("Tile<2, 4, 4>", 1300, 4099, 4096),
        ("Tile<2, 4, 4>", 2048, 5000, 2176), ("Tile<2, 2, 2>", 2048, 2300, 4224),
        ("Tile<2, 1, 1>", 50, 33000, 1152)]


@pytest.mark.parametrize("form,T,m,n", LONG)
@pytest.mark.parametrize("K", [1, 2, 3, 4])
def test_long_contractions_exact(form, T, m, n, K):
    """Sums below 2^15 (n K / 2) and multiples of 2^-8: exact in fp32."""
    say(f"linear long T={T} m={m} n={n} K={K}")
    check = exact_case(T, m, n, K, exact_layer, ints(T, n, T + n))
    launches(lambda: check(bw.mbok_linear), "linear_mfma_kernel", f"{form}, false")


@pytest.mark.parametrize("form,T,m,n", LONG + [("Tile<2, 1, 1>, 4", 200, 4090, 4096),
                                               ("Tile<2, 2, 2>, 2", 700, 4000, 4096)])
@pytest.mark.parametrize("K", [2, 3])
def test_long_contractions_gaussian(form, T, m, n, K):
    """Both forms, with bias, activation and residual."""
    say(f"linear long gaussian T={T} m={m} n={n} K={K}")
    S, A = gauss_layer(m, n, K, "f16", m + n)
    d, packed = pack_on_gpu(S, A, "f16")
    X, R = gauss(T, n, T + n), gauss(T, m, T + m)
    bias = gauss(1, m, 4, 0.3)[0].to(DEV)
    W, Xd, Rd = finetune_ref.dense(S, A).to(DEV), X.to(F64).to(DEV), R.to(F64).to(DEV)
    want, z = ref.linear(W, Xd, bias, "gelu", Rd)
    for name in ("mbok_linear", "mbok_linear_precise"):
        y = torch.empty(T, m, device=DEV)
        pre = torch.empty(T, m, dtype=BF, device=DEV)
        getattr(bw, name)(d, packed, wide(X, n), y, bias=bias, act=ACTS["gelu"],
                          residual=R.to(DEV), pre=pre)
        D = bound_of(16 if name.endswith("precise") else T, W, Xd, z)
        tol = 1.13 * D + 4 * EPS * (z.abs() + Rd.abs() + want.abs()) + EPS * want.abs()
        assert ((y.to(F64) - want).abs() <= tol).all(), name
        assert ((pre.to(F64) - z).abs() <= D + U * z.abs()).all(), name
