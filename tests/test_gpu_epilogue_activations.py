"""The activations of bonsai_ternary_linear_epilogue by themselves: activations x of zero make the
product exactly zero, so that the bias alone is the argument and each output is held to half a
step of FP16 and the arithmetic of its own activation, on every kernel that has an epilogue."""
import numpy as np
import pytest

import oracle
from tests import layer_ref as ref
from tests.gpu_util import Problem, to_numpy_f16
from tests.test_gpu_epilogue import GEMM, GEMV, IMMA, KERNELS, PQ2, SIMPLE, SKINNY, f16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bz():
    import torch
    from ternary_weight_02_b200 import bonsai
    assert bonsai.bonsai_check_device() == bonsai.BONSAI_OK
    torch.cuda.init()
    return bonsai


def all_f16_to_12():
    """Every FP16 value of magnitude 12 or less, in order."""
    pos = np.arange(0, np.float16(12).view(np.uint16) + 1, dtype=np.uint16)
    return np.concatenate([(pos[::-1] | 0x8000).astype(np.uint16).view(np.float16), pos.view(np.float16)])


def slack(z, act):
    """Error of an activation's FP32 evaluation.  With u = 2^-24: 2^x and 1 / x of the special
    function unit are off by 4u and 2u, a product by u, an exponent w by 3u |w| of itself (its
    constant, one or two products), which moves 2^w by 3u |w| ln 2 of itself.
      SiLU, tanh-GELU: z / (1 + 2^w), relative: exponent, exponential, sum, reciprocal, product.
      GELU: erfc's rational form is off by 1.5e-7 (its publication), halved and times z; its
      five terms (coefficients of 2.2 in all, with k |c_k| of 8.1 for the error of t) carry 2^-18
      of their factor e^(-z^2 / 2); the exponent z^2 / 2 as above; one subtraction."""
    u, a = 2.0 ** -24, np.abs(z)
    value = np.abs(ref.activate(z, act))
    if act == 2:
        return value * u * (9 + 3 * a)
    if act == 4:  # w = 1.6 (z + 0.0447 z^3) log2 e, three more roundings in the polynomial
        return value * u * (12 + 6 * 1.6 * (a + 0.0447 * a ** 3))
    if act == 3:
        return a * (0.75e-7 + 2.0 ** -18 * np.exp(-z * z / 2)) + value * u * (8 + 1.5 * z * z) + u * a
    return np.zeros_like(a)


def check(got, z, residual, act):
    value = ref.activate(z, act)
    want = value if residual is None else value + residual
    bound = ref.H16 * np.abs(want) + ref.TINY16 + (slack(z, act) + 2.0 ** -24 * np.abs(want)) * (1 + ref.H16)
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), np.broadcast_to(z, got.shape)[bad][:4], got[bad][:4], np.broadcast_to(want, got.shape)[bad][:4])


def test_the_bound_tells_the_two_gelus_apart():
    """(On the host's numbers alone.)  Each form, rounded to FP16, is outside the other's bound."""
    z = all_f16_to_12().astype(np.float64)
    for act, other in ((3, 4), (4, 3)):
        with pytest.raises(AssertionError):
            check(ref.activate(z, other).astype(np.float16).astype(np.float64)[None], z, None, act)
        check(ref.activate(z, act).astype(np.float16).astype(np.float64)[None], z, None, act)


def run(bz, p, dev, bias, residual, act, algo, split_k):
    import torch
    _, packed, scales = dev
    x = torch.zeros((p.M, p.K), dtype=torch.float16, device="cuda")
    y = torch.full((p.M, p.N), float("nan"), dtype=torch.float16, device="cuda")
    bz.bonsai_ternary_linear_epilogue(x, packed, scales, f16(bias), None if residual is None else f16(residual), y, p.M, p.N,
                                      p.K, p.fmt, act, algo, split_k)
    torch.cuda.synchronize()
    return to_numpy_f16(y)


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: "algo%d-s%d-f%d-%dx%dx%d" % k)
def test_activations_of_the_bias_on_every_kernel(bz, kernel):
    algo, split_k, fmt, M, N, K = kernel
    p = Problem(M, N, K, fmt, seed=1)
    dev = p.device()
    values = all_f16_to_12()
    rng = np.random.default_rng(N)
    bias = values[(np.arange(N) * (len(values) - 1)) // max(N - 1, 1)]
    bias[: min(N, 40)] = rng.uniform(-5, 5, min(N, 40)).astype(np.float16)  # where the activations bend
    residual = rng.normal(0, 0.05, (M, N)).astype(np.float16)
    z = bias.astype(np.float64)
    for act in range(5):
        check(run(bz, p, dev, bias, None, act, algo, split_k), z, None, act)
    for act in (3, 4):
        check(run(bz, p, dev, bias, residual, act, algo, split_k), z, residual.astype(np.float64), act)


@pytest.mark.parametrize("algo,M", [(SIMPLE, 1), (GEMV, 1), (IMMA, 1), (SKINNY, 4), (SKINNY, 40), (GEMM, 20)])
def test_every_f16_value_to_12(bz, algo, M):
    values = all_f16_to_12()
    p = Problem(M, len(values), 512, PQ2, seed=2)
    dev = p.device()
    for act in range(5):
        check(run(bz, p, dev, values, None, act, algo, 0), values.astype(np.float64), None, act)
