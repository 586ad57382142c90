"""bonsai_ternary_linear_epilogue on the GPU: bias, activation and residual on every kernel
and packing, against the float64 checker's product and the float64 epilogue."""
import numpy as np
import pytest

import oracle
from tests import layer_ref as ref
from tests.gpu_util import Problem, to_numpy_f16

pytestmark = pytest.mark.gpu

PTQ1, PQ2, Q1, G64 = oracle.FMT_PTQ1_0, oracle.FMT_PQ2_0, oracle.FMT_Q1_0, oracle.FMT_PQ2_0_G64
AUTO, SIMPLE, GEMV, SKINNY, GEMM, IMMA = range(6)


@pytest.fixture(scope="module")
def bz():
    import torch
    from ternary_weight_02_b200 import bonsai
    assert bonsai.bonsai_check_device() == bonsai.BONSAI_OK
    torch.cuda.init()
    return bonsai


def f16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.float16)


def inputs_of(p, seed):
    rng = np.random.default_rng(seed)
    return rng.normal(0, 1, p.N).astype(np.float16), rng.normal(0, 4, (p.M, p.N)).astype(np.float16)


def run(bz, p, dev, bias, residual, act, algo=AUTO, split_k=0, in_place=False):
    import torch
    x, packed, scales = dev
    y = torch.full((p.M, p.N), float("nan"), dtype=torch.float16, device="cuda")
    r = None if residual is None else f16(residual)
    if in_place:
        y = r
    bz.bonsai_ternary_linear_epilogue(x, packed, scales, None if bias is None else f16(bias), r, y, p.M, p.N, p.K, p.fmt,
                                      act, algo, split_k)
    torch.cuda.synchronize()
    return to_numpy_f16(y)


def check(got, prod, bias, residual, act):
    """The product's bar carried through the epilogue: the product z may be off by 1e-2 rms(z)
    anywhere and by 1e-3 in rel-L2 (the linear layer's bar); no activation's slope exceeds
    1.13; its own FP32 evaluation adds 2^-20 |.|, the rounding half a step."""
    z = prod if bias is None else prod + bias.astype(np.float64)
    a = ref.activate(z, act)
    want = a if residual is None else a + residual.astype(np.float64)
    rms = np.sqrt(np.mean(prod ** 2))
    err = np.abs(got - want)
    fp32 = 2.0 ** -20 * (np.abs(a) + np.abs(z))
    bound = 1.13e-2 * rms + ref.H16 * np.abs(want) + ref.TINY16 + fp32
    assert (err <= bound).all(), (float((err / bound).max()), float(rms))
    l2 = 1.13e-3 * np.linalg.norm(prod) + ref.H16 * np.linalg.norm(want) + np.linalg.norm(fp32)
    assert np.linalg.norm(err) <= l2, (np.linalg.norm(err), l2)


KERNELS = [  # algo, split_k, fmt, M, N, K
    (SIMPLE, 0, PTQ1, 3, 40, 256), (SIMPLE, 0, PQ2, 1, 33, 128), (SIMPLE, 0, Q1, 5, 17, 384), (SIMPLE, 0, G64, 2, 64, 256),
    (GEMV, 1, PQ2, 1, 1001, 5120), (GEMV, 2, PQ2, 1, 1001, 1024), (GEMV, 2, PTQ1, 1, 777, 2048), (GEMV, 1, PTQ1, 1, 333, 5120),
    (GEMV, 0, PQ2, 1, 50, 512), (GEMV, 0, Q1, 1, 1001, 2048), (GEMV, 0, G64, 1, 100, 1024),
    (IMMA, 0, PQ2, 1, 5120, 5120), (IMMA, 0, PQ2, 1, 1, 128), (IMMA, 0, PQ2, 1, 1001, 640), (IMMA, 0, G64, 1, 1000, 1024),
    (IMMA, 0, PQ2, 2, 777, 2048), (IMMA, 0, G64, 2, 129, 384), (IMMA, 0, PQ2, 3, 1001, 1152),
    (SKINNY, 0, PQ2, 4, 1001, 1024), (SKINNY, 1, PQ2, 8, 200, 2048), (SKINNY, 4, PQ2, 16, 333, 4096), (SKINNY, 0, PTQ1, 2, 100, 640),
    (SKINNY, 3, PTQ1, 9, 1001, 1920), (SKINNY, 0, Q1, 7, 65, 1024), (SKINNY, 0, Q1, 16, 500, 384), (SKINNY, 0, G64, 5, 130, 2048),
    (SKINNY, 2, G64, 12, 64, 1280),
    (SKINNY, 0, PQ2, 17, 1001, 1024), (SKINNY, 0, Q1, 100, 1001, 1024), (SKINNY, 3, PTQ1, 37, 129, 1920), (SKINNY, 1, G64, 256, 64, 2048),
    (SKINNY, 4, G64, 33, 500, 4096), (SKINNY, 0, PQ2, 1000, 700, 128), (SKINNY, 2, PTQ1, 48, 16, 640), (SKINNY, 0, PQ2, 64, 5120, 5120),
    (GEMM, 1, PQ2, 100, 1001, 1024), (GEMM, 2, PQ2, 300, 520, 640), (GEMM, 0, PTQ1, 33, 300, 1280), (GEMM, 0, Q1, 129, 257, 512),
    (GEMM, 0, G64, 257, 256, 384), (GEMM, 2, PTQ1, 513, 1000, 256), (GEMM, 0, PQ2, 17, 5, 128), (GEMM, 0, Q1, 20, 1024, 5120)]


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: "algo%d-s%d-f%d-%dx%dx%d" % k)
def test_epilogue_on_every_kernel(bz, kernel):
    algo, split_k, fmt, M, N, K = kernel
    p = Problem(M, N, K, fmt, seed=M + N + K)
    dev, prod = p.device(), p.oracle_y()
    bias, residual = inputs_of(p, N)
    for b, r, act in ((bias, residual, 2), (bias, None, 3), (None, residual, 0), (bias, residual, 4), (None, None, 1),
                      (bias, None, 0)):
        got = run(bz, p, dev, b, r, act, algo, split_k)
        check(got, prod, b, r, act)
    # the residual stream updated in place gives the same bits
    assert np.array_equal(run(bz, p, dev, bias, residual, 1, algo, split_k, in_place=True),
                          run(bz, p, dev, bias, residual, 1, algo, split_k))
    assert bz.bonsai_device_status(clear=True) == 0


@pytest.mark.parametrize("kernel", [k for k in KERNELS if not (k[0] == SKINNY and k[3] > 16)],
                         ids=lambda k: "algo%d-s%d-f%d-%dx%dx%d" % k)
def test_no_epilogue_is_the_plain_product(bz, kernel):
    """Without bias, activation and residual the call gives the bits of bonsai_ternary_linear_algo."""
    import torch
    algo, split_k, fmt, M, N, K = kernel
    p = Problem(M, N, K, fmt, seed=M + N + K)
    x, packed, scales = dev = p.device()
    y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    bz.bonsai_ternary_linear_algo(x, packed, scales, y, M, N, K, fmt, algo, split_k)
    torch.cuda.synchronize()
    assert np.array_equal(run(bz, p, dev, None, None, 0, algo, split_k), to_numpy_f16(y))


@pytest.mark.parametrize("fmt", [PTQ1, PQ2, Q1, G64])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 16, 17, 130])
def test_automatic_choice(bz, fmt, M):
    p = Problem(M, 600, 1024, fmt, seed=M)
    bias, residual = inputs_of(p, M)
    check(run(bz, p, p.device(), bias, residual, 3), p.oracle_y(), bias, residual, 3)


@pytest.mark.parametrize("N,K,M", [(5120, 5120, 1), (5120, 17408, 1), (5120, 17408, 700)])
def test_full_projections(bz, N, K, M):
    p = Problem(M, N, K, PQ2, seed=3)
    _, residual = inputs_of(p, 3)
    rows = slice(0, 4)  # the checker on the first rows only
    got = run(bz, p, p.device(), None, residual, 0, in_place=True)
    p2 = p.x
    p.x, p.M = p2[rows], len(p2[rows])
    check(got[rows], p.oracle_y(), None, residual[rows], 0)
    assert np.isfinite(got).all()


def test_nan_stays_nan_through_activations(bz):
    """A NaN activation makes its token's row NaN for every activation; the other rows stay finite."""
    for M, N, K, algo in ((1, 64, 512, AUTO), (4, 64, 512, AUTO), (20, 64, 512, AUTO), (2, 64, 512, SIMPLE)):
        p = Problem(M, N, K, PTQ1, seed=1)
        p.x = p.x.copy()
        p.x[M - 1, 5] = np.nan
        for act in range(5):
            got = run(bz, p, p.device(), None, None, act, algo)
            assert np.isnan(got[M - 1]).all(), (M, act)
            assert np.isfinite(got[: M - 1]).all(), (M, act)


@pytest.mark.parametrize("M,N,K,algo", [(1, 4000, 5120, IMMA), (3, 2000, 2048, IMMA), (300, 1000, 4096, GEMM)])
def test_forced_timeouts_reach_the_output(bz, M, N, K, algo):
    """Where a hand-over is made to give up, the epilogue leaves NaN exactly where the plain product
    has it (the same tiles are split in both), and the next call is right."""
    import torch
    p = Problem(M, N, K, PQ2, seed=2)
    bias, residual = inputs_of(p, 2)
    x, packed, scales = dev = p.device()
    y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    bz.bonsai_debug_force_timeouts(True)
    try:
        bz.bonsai_ternary_linear_algo(x, packed, scales, y, M, N, K, PQ2, algo)
        torch.cuda.synchronize()
        got = run(bz, p, dev, bias, residual, 1, algo)
    finally:
        bz.bonsai_debug_force_timeouts(False)
    assert np.array_equal(np.isnan(got), np.isnan(to_numpy_f16(y)))
    assert bz.bonsai_device_status(clear=True) != 0
    check(run(bz, p, dev, bias, residual, 1, algo), p.oracle_y(), bias, residual, 1)
    assert bz.bonsai_device_status(clear=True) == 0


@pytest.mark.parametrize("algo", [SIMPLE, GEMV, SKINNY, GEMM])
@pytest.mark.parametrize("act", range(5))
def test_infinite_sums(bz, act, algo):
    """A bias of +-infinity gives the activation's value there (0 times infinity is a NaN); its
    neighbours are what they are without it."""
    import warnings
    p = Problem(1, 300, 512, PQ2, seed=41)
    dev = p.device()
    bias, _ = inputs_of(p, 42)
    plain = run(bz, p, dev, bias, None, act, algo)
    bias[[5, 299]], bias[[6, 17]] = np.inf, -np.inf
    got = run(bz, p, dev, bias, None, act, algo)
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        up, down = float(ref.activate(np.array([np.inf]), act)[0]), float(ref.activate(np.array([-np.inf]), act)[0])
    assert up == np.inf and (got[0, [5, 299]] == np.inf).all()
    assert np.array_equal(got[0, [6, 17]], [down, down], equal_nan=True)
    others = np.setdiff1d(np.arange(300), [5, 6, 17, 299])
    assert np.array_equal(got[0, others], plain[0, others])
