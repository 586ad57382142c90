"""The skinny kernel's wait after its rotation phase, made to give up by the library's test hook,
with and without an epilogue: NaN everywhere, the status bit, and nothing left behind (arrival
counters, partial sums, the call counter) for the calls that follow."""
import numpy as np
import pytest

import oracle
from tests.gpu_util import Problem, to_numpy_f16
from tests.test_gpu_epilogue import G64, PQ2, PTQ1, Q1, SKINNY, bz, inputs_of, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("split_k,fmt,M,N,K", [
    (0, PQ2, 4, 1001, 1024), (4, PQ2, 16, 333, 4096), (1, Q1, 8, 200, 2048), (0, G64, 5, 130, 2048), (3, PTQ1, 9, 1001, 1920),
    (0, PQ2, 40, 1001, 1024), (3, PTQ1, 37, 129, 1920), (2, Q1, 100, 64, 640)])  # more than 16 tokens: with an epilogue only
def test_forced_timeouts_nan_status_and_recovery(bz, split_k, fmt, M, N, K):  # noqa: F811
    import torch
    p = Problem(M, N, K, fmt, seed=M + N)
    x, packed, scales = dev = p.device()
    bias, residual = inputs_of(p, 3)

    def plain():
        y = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
        bz.bonsai_ternary_linear_algo(x, packed, scales, y, M, N, K, fmt, SKINNY, split_k)
        torch.cuda.synchronize()
        return to_numpy_f16(y)

    calls = [lambda: run(bz, p, dev, bias, residual, 2, SKINNY, split_k)] + ([plain] if M <= 16 else [])
    bz.bonsai_device_status(clear=True)
    first = [c() for c in calls]
    assert all(np.isfinite(f).all() for f in first)
    if M <= 16:
        ok, rel, worst = oracle.compare(first[1], p.oracle_y())
        assert ok, (rel, worst)
    for c, f in zip(calls, first):
        bz.bonsai_debug_force_timeouts(True)
        try:
            got = c()
        finally:
            bz.bonsai_debug_force_timeouts(False)
        assert bz.bonsai_device_status(clear=True) == bz.BONSAI_DEVICE_SKINNY_TIMEOUT
        assert np.isnan(got).all()
        for _ in range(2):
            assert np.array_equal(c(), f)
        assert bz.bonsai_device_status() == 0
