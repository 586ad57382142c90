"""The kernel that calls with an epilogue choose, where the automatic choice meets an argument
that is the GEMM's."""
import pytest

import oracle
from tests.gpu_util import Problem, to_numpy_f16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bz():
    import torch
    from ternary_weight_02_b200 import bonsai
    assert bonsai.bonsai_check_device() == bonsai.BONSAI_OK
    torch.cuda.init()
    return bonsai


@pytest.mark.parametrize("with_residual", [False, True])
def test_cta_pairs_are_refused_whatever_chose_the_gemm(bz, with_residual):
    """split_k = 3 asks the GEMM for CTA pairs, which calls with an epilogue do not have: refused
    where the automatic choice is the GEMM as where the caller's is, with or without the three;
    three K chunks where the choice is the skinny kernel."""
    import torch
    p = Problem(1040, 256, 256, oracle.FMT_PQ2_0, seed=1)  # more tokens than the skinny kernel takes
    x, packed, scales = p.device()
    y = torch.full((p.M, p.N), 7.0, dtype=torch.float16, device="cuda")
    r = torch.zeros_like(y) if with_residual else None
    for algo in (bz.BONSAI_ALGO_AUTO, bz.BONSAI_ALGO_GEMM):
        with pytest.raises(bz.BonsaiError) as e:
            bz.bonsai_ternary_linear_epilogue(x, packed, scales, None, r, y, p.M, p.N, p.K, p.fmt, 0, algo, 3)
        assert e.value.status == bz.BONSAI_ERR_ALGO
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())
    bz.bonsai_ternary_linear_epilogue(x, packed, scales, None, r, y, 4, p.N, p.K, p.fmt, 0, bz.BONSAI_ALGO_AUTO, 3)
    ok, rel, worst = oracle.compare(to_numpy_f16(y[:4]), oracle.ternary_linear(p.x[:4], p.oracle_packed(), p.scales, p.N, p.K,
                                                                             p.fmt))
    assert ok, (rel, worst)
