"""Captured calls stay valid when a later call makes the library's workspace grow."""
import numpy as np
import pytest

import oracle
from tests import layer_ref as ref
from tests.gpu_util import Problem, to_numpy_f16
from tests.test_gpu_attention import f16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bz():
    import torch
    from ternary_weight_02_b200 import bonsai
    assert bonsai.bonsai_check_device() == bonsai.BONSAI_OK
    torch.cuda.init()
    return bonsai


def test_captured_calls_survive_growth(bz):
    """Attention, a split GEMM, a split skinny product and a split integer GEMV, captured with the
    smallest workspace, replayed after both its regions have grown and other memory was filled."""
    import torch
    torch.cuda.synchronize()
    bz.bonsai_shutdown()  # (no captured call of another test is replayed after this)
    bz.bonsai_reserve(1, 128, 128)
    rng = np.random.default_rng(1)
    pool = ref.Pool(rng, [3000, 20], 2, 128, 16, 0)
    d, q = pool.device(), f16(rng.normal(0, 2, (2, 8 * 128)).astype(np.float16))
    out = torch.zeros((2, 8 * 128), dtype=torch.float16, device="cuda")
    linears = []
    for M, N, K, algo, split in ((300, 1000, 640, bz.BONSAI_ALGO_GEMM, 0), (16, 333, 4096, bz.BONSAI_ALGO_SKINNY, 4),
                                 (1, 3000, 5120, bz.BONSAI_ALGO_IMMA, 0)):
        p = Problem(M, N, K, oracle.FMT_PQ2_0, seed=M)
        y = torch.zeros((M, N), dtype=torch.float16, device="cuda")
        linears.append((p.device(), p.oracle_y(), y, (M, N, K, p.fmt, algo, split)))

    def calls():
        bz.bonsai_paged_attention(q, *d, out, 2, 8)
        for (x, packed, scales), _, y, rest in linears:
            bz.bonsai_ternary_linear_algo(x, packed, scales, y, *rest)

    calls()
    torch.cuda.synchronize()
    first = [t.clone() for t in (out, *(y for _, _, y, _ in linears))]
    for _, want, y, _ in linears:
        assert oracle.compare(to_numpy_f16(y), want)[0]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        calls()
    filled = []
    for grow in ((1, 128, 128), (4096, 5120, 17408), (3, 4_000_000, 512)):  # nothing; the data; the zeroed region
        bz.bonsai_reserve(*grow)
        filled.append(torch.full((48 << 20,), 0x55555555, dtype=torch.int32, device="cuda"))
        for t in (out, *(y for _, _, y, _ in linears)):
            t.zero_()
        torch.cuda.synchronize()
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        for got, want in zip((out, *(y for _, _, y, _ in linears)), first):
            assert torch.equal(got, want)
        calls()  # and calls on the new one
        torch.cuda.synchronize()
        for got, want in zip((out, *(y for _, _, y, _ in linears)), first):
            assert torch.equal(got, want)
        assert all(bool((t == 0x55555555).all()) for t in filled)
        assert bz.bonsai_device_status() == 0
    # what a captured call reports is read, and cleared, in the region it was captured with
    d[5].fill_(-1)
    g.replay()
    assert bz.bonsai_device_status(clear=True) == bz.BONSAI_DEVICE_CACHE_RANGE
    assert bz.bonsai_device_status() == 0
    del g


def test_shutdown_after_growth_leaves_the_library_usable(bz):
    import torch
    bz.bonsai_reserve(2048, 5120, 17408)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    bz.bonsai_shutdown()
    assert torch.cuda.mem_get_info()[0] > free
    p = Problem(20, 64, 256, oracle.FMT_PQ2_0, seed=4)
    x, packed, scales = p.device()
    y = bz.ternary_linear(x, packed, scales, p.N, p.fmt)
    assert oracle.compare(to_numpy_f16(y), p.oracle_y())[0]
