"""Without a GPU: the frequencies of rotary positions, and the refusals of the decode layer's
operators, which are made on the host before any device is touched."""
import math

import numpy as np
import pytest

from tests import layer_ref as ref

GOOD = 1 << 20  # an aligned non-null value; a refused call never uses it
SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


@pytest.fixture(scope="module")
def bz():
    from ternary_weight_02_b200 import build
    build.build()
    from ternary_weight_02_b200 import bonsai
    return bonsai


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("R,base,factor,original,low,high", [
    (128, 1e6, 4.0, 32768, 1.0, 32.0), (64, 1e4, 8.0, 8192, 1.0, 4.0), (2, 1e4, 2.0, 4096, 1.0, 32.0),
    (0, 1e4, 2.0, 4096, 1.0, 32.0), (6, 500000.0, 1.0, 2048, 0.5, 2.0), (256, 1e7, 32.0, 100, 1.0, 32.0)])
def test_frequencies(bz, scaling, R, base, factor, original, low, high):
    f, mag = bz.bonsai_rope_frequencies(R, base, SCALINGS[scaling], factor, original, low, high)
    want, want_mag = ref.frequencies(R, base, scaling, factor, original, low, high)
    # a power, a product and a blend in FP64: a few roundings, and the exponent's own rounding
    # (2^-53 of up to ln(base) ~ 19) carried through the power
    assert f.shape == (R // 2,)
    np.testing.assert_allclose(f.numpy(), want, rtol=1e-13)
    assert math.isclose(mag, want_mag, rel_tol=1e-14)


def test_frequencies_ends(bz):
    """YaRN and bands keep the fast pairs and divide the slow ones by the factor."""
    plain, _ = bz.bonsai_rope_frequencies(128, 1e6)
    for scaling in (bz.BONSAI_ROPE_YARN, bz.BONSAI_ROPE_BANDS):
        f, _ = bz.bonsai_rope_frequencies(128, 1e6, scaling, 4.0, 32768.0, 1.0, 32.0)
        assert f[0] == plain[0] and f[-1] == plain[-1] / 4
        assert bool(((f <= plain) & (f >= plain / 4)).all())


def test_frequencies_refusals(bz):
    import ctypes
    L = bz.raw()
    buf = (ctypes.c_double * 64)()
    mag = ctypes.c_double()

    def call(R=128, base=1e4, scaling=0, factor=2.0, original=4096.0, low=1.0, high=32.0, out=buf, m=mag):
        return L.bonsai_rope_frequencies(out, ctypes.byref(m) if m is not None else None, R, base, scaling, factor,
                                         original, low, high)
    assert call() == bz.BONSAI_OK
    assert call(R=7) == call(R=-2) == call(R=2048) == bz.BONSAI_ERR_SHAPE
    nan, inf = float("nan"), float("inf")
    for base in (1.0, 0.5, -3.0, nan, inf):
        assert call(base=base) == bz.BONSAI_ERR_ARG, base
    for scaling in (-1, 5):
        assert call(scaling=scaling) == bz.BONSAI_ERR_ARG
    for scaling in (1, 2, 3, 4):
        for factor in (0.5, 0.0, nan, inf):
            assert call(scaling=scaling, factor=factor) == bz.BONSAI_ERR_ARG
    for scaling in (3, 4):
        for kw in ({"original": 0.0}, {"original": nan}, {"low": 0.0}, {"low": 32.0}, {"high": nan}, {"high": inf}):
            assert call(scaling=scaling, **kw) == bz.BONSAI_ERR_ARG, kw
    assert call(out=None) == bz.BONSAI_ERR_NULL
    assert call(m=None) == bz.BONSAI_ERR_NULL
    assert call(R=0, out=None) == bz.BONSAI_OK


def test_epilogue_refusals(bz):
    def call(x=GOOD, packed=GOOD, scales=GOOD, bias=GOOD, residual=GOOD, y=GOOD, M=1, N=8, K=128, fmt=2, act=0, algo=0,
             split_k=0):
        return bz.raw().bonsai_ternary_linear_epilogue(x, packed, scales, bias, residual, y, M, N, K, fmt, act, algo,
                                                       split_k, None)
    for name in ("x", "packed", "scales", "y"):
        assert call(**{name: None}) == bz.BONSAI_ERR_NULL, name
    for name in ("x", "packed", "scales", "bias", "residual", "y"):
        assert call(**{name: GOOD + 2}) == bz.BONSAI_ERR_ALIGN, name
    assert call(fmt=0) == call(fmt=5) == bz.BONSAI_ERR_FMT
    assert call(act=-1) == call(act=5) == bz.BONSAI_ERR_ARG
    for kw in ({"K": 100}, {"K": 0}, {"M": -1}, {"N": -1}, {"split_k": -1}, {"M": 1 << 32}):
        assert call(**kw) == bz.BONSAI_ERR_SHAPE, kw
    assert call(algo=9) == bz.BONSAI_ERR_ALGO
    assert call(algo=bz.BONSAI_ALGO_GEMV, M=2) == bz.BONSAI_ERR_ALGO
    assert call(algo=bz.BONSAI_ALGO_GEMM, split_k=3) == bz.BONSAI_ERR_ALGO
    assert call(M=0, x=None) == call(N=0, y=None) == bz.BONSAI_OK


def test_rope_refusals(bz):
    def call(x=GOOD, out=GOOD, freqs=GOOD, positions=GOOD, T=4, H=2, D=64, R=64, ld_x=128, ld_out=128, layout=0):
        return bz.raw().bonsai_rope(x, out, freqs, positions, T, H, D, R, ld_x, ld_out, 1.0, layout, None)
    for name in ("x", "out", "freqs", "positions"):
        assert call(**{name: None}) == bz.BONSAI_ERR_NULL, name
    for name, off in (("x", 8), ("out", 2), ("freqs", 4), ("positions", 2)):
        assert call(**{name: GOOD + off}) == bz.BONSAI_ERR_ALIGN, name
    assert call(layout=2) == call(layout=-1) == bz.BONSAI_ERR_ARG
    for kw in ({"T": -1}, {"H": -1}, {"D": 0}, {"D": 60}, {"D": 2048}, {"R": 3}, {"R": -2}, {"R": 66}, {"ld_x": 120},
               {"ld_out": 120}, {"ld_x": 129}, {"ld_out": 132}):
        assert call(**kw) == bz.BONSAI_ERR_SHAPE, kw
    assert call(ld_x=256) == bz.BONSAI_ERR_SHAPE  # x is out here: in place, the rows are the same
    assert call(T=0, x=None) == bz.BONSAI_OK
    assert call(H=0, ld_x=0, ld_out=0, x=None) == bz.BONSAI_OK


CACHE_SHAPES = [{"Hkv": 0}, {"Hkv": 3}, {"Hkv": -2}, {"D": 96}, {"D": 512}, {"page_size": 8}, {"page_size": 48},
                {"page_size": 512}, {"pages": 0}, {"pages": -1}, {"pages": 1 << 31}]


def test_append_refusals(bz):
    def call(qkv=GOOD, q_out=2 * GOOD, k=GOOD, v=GOOD, ks=GOOD, vs=GOOD, freqs=GOOD, positions=GOOD, slots=GOOD, T=4, Hq=4,
             Hkv=2, D=64, R=64, ld_qkv=512, ld_q=256, pages=8, page_size=16, layout=0, kv_type=1):
        return bz.raw().bonsai_rope_append(qkv, q_out, k, v, ks, vs, freqs, positions, slots, T, Hq, Hkv, D, R, ld_qkv,
                                           ld_q, pages, page_size, 1.0, layout, kv_type, None)
    for name in ("qkv", "q_out", "k", "v", "ks", "vs", "freqs", "positions", "slots"):
        assert call(**{name: None}) == bz.BONSAI_ERR_NULL, name
    for name, off in (("qkv", 2), ("q_out", 8), ("k", 1), ("v", 8), ("ks", 2), ("vs", 1), ("freqs", 4),
                      ("positions", 2), ("slots", 4)):
        assert call(**{name: GOOD + off}) == bz.BONSAI_ERR_ALIGN, name
    assert call(layout=2) == call(kv_type=2) == call(kv_type=-1) == bz.BONSAI_ERR_ARG
    for kw in CACHE_SHAPES + [{"T": -1}, {"R": 66}, {"R": 5}, {"ld_qkv": 504}, {"ld_q": 248}, {"ld_q": 257}]:
        assert call(**kw) == bz.BONSAI_ERR_SHAPE, kw
    assert call(q_out=GOOD) == bz.BONSAI_ERR_SHAPE  # in place, but with another row stride
    assert call(T=0, qkv=None) == bz.BONSAI_OK


def test_attention_refusals(bz):
    def call(q=GOOD, k=GOOD, v=GOOD, ks=GOOD, vs=GOOD, table=GOOD, lengths=GOOD, out=GOOD, lse=GOOD, B=2, Hq=4, Hkv=2,
             D=64, ld_q=256, ld_out=256, pages=8, page_size=16, max_pages=4, window=0, kv_type=1):
        return bz.raw().bonsai_paged_attention(q, k, v, ks, vs, table, lengths, out, lse, B, Hq, Hkv, D, ld_q, ld_out,
                                               pages, page_size, max_pages, window, 1.0, kv_type, None)
    for name in ("q", "k", "v", "ks", "vs", "table", "lengths", "out"):
        assert call(**{name: None}) == bz.BONSAI_ERR_NULL, name
    for name, off in (("q", 2), ("k", 8), ("v", 1), ("ks", 2), ("vs", 1), ("table", 2), ("lengths", 1), ("out", 8),
                      ("lse", 2)):
        assert call(**{name: GOOD + off}) == bz.BONSAI_ERR_ALIGN, name
    assert call(kv_type=2) == bz.BONSAI_ERR_ARG
    for kw in CACHE_SHAPES + [{"B": -1}, {"Hq": 0}, {"ld_q": 248}, {"ld_out": 260}, {"max_pages": 0}, {"window": -1},
                              {"B": (1 << 20) + 1}]:
        assert call(**kw) == bz.BONSAI_ERR_SHAPE, kw
    assert call(B=0, q=None) == bz.BONSAI_OK


def test_binding_refuses_host_tensors_and_mixed_pools(bz):
    """The binding's own checks, which need no device: the current one is asked for first."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("the binding asks for the current device")
    cpu = torch.zeros(4, 128, dtype=torch.float16)
    gpu = cpu.cuda()
    f, pos = torch.ones(32, dtype=torch.float64).cuda(), torch.zeros(4, dtype=torch.int32).cuda()
    for args in ((cpu, gpu, f, pos), (gpu, cpu, f, pos), (gpu, gpu, f.float(), pos), (gpu, gpu, f, pos.long()),
                 (gpu, gpu, f[:8], pos), (gpu, gpu, f, pos[:2]), (gpu[:2], gpu, f, pos), (gpu.float(), gpu, f, pos)):
        with pytest.raises(ValueError):
            bz.bonsai_rope(*args, 4, 2, 64, 64)
    pool = torch.zeros(2, 1, 16, 64, dtype=torch.float16).cuda()
    table, n = torch.zeros(1, 2, dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda()
    q = torch.zeros(1, 64, dtype=torch.float16).cuda()
    for k, v in ((pool, pool[:1]), (pool.float(), pool.float()), (pool, pool.to(torch.float8_e4m3fn)),
                 (pool[0], pool[0])):
        with pytest.raises(ValueError):
            bz.bonsai_paged_attention(q, k, v, None, None, table, n, q, 1, 1)


def test_binding_row_strides(bz):
    """Rows of heads keep their place when the tensor has more or wider rows than the call takes."""
    import torch
    def ld(*shape, rows=3, width=64, given=None):
        return bz._rows(torch.zeros(*shape, dtype=torch.float16), rows, width, given, -1)[1]
    assert ld(3, 64) == ld(8, 64) == ld(3 * 64) == ld(3, 4, 16) == ld(12, 16) == 64
    assert ld(3, 96) == ld(8, 96) == ld(3, 6, 16) == 96  # wider rows, more rows
    assert ld(1, 80, rows=1) == 80 and ld(0, 64, rows=0) == 64
    assert ld(8 * 64, given=64) == 64 and ld(3 * 128, given=128) == 128
    for shape, given in (((8, 4, 16), None), ((512,), None), ((2, 64), None), ((100,), None), ((3, 64), 96)):
        with pytest.raises(ValueError):
            ld(*shape, given=given)
