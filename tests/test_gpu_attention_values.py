"""Attention of one new token over a paged cache where the values are hard: scores of up to 10^9
(of finite FP16 inputs) of either sign, alone and together in one call, with winners in several
warps and CTAs, and probabilities held to the bound that the interface states."""
import math

import numpy as np
import pytest

from tests import layer_ref as ref
from tests.gpu_util import to_numpy_f16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bz():
    import torch
    from ternary_weight_02_b200 import bonsai
    assert bonsai.bonsai_check_device() == bonsai.BONSAI_OK
    torch.cuda.init()
    return bonsai


def cache(keys, values, page, kv):
    """Pools (one key/value head) and a table of one sequence, keys and values of shape n x D."""
    import torch
    n, D = keys.shape
    pages = -(-n // page)
    kind = torch.float8_e4m3fn if kv else torch.float16
    pools = []
    for a in (keys, values):
        full = np.full((pages * page, D), np.nan, np.float32)
        full[:n] = a
        pools.append(torch.from_numpy(full.reshape(pages, 1, page, D)).cuda().to(kind))
    one = torch.ones(1, device="cuda") if kv else None
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    return [*pools, one, one, table, torch.tensor([n], dtype=torch.int32, device="cuda")]


def attend(bz, q, dev, scale):
    import torch
    _, Hq, D = q.shape
    out = torch.full((1, Hq * D), float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.full((1, Hq), float("nan"), device="cuda")
    qd = torch.from_numpy(np.ascontiguousarray(q.reshape(1, -1)).view(np.int16)).cuda().view(torch.float16)
    bz.bonsai_paged_attention(qd, *dev, out, 1, Hq, scale=scale, lse=lse)
    torch.cuda.synchronize()
    return to_numpy_f16(out).reshape(Hq, D), lse.cpu().numpy().astype(np.float64)[0]


# times the scale of 10^4: scores of +-1e7, 2.3e7, 4e7, 5e7, 6.5e7, 1e8, 2e8, 6e8
QUERIES = [1000, -1000, 2300, 4000, 5000, -5000, 6500, 10000, 20000, -20000, 60000, -60000, 100, 1, -2300, -4000]


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("heads", [1, 16])
@pytest.mark.parametrize("n", [40, 20000])
@pytest.mark.parametrize("winners", [1, 3, 8])
def test_large_scores(bz, n, heads, kv, winners):
    """Keys of 1 and 1/2 in one dimension: the winners' scores are all the same number, the other
    keys' half as large (or twice, for a negative query), 5000 below at least, where e^x is 0 in
    any arithmetic.  The result is the winners' mean value: the products with the values and the
    sum of up to 8 of them in FP32 (2^-20 with room), one rounding to FP16.  lse is the winners'
    score, of a product with scale log2 e and back (four roundings of 2^-24, two constants of half
    that) plus ln(winners)."""
    rng = np.random.default_rng(n + heads + winners)
    D, page = 128, 64
    queries = np.array(QUERIES if heads == 16 else [5000], np.float64)
    spots = np.unique(np.linspace(1, n - 2, winners).astype(int))  # in several tiles and CTAs
    assert len(spots) == winners
    values = np.where(rng.random((n, D)) < 0.5, -1.0, 1.0) * 2.0 ** rng.integers(-3, 3, (n, D))  # exact in both types
    for sign in (1, -1):
        q = np.zeros((1, heads, D), np.float16)
        q[0, :, 5] = np.abs(queries) * sign
        keys = np.zeros((n, D))
        keys[:, 5] = 0.5 if sign > 0 else 1.0
        keys[spots, 5] = 1.0 if sign > 0 else 0.5
        got, lse = attend(bz, q, cache(keys, values, page, kv), 1e4)
        z = np.abs(queries) * (1e4 if sign > 0 else -5e3)
        want = values[spots].mean(0)
        tol = ref.H16 * np.abs(want) + ref.TINY16 + 2.0 ** -20 * np.abs(values[spots]).mean(0)
        assert (np.abs(got - want) <= tol).all(), (sign, queries[~(np.abs(got - want) <= tol).all(1)], got[:, :4], want[:4])
        want_lse = z + math.log(winners)
        assert (np.abs(lse - want_lse) <= 5 * 2.0 ** -24 * np.abs(want_lse) + 2.0 ** -20).all(), (lse, want_lse)


@pytest.mark.parametrize("kv", [0, 1])
def test_large_scores_of_both_signs_in_one_call(bz, kv):
    """Sixteen heads whose scores lie 10^9 apart from one another."""
    rng = np.random.default_rng(5)
    D, page, n = 64, 16, 3000
    queries = np.array(QUERIES, np.float64)
    q = np.zeros((1, 16, D), np.float16)
    q[0, :, 9] = queries
    keys = np.zeros((n, D))
    keys[:, 9] = 0.5
    keys[2900, 9], keys[31, 9] = 1.0, 0.25  # the largest for a positive query, for a negative one
    values = rng.choice([-2.0, -1.0, 0.0, 0.5, 1.0, 4.0], (n, D))
    got, lse = attend(bz, q, cache(keys, values, page, kv), 1e4)
    for h, c in enumerate(queries):
        best, z = (2900, c * 1e4) if c > 0 else (31, c * 2500)
        assert np.array_equal(got[h], values[best]), (c, got[h][:4], values[best][:4])
        assert abs(lse[h] - z) <= 5 * 2.0 ** -24 * abs(z)


@pytest.mark.parametrize("D,size,scale", [(128, 2048.0, None), (256, 512.0, 1.0), (256, 16.0, 4.0)])
def test_large_scores_of_whole_heads(bz, D, size, scale):
    """Queries and keys that are large in every dimension, at the default scale and at others."""
    rng = np.random.default_rng(D)
    n, page, heads = 700, 32, 16
    signs = np.where(rng.random(D) < 0.5, -1.0, 1.0)
    sizes = size * (1 - np.arange(heads) / 32)  # of the heads' queries, exact in FP16
    q = (sizes[:, None] * signs).astype(np.float16)[None]
    keys = np.broadcast_to(size * signs * 0.5, (n, D)).copy()
    keys[333] = size * signs
    values = rng.choice([-2.0, 0.0, 0.25, 3.0], (n, D))
    got, lse = attend(bz, q, cache(keys, values, page, 0), scale)
    s = D ** -0.5 if scale is None else scale
    assert np.array_equal(got, np.broadcast_to(values[333], got.shape))
    z = D * sizes * size * s
    assert (np.abs(lse - z) <= (D + 4) * 2.0 ** -24 * z).all()


def bound(q, k, v, scale):
    """Output and its bound for one head, probabilities held as the interface states: 2^-11 of each,
    below 2^-28 of the largest 2^-39 of that (layer_ref.attention's form otherwise: scores off by
    (D + 4) 2^-24 sum |q k| scale, 2^-20 for the exponential, rescalings and joins)."""
    z = k @ q * scale
    p = np.exp(z - z.max())
    l = p.sum()
    out = p @ v / l
    r = 2 * (len(q) + 4) * 2.0 ** -24 * (np.abs(k) @ np.abs(q)) * abs(scale) + 2.0 ** -20
    # the maximum's own score is off too, which moves every probability alike (numerator and sum)
    num = (p * (ref.H16 + r) + 2.0 ** -39) @ np.abs(v)
    return out, num / l + (p * r).sum() / l * np.abs(out) + ref.H16 * np.abs(out) + ref.TINY16


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("lengths,Hq,Hkv,D,page", [([4000, 33], 8, 2, 64, 16), ([9000], 16, 1, 128, 64), ([700, 1500], 4, 4, 256, 32)])
def test_probabilities_keep_their_relative_precision(bz, lengths, Hq, Hkv, D, page, kv):
    """Scores spread over +-30: most probabilities lie far below FP16's normal range of the largest."""
    import torch
    rng = np.random.default_rng(sum(lengths) + kv)
    pool = ref.Pool(rng, lengths, Hkv, D, page, kv)
    B = len(lengths)
    q = rng.normal(0, 1, (B, Hq, D)).astype(np.float16)
    spread = np.sqrt(np.mean([np.mean(k ** 2) for k in pool.k]) * D)
    scale = float(np.float32(10.0 / spread))
    out = torch.full((B, Hq * D), float("nan"), dtype=torch.float16, device="cuda")
    qd = torch.from_numpy(np.ascontiguousarray(q.reshape(B, -1)).view(np.int16)).cuda().view(torch.float16)
    bz.bonsai_paged_attention(qd, *pool.device(), out, B, Hq, scale=scale)
    got = to_numpy_f16(out).reshape(B, Hq, D)
    for b in range(B):
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            want, tol = bound(q[b, h].astype(np.float64), pool.k[b][:, hk], pool.v[b][:, hk], scale)
            assert (np.abs(got[b, h] - want) <= tol).all(), (b, h, float((np.abs(got[b, h] - want) / tol).max()))
