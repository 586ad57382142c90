"""Attention of one new token over a paged cache on the GPU, against the float64 form of
tests/layer_ref.py (with its derived bounds).  Every position outside a sequence's window is
NaN in the pools, the table holds invalid numbers where no page is in use."""
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


def f16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.float16)


def run(bz, q, pool_dev, Hq, window=0, scale=None, lse=True, **kw):
    import torch
    B = q.shape[0]
    out = torch.full((B, q.shape[1] * q.shape[2]), float("nan"), dtype=torch.float16, device="cuda")
    l = torch.full((B, Hq), float("nan"), device="cuda") if lse else None
    bz.bonsai_paged_attention(f16(q.reshape(B, -1)), *pool_dev, out, B, Hq, window=window, scale=scale, lse=l, **kw)
    torch.cuda.synchronize()
    return to_numpy_f16(out).reshape(q.shape), None if l is None else l.cpu().numpy().astype(np.float64)


def check(got, lse, q, pool, window, scale):
    want, want_lse, tol, lse_tol = ref.attention(q.astype(np.float64), pool.k, pool.v, pool.lengths, window, scale)
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], tol[bad][:3])
    if lse is not None:
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(lse), empty)
        assert (np.abs(lse[~empty] - want_lse[~empty]) <= lse_tol[~empty]).all()


CASES = [  # lengths, Hq, Hkv, D, page, window
    ([1], 1, 1, 128, 16, 0),
    ([0], 5, 1, 128, 16, 0),
    ([333], 40, 8, 128, 16, 0),
    ([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0], 8, 2, 128, 16, 0),
    ([31, 32, 33, 255, 256, 257, 1], 6, 6, 64, 32, 0),
    ([700, 3, 1500], 10, 2, 256, 64, 0),
    ([1000, 1], 16, 1, 128, 128, 0),
    ([513, 77], 24, 1, 64, 256, 0),
    ([300, 9, 0], 40, 1, 128, 16, 0),
    ([200], 7, 1, 256, 16, 0),
    ([2000, 500, 3, 64], 8, 2, 128, 16, 100),
    ([2000, 500, 3, 64], 8, 2, 128, 64, 1),
    ([1024, 1000, 64, 65], 4, 4, 64, 32, 64),
    ([90, 5], 12, 2, 256, 256, 33),
    ([20000], 40, 8, 128, 64, 0),
    ([9000, 1, 8000], 2, 2, 64, 16, 5000),
    (list(range(0, 150)), 4, 2, 64, 16, 0),
]


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{len(c[0])}n{max(c[0])}h{c[1]}-{c[2]}d{c[3]}p{c[4]}w{c[5]}")
def test_attention(bz, case, kv):
    lengths, Hq, Hkv, D, page, window = case
    rng = np.random.default_rng(sum(lengths) + Hq + D + kv)
    pool = ref.Pool(rng, lengths, Hkv, D, page, kv, window=window)
    q = rng.normal(0, 2, (len(lengths), Hq, D)).astype(np.float16)
    got, lse = run(bz, q, pool.device(), Hq, window)
    check(got, lse, q, pool, window, D ** -0.5)
    assert bz.bonsai_device_status(clear=True) == 0


@pytest.mark.parametrize("seed", range(12))
def test_attention_random_shapes(bz, seed):
    rng = np.random.default_rng(100 + seed)
    D, page, kv = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 64, 128, 256])), int(rng.integers(0, 2))
    Hkv, G = int(rng.choice([1, 2, 3, 8])), int(rng.choice([1, 2, 3, 5, 8, 9, 16, 17]))
    B = int(rng.integers(1, 20))
    lengths = [int(v) for v in np.exp(rng.uniform(0, np.log(1500), B)).astype(int) - rng.integers(0, 2, B)]
    window = int(rng.choice([0, 0, 1, 50, 400]))
    scale = float(rng.choice([D ** -0.5, 0.02, 0.3 * D ** -0.5]))
    pool = ref.Pool(rng, lengths, Hkv, D, page, kv, window=window)
    q = rng.normal(0, 2, (B, Hkv * G, D)).astype(np.float16)
    got, lse = run(bz, q, pool.device(), Hkv * G, window, scale)
    check(got, lse, q, pool, window, float(np.float32(scale)))


def test_attention_strides_and_rows_behind(bz):
    """q read from a fused projection's rows, out written into a wider matrix; nothing else of it
    changes, nor do rows behind the last sequence; lse may be absent."""
    import torch
    rng = np.random.default_rng(8)
    lengths, Hq, Hkv, D, page = [70, 0, 200], 4, 2, 64, 16
    pool = ref.Pool(rng, lengths, Hkv, D, page, 0)
    rows = rng.normal(0, 2, (3, (Hq + 2 * Hkv) * D)).astype(np.float16)
    q = rows[:, : Hq * D].reshape(3, Hq, D)
    out = torch.full((6, Hq * D + 24), 3.0, dtype=torch.float16, device="cuda")
    bz.bonsai_paged_attention(f16(rows)[:, : Hq * D], *pool.device(), out[:, : Hq * D], 3, Hq)
    got = to_numpy_f16(out)
    check(got[:3, : Hq * D].reshape(3, Hq, D), None, q, pool, 0, D ** -0.5)
    assert (got[3:] == 3).all() and (got[:, Hq * D:] == 3).all()


@pytest.mark.parametrize("kv", [0, 1])
def test_attention_bad_pages_and_lengths(bz, kv):
    """A page number outside the cache, a negative length and one past the table's row make that
    sequence NaN and set the status bit; the others are right."""
    import torch
    rng = np.random.default_rng(9)
    lengths, Hq, Hkv, D, page = [100, 90, 80, 70, 40, 60], 6, 2, 128, 16
    pool = ref.Pool(rng, lengths, Hkv, D, page, kv)
    q = rng.normal(0, 2, (6, Hq, D)).astype(np.float16)
    d = list(pool.device())
    d[4][1, 3], d[4][2, 0] = pool.pages, -1
    d[5][3], d[5][4] = -5, pool.width * page + 1
    bz.bonsai_device_status(clear=True)
    got, lse = run(bz, q, d, Hq)
    assert bz.bonsai_device_status(clear=True) == bz.BONSAI_DEVICE_CACHE_RANGE
    assert np.isnan(got[1:5]).all() and np.isnan(lse[1:5]).all()
    good = [0, 5]
    want, _, tol, _ = ref.attention(q[good].astype(np.float64), [pool.k[i] for i in good], [pool.v[i] for i in good],
                                    [100, 60], 0, D ** -0.5)
    assert (np.abs(got[good] - want) <= tol).all()
    # the next call is clean
    got, lse = run(bz, q, pool.device(), Hq)
    check(got, lse, q, pool, 0, D ** -0.5)
    assert bz.bonsai_device_status(clear=True) == 0


def test_attention_extreme_scores(bz):
    """Scores far apart and large: the running maximum moves, small terms vanish, nothing overflows."""
    rng = np.random.default_rng(10)
    lengths, Hq, Hkv, D, page = [600, 257], 4, 1, 64, 16
    pool = ref.Pool(rng, lengths, Hkv, D, page, 0)
    q = (rng.normal(0, 40, (2, Hq, D))).astype(np.float16)
    got, lse = run(bz, q, pool.device(), Hq, scale=1.0)
    # scores of up to ~1500: their FP32 error is 1e-3 and more, which layer_ref.attention carries
    check(got, lse, q, pool, 0, 1.0)


def test_attention_repeats_bitwise_and_on_other_streams(bz):
    import torch
    rng = np.random.default_rng(11)
    lengths, Hq, Hkv, D, page = [5000, 17, 900, 0, 333], 40, 8, 128, 16
    pool = ref.Pool(rng, lengths, Hkv, D, page, 0)
    d, q = pool.device(), rng.normal(0, 2, (5, Hq, D)).astype(np.float16)
    first, _ = run(bz, q, d, Hq)
    for _ in range(5):
        assert np.array_equal(run(bz, q, d, Hq)[0], first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert np.array_equal(run(bz, q, d, Hq)[0], first)


def test_attention_in_a_graph_follows_lengths(bz):
    """A captured call replays with the lengths, table and queries of the moment."""
    import torch
    rng = np.random.default_rng(12)
    Hq, Hkv, D, page = 8, 2, 128, 16
    pool = ref.Pool(rng, [1200, 800, 640], Hkv, D, page, 0)
    d = pool.device()
    q = rng.normal(0, 2, (3, Hq, D)).astype(np.float16)
    qd, out = f16(q.reshape(3, -1)), torch.zeros((3, Hq * D), dtype=torch.float16, device="cuda")
    bz.bonsai_reserve(1, 128, 128)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        bz.bonsai_paged_attention(qd, *d, out, 3, Hq)
    for lengths in ([1200, 800, 640], [1, 0, 64], [700, 799, 33]):
        d[5].copy_(torch.tensor(lengths, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        pool.lengths = lengths
        check(to_numpy_f16(out).reshape(3, Hq, D), None, q, pool, 0, D ** -0.5)
    del g


def test_attention_entries_past_32_bits(bz):
    """Pages whose first element lies beyond 2^32 elements of the pool."""
    import torch
    rng = np.random.default_rng(13)
    Hq, Hkv, D, page, n = 16, 8, 256, 256, 300
    pages = (1 << 32) // (Hkv * page * D) + 3
    small = ref.Pool(rng, [n], Hkv, D, page, 1, spare=0)
    d = list(small.device())
    big = [torch.zeros((pages, Hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    where = [pages - 1, pages - 2]
    for i in range(2):
        for j, p in enumerate(where):
            big[i].view(torch.uint8)[p] = d[i].view(torch.uint8)[int(small.table[0, j])]
    d[4][0, :2] = torch.tensor(where, dtype=torch.int32)
    q = rng.normal(0, 2, (1, Hq, D)).astype(np.float16)
    got, lse = run(bz, q, [*big, *d[2:]], Hq)
    check(got, lse, q, small, 0, D ** -0.5)


def test_attention_large_batch(bz):
    """More sequences than a CTA has threads, most of them short."""
    rng = np.random.default_rng(14)
    lengths = [int(v) for v in rng.integers(0, 40, 1500)]
    Hq, Hkv, D, page = 4, 2, 64, 16
    pool = ref.Pool(rng, lengths, Hkv, D, page, 0)
    q = rng.normal(0, 2, (len(lengths), Hq, D)).astype(np.float16)
    got, lse = run(bz, q, pool.device(), Hq)
    check(got, lse, q, pool, 0, D ** -0.5)


def test_attention_scores_of_minus_infinity(bz):
    """Keys of -infinity among others have no weight; where there is nothing else the result is the
    formula's NaN, with an lse of -infinity; the other heads and sequences are untouched."""
    rng = np.random.default_rng(15)
    lengths, Hq, Hkv, D, page = [40, 40, 200], 4, 2, 64, 16
    pool = ref.Pool(rng, lengths, Hkv, D, page, 0)
    q = np.abs(rng.normal(0, 2, (3, Hq, D))).astype(np.float16) + np.float16(0.1)
    for b, keys in ((0, range(40)), (1, range(0, 40, 3)), (2, range(200))):
        for j in keys:  # head 0's keys
            pool.kbits[pool.table[b, j // page], 0, j % page] = 0xfc00
            pool.k[b][j, 0] = -np.inf
    got, lse = run(bz, q, pool.device(), Hq)
    for b in (0, 2):
        assert np.isnan(got[b, :2]).all() and np.isneginf(lse[b, :2]).all()
        assert np.isfinite(got[b, 2:]).all() and np.isfinite(lse[b, 2:]).all()
    keep = np.array([j for j in range(40) if j % 3])
    want, want_lse, tol, lse_tol = ref.attention(q[1:2].astype(np.float64), [pool.k[1][keep]], [pool.v[1][keep]], [len(keep)], 0,
                                                 D ** -0.5)
    assert (np.abs(got[1:2, :2] - want[:, :2]) <= tol[:, :2]).all()
    assert (np.abs(lse[1:2, :2] - want_lse[:, :2]) <= lse_tol[:, :2]).all()


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("heads", [1, 16])
def test_attention_of_many_small_probabilities(bz, kv, heads):
    """One key far above 32767 equal ones, whose probabilities of 2^-24.6 make up the result: each is
    rounded by 2^-11 of itself (all alike, so the roundings do not cancel) and the output once more."""
    import torch
    D, page, n, z = 64, 64, 32768, 17.0625
    kind = torch.float8_e4m3fn if kv else torch.float16
    k = torch.zeros((n // page, 1, page, D), device="cuda")
    k[0, 0, 0, 0] = 1
    v = torch.ones_like(k)
    v[0, 0, 0] = 0
    one = torch.ones(1, device="cuda") if kv else None
    q = np.zeros((1, heads, D), np.float16)
    q[:, :, 0] = z
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]
    got, lse = run(bz, q, [k.to(kind), v.to(kind), one, one, table, torch.tensor([n], dtype=torch.int32, device="cuda")],
                   heads, scale=1.0)
    tail = (n - 1) * np.exp(-z)
    want = tail / (1 + tail)
    assert (np.abs(got - want) <= want * (2 * 2.0 ** -11 + 2.0 ** -19)).all(), (got.min(), got.max(), want)
    assert (np.abs(lse - (z + np.log1p(tail))) <= 2.0 ** -19 * z).all()


def test_attention_of_fewer_sequences_than_rows(bz):
    """Matrices with more rows than the batch (padded buffers): the first rows are the batch's."""
    import torch
    rng = np.random.default_rng(16)
    lengths, Hq, Hkv, D, page = [70, 5], 4, 2, 64, 16
    pool = ref.Pool(rng, lengths, Hkv, D, page, 0)
    q = rng.normal(0, 2, (8, Hq, D)).astype(np.float16)
    out = torch.full((8, Hq * D), 3.0, dtype=torch.float16, device="cuda")
    bz.bonsai_paged_attention(f16(q.reshape(8, -1)), *pool.device(), out, 2, Hq)
    got = to_numpy_f16(out).reshape(8, Hq, D)
    check(got[:2], None, q[:2], pool, 0, D ** -0.5)
    assert (got[2:] == 3).all()
