"""Calls of the decode layer's operators that the interface allows at its ends: the largest numbers
of sequences and heads, pages that sequences share, buffers wider than what is used, and calls that
may overlap on the GPU doing so."""
import numpy as np
import pytest

from tests import layer_ref as ref
from tests.gpu_util import to_numpy_f16
from tests.test_gpu_attention import bz, check, f16, run  # noqa: F401

pytestmark = pytest.mark.gpu


def plain_attention(q, k, v, table, lengths, Hq, page):
    """Float64 on the device, one key/value head: q (B, Hq, D), pools (pages, 1, page, D)."""
    import torch
    B, width = table.shape
    at = table.long().clamp(min=0)
    kk, vv = (p[:, 0][at].reshape(B, width * page, -1).double() for p in (k, v))
    z = torch.einsum("bhd,bnd->bhn", q.double(), kk) * q.shape[-1] ** -0.5
    live = torch.arange(width * page, device=q.device)[None] < lengths[:, None]
    z = z.masked_fill(~live[:, None], -float("inf"))
    p = torch.softmax(z, -1).nan_to_num(0.0)  # (a sequence without keys: zeros)
    return torch.einsum("bhn,bnd->bhd", p, vv), torch.einsum("bhn,bnd->bhd", p, vv.abs())


@pytest.mark.parametrize("B", [(1 << 20), 70001])
def test_most_sequences(bz, B):  # noqa: F811
    """The largest batch, all of it on a few shared pages; every output compared."""
    import torch
    g = torch.Generator("cuda").manual_seed(B)
    Hq, D, page, pages = 1, 64, 16, 7
    k, v = (torch.randn((pages, 1, page, D), generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    table = torch.randint(0, pages, (B, 1), generator=g, device="cuda", dtype=torch.int32)
    lengths = torch.randint(0, page + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn((B, Hq * D), generator=g, device="cuda").half()
    out = torch.full_like(q, float("nan"))
    bz.bonsai_paged_attention(q, k, v, None, None, table, lengths, out, B, Hq)
    for b0 in range(0, B, 1 << 17):
        b = slice(b0, min(B, b0 + (1 << 17)))
        want, size = plain_attention(q[b].view(-1, Hq, D), k, v, table[b], lengths[b], Hq, page)
        # scores of normal values: 2^-16 covers their FP32 error; P's and the output's roundings 2^-11 each
        bound = (2 * ref.H16 + 2.0 ** -16) * size + ref.TINY16
        assert bool(((out[b].view(-1, Hq, D).double() - want).abs() <= bound).all())
    assert bz.bonsai_device_status(clear=True) == 0


@pytest.mark.parametrize("kv", [0, 1])
def test_many_heads_of_one_key_head(bz, kv):  # noqa: F811
    rng = np.random.default_rng(3)
    lengths, Hq, Hkv, D, page = [130, 0, 7], 1000, 1, 64, 16
    pool = ref.Pool(rng, lengths, Hkv, D, page, kv)
    q = rng.normal(0, 2, (3, Hq, D)).astype(np.float16)
    got, lse = run(bz, q, pool.device(), Hq)
    check(got, lse, q, pool, 0, D ** -0.5)


def test_shared_pages_and_a_wide_table(bz):  # noqa: F811
    """Sequences with a common prefix, a page used twice by one of them, a table far wider than any
    length, a batch padded with sequences of length zero."""
    import torch
    rng = np.random.default_rng(4)
    Hq, Hkv, D, page, B = 8, 2, 128, 16, 6
    pool = ref.Pool(rng, [160, 20], Hkv, D, page, 0)
    d = list(pool.device())
    own = pool.table[0, :10]
    rows = [own, own[[0, 1, 2, 3]], own[[0, 1, 5, 5, 1]], own[[9]]]
    lengths = [160, 60, 80, 16, 0, 0]
    table = np.full((B, 1 << 16), -3, np.int32)
    for b, r in enumerate(rows):
        table[b, : len(r)] = r
    d[4], d[5] = torch.from_numpy(table).cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q = rng.normal(0, 2, (B, Hq, D)).astype(np.float16)
    got, lse = run(bz, q, d, Hq)
    keys = [np.concatenate([a[0][16 * list(own).index(p): 16 * list(own).index(p) + 16] for p in r])
            for a in (pool.k, pool.v) for r in rows]
    empty = np.zeros((0, Hkv, D))
    want, want_lse, tol, lse_tol = ref.attention(q.astype(np.float64), keys[:4] + [empty, empty], keys[4:] + [empty, empty],
                                                 lengths, 0, D ** -0.5)
    assert (np.abs(got - want) <= tol).all()
    assert np.isneginf(lse[4:]).all() and (np.abs(lse[:4] - want_lse[:4]) <= lse_tol[:4]).all()
    assert bz.bonsai_device_status(clear=True) == 0


@pytest.mark.parametrize("T,H,D,R,layout", [(2, 65536, 8, 8, 0), (3, 65536, 8, 6, 1), (200001, 1, 16, 16, 0), (65537, 3, 8, 2, 1)])
def test_most_heads_and_tokens(bz, T, H, D, R, layout):  # noqa: F811
    import torch
    rng = np.random.default_rng(T)
    x = rng.normal(0, 1, (T, H, D)).astype(np.float16)
    freqs, pos = ref.frequencies(R, 1e4)[0], rng.integers(0, 1 << 20, T).astype(np.int32)
    want, slack = ref.rope(x, pos, freqs, R, layout, 1.0)
    out = torch.empty((T, H * D), dtype=torch.float16, device="cuda")
    bz.bonsai_rope(f16(x).view(T, -1), out, torch.from_numpy(freqs).cuda(), torch.from_numpy(pos).cuda(), T, H, D, R, layout)
    got = to_numpy_f16(out).reshape(T, H, D)
    assert (np.abs(got - want) <= ref.f16_bound(want, slack)).all()


def test_calls_that_may_overlap(bz):  # noqa: F811
    """Rotations and appends use no workspace: on two streams of their own beside an attention and a
    product on a third, every result is what it is alone."""
    import torch
    rng = np.random.default_rng(6)
    T, Hq, Hkv, D, page = 300, 8, 2, 128, 16
    freqs = torch.from_numpy(ref.frequencies(D, 1e6)[0]).cuda()
    pos = torch.from_numpy(rng.integers(0, 9999, T).astype(np.int32)).cuda()
    qkv = f16(rng.normal(0, 1, (T, (Hq + 2 * Hkv) * D)).astype(np.float16))
    pools = [torch.zeros((T // page + 2, Hkv, page, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    slots = torch.from_numpy(rng.permutation(T).astype(np.int64)).cuda()
    pool = ref.Pool(rng, [4000, 900, 31], Hkv, D, page, 0)
    d, q = pool.device(), f16(rng.normal(0, 2, (3, Hq * D)).astype(np.float16))
    q_rot, out, att = torch.empty((T, Hq * D), dtype=torch.float16, device="cuda"), torch.empty_like(qkv), torch.empty_like(q)

    def append(stream=None):
        bz.bonsai_rope_append(qkv, q_rot, *pools, None, None, freqs, pos, slots, T, Hq, D, stream=stream)

    def rope(stream=None):
        bz.bonsai_rope(qkv, out, freqs, pos, T, Hq + 2 * Hkv, D, D, 1, stream=stream)

    def attend(stream=None):
        bz.bonsai_paged_attention(q, *d, att, 3, Hq, stream=stream)

    results = [q_rot, *pools, out, att]
    for f in (append, rope, attend):
        f()
    torch.cuda.synchronize()
    want = [t.clone() for t in results]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for t in results:
            t.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for f, s in zip((append, rope, attend), streams):
                f(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results, want))
    assert bz.bonsai_device_status(clear=True) == 0
