"""Rotary positions and their append to a paged cache on the GPU, against the float64 forms of
tests/layer_ref.py.  Bounds: half a step of the output's type plus the FP32 error of the
rotation (layer_ref.rope, f16_bound, e4m3_bound)."""
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


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.float16)


def check(got, want, bound):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4], bound[bad][:4])


def positions_of(rng, T, span=1 << 20):
    p = rng.integers(0, span, T).astype(np.int32)
    p[:3] = np.array([0, span - 1, 1])[:T]
    return p


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T,H,D,R", [
    (1, 48, 128, 128), (3, 1, 64, 64), (7, 5, 128, 64), (2, 3, 256, 256), (5, 2, 64, 38), (33, 9, 128, 2), (4, 2, 8, 8),
    (6, 3, 128, 0), (1, 1, 1024, 1024), (2, 3, 72, 70), (300, 48, 128, 128), (17, 7, 24, 16)])
def test_rope(bz, T, H, D, R, layout):
    import torch
    rng = np.random.default_rng(T * 1000 + H * 10 + R + layout)
    x = rng.normal(0, 2, (T, H, D)).astype(np.float16)
    freqs, _ = ref.frequencies(R, 1e4)
    pos = positions_of(rng, T)
    want, slack = ref.rope(x, pos, freqs, R, layout, 1.0)
    xd, out = f16(x), torch.full((T, H * D), float("nan"), dtype=torch.float16, device="cuda")
    bz.bonsai_rope(xd, out, dev(freqs), dev(pos), T, H, D, R, layout)
    got = to_numpy_f16(out).reshape(T, H, D)
    check(got, want, ref.f16_bound(want, slack))
    assert np.array_equal(got[..., R:], x[..., R:].astype(np.float64))  # what is not rotated passes unchanged
    # in place gives the same bits
    bz.bonsai_rope(xd, xd, dev(freqs), dev(pos), T, H, D, R, layout)
    assert torch.equal(xd.view(T, -1), out)


def test_rope_strided_rows(bz):
    """The query and key heads of a fused projection's rows, in place and into a wider matrix;
    everything else keeps its bits."""
    import torch
    rng = np.random.default_rng(5)
    T, H, D, R, ld, ldo = 19, 6, 64, 32, 10 * 64, 8 * 64 + 8
    x = rng.normal(0, 1, (T, ld)).astype(np.float16)
    freqs, pos = ref.frequencies(R, 1e6)[0], positions_of(rng, T)
    want, slack = ref.rope(x[:, : H * D].reshape(T, H, D), pos, freqs, R, 0, 1.0)
    want, bound = want.reshape(T, -1), ref.f16_bound(want, slack).reshape(T, -1)
    xd, out = f16(x), torch.full((T, ldo), 7.0, dtype=torch.float16, device="cuda")
    bz.bonsai_rope(xd[:, : H * D], out[:, : H * D], dev(freqs), dev(pos), T, H, D, R)
    check(to_numpy_f16(out)[:, : H * D], want, bound)
    assert bool((out[:, H * D:] == 7.0).all())
    bz.bonsai_rope(xd, xd, dev(freqs), dev(pos), T, H, D, R, ld_x=ld, ld_out=ld)
    check(to_numpy_f16(xd)[:, : H * D], want, bound)
    assert np.array_equal(to_numpy_f16(xd)[:, H * D:], x[:, H * D:].astype(np.float64))


def test_rope_magnitude_negative_positions_and_specials(bz):
    import torch
    rng = np.random.default_rng(6)
    T, H, D, R = 8, 2, 64, 64
    x = rng.normal(0, 1, (T, H, D)).astype(np.float16)
    freqs, mag = ref.frequencies(R, 1e6, "yarn", 4.0, 4096.0)
    mag = float(np.float32(mag))
    pos = np.array([0, -1, -5000, 2 ** 31 - 1, -2 ** 31, 77, 4095, 262143], dtype=np.int32)
    want, slack = ref.rope(x, pos, freqs, R, 1, mag)
    out = torch.empty((T, H * D), dtype=torch.float16, device="cuda")
    bz.bonsai_rope(f16(x), out, dev(freqs), dev(pos), T, H, D, R, 1, magnitude=mag)
    check(to_numpy_f16(out).reshape(T, H, D), want, ref.f16_bound(want, slack))
    # a rotation taken back: the same values within two roundings and both rotations' slack
    back = torch.empty_like(out)
    bz.bonsai_rope(out, back, dev(freqs), dev((-pos.astype(np.int64)).clip(-2 ** 31, 2 ** 31 - 1).astype(np.int32)), T, H,
                   D, R, 1, magnitude=1.0 / mag)
    keep = pos != -2 ** 31
    err = np.abs(to_numpy_f16(back).reshape(T, H, D) - x.astype(np.float64))[keep]
    pair = np.abs(x.astype(np.float64)).reshape(T, H, R // 2, 2).sum(-1).repeat(2, -1)[keep]
    assert (err <= 4 * ref.H16 * pair + 4 * ref.TINY16).all()
    # NaN and infinity stay within their pair
    x2 = x.copy()
    x2[0, 0, 6], x2[1, 1, 8] = np.nan, np.inf
    bz.bonsai_rope(f16(x2), out, dev(freqs), dev(pos), T, H, D, R, 1)
    got = to_numpy_f16(out).reshape(T, H, D)
    assert np.isnan(got[0, 0, 6:8]).all() and not np.isfinite(got[1, 1, 8:10]).all()
    got[0, 0, 6:8] = got[1, 1, 8:10] = 0
    assert np.isfinite(got).all()


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,page,layout", [
    (1, 40, 8, 128, 128, 16, 0), (5, 4, 1, 64, 32, 32, 1), (33, 8, 8, 64, 64, 64, 0), (3, 6, 2, 256, 256, 16, 1),
    (130, 40, 8, 128, 64, 128, 0), (9, 0, 2, 128, 128, 256, 0), (4, 3, 3, 128, 0, 16, 1), (6, 2, 1, 64, 38, 16, 0)])
def test_append(bz, T, Hq, Hkv, D, R, page, layout, kv):
    import torch
    rng = np.random.default_rng(T + Hq + D + kv)
    H = Hq + 2 * Hkv
    x = rng.normal(0, 1, (T, H, D)).astype(np.float16)
    freqs, pos = ref.frequencies(R, 1e6)[0], positions_of(rng, T)
    pages = -(-T // page) + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T >= 3:
        slots[1] = -1  # a padded row
    scales = rng.uniform(0.005, 0.02, (2, Hkv)).astype(np.float32)
    kind = torch.float8_e4m3fn if kv else torch.float16
    fill = 0x35 if kv else 0x3555
    ibits, nbits = (torch.uint8, np.uint8) if kv else (torch.int16, np.uint16)
    pools = [torch.full((pages, Hkv, page, D), fill, dtype=ibits, device="cuda").view(kind) for _ in range(2)]
    q_out = torch.full((T, max(Hq * D, 8)), float("nan"), dtype=torch.float16, device="cuda")
    sc = [dev(scales[0]), dev(scales[1])] if kv else [None, None]
    bz.bonsai_rope_append(f16(x.reshape(T, -1)), q_out, *pools, *sc, dev(freqs), dev(pos), dev(slots), T, Hq, R, layout)
    assert bz.bonsai_device_status(clear=True) == 0
    want, slack = ref.rope(x[:, : Hq + Hkv], pos, freqs, R, layout, 1.0)
    bound = ref.f16_bound(want, slack)
    if Hq:
        check(to_numpy_f16(q_out).reshape(T, Hq, D), want[:, :Hq], bound[:, :Hq])
    touched = np.zeros((pages, page), dtype=bool)
    for t in range(T):
        if slots[t] >= 0:
            touched[slots[t] // page, slots[t] % page] = True
    for i, (exact, slk) in enumerate(((want[:, Hq:], slack[:, Hq:]),
                                      (x[:, Hq + Hkv:].astype(np.float64), np.zeros((T, Hkv, D))))):
        bits = pools[i].view(ibits).cpu().numpy().view(nbits)
        # entries of no token keep their bits
        assert (bits.transpose(0, 2, 1, 3)[~touched] == fill).all()
        for t in range(T):
            if slots[t] < 0:
                continue
            e = bits[slots[t] // page, :, slots[t] % page]
            if kv:
                s = scales[i][:, None].astype(np.float64)
                u = np.clip(exact[t] / s, -448, 448)
                check(ref.e4m3_values(e), u, ref.e4m3_bound(u, slk[t] / s))
            else:
                check(e.view(np.float16).astype(np.float64), exact[t], ref.f16_bound(exact[t], slk[t]))


def test_append_saturates_and_keeps_nan(bz):
    import torch
    T, D = 16, 64
    x = np.zeros((T, 3, D), dtype=np.float16)
    x[0, 2, :4] = [1000, -1000, np.inf, np.nan]
    x[1, 2, :4] = [448, 464, 465, 2.0 ** -10]
    pools = [torch.zeros((1, 1, 16, D), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    one = torch.ones(1, device="cuda")
    q = torch.empty((T, D), dtype=torch.float16, device="cuda")
    bz.bonsai_rope_append(f16(x.reshape(T, -1)), q, *pools, one, one, None, dev(np.zeros(T, np.int32)),
                          dev(np.arange(T, dtype=np.int64)), T, 1, 0)
    v = ref.e4m3_values(pools[1].view(torch.uint8).cpu().numpy())[0, 0]
    assert v[0, :3].tolist() == [448, -448, 448] and np.isnan(v[0, 3])
    assert v[1, :4].tolist() == [448, 448, 448, 0]  # 2^-10 is half the smallest step: to even


def test_append_out_of_range_slots(bz):
    """Slots at and past the pools' end write nothing and set the status bit; the good tokens of the
    same call are stored."""
    import torch
    T, Hq, Hkv, D, page, pages = 5, 2, 1, 64, 16, 2
    x = np.random.default_rng(3).normal(0, 1, (T, Hq + 2 * Hkv, D)).astype(np.float16)
    buf = torch.zeros((pages + 2, Hkv, page, D), dtype=torch.float16, device="cuda")
    k, v = buf[1: 1 + pages].clone(), torch.zeros((pages, Hkv, page, D), dtype=torch.float16, device="cuda")
    slots = np.array([3, pages * page, -1, 2 ** 62, 31], dtype=np.int64)
    q = torch.empty((T, Hq * D), dtype=torch.float16, device="cuda")
    bz.bonsai_device_status(clear=True)
    bz.bonsai_rope_append(f16(x.reshape(T, -1)), q, k, v, None, None, None, dev(np.zeros(T, np.int32)), dev(slots), T, Hq, 0)
    assert bz.bonsai_device_status(clear=True) == bz.BONSAI_DEVICE_CACHE_RANGE
    assert bz.bonsai_device_status() == 0
    want = np.zeros((pages * page, D))
    want[3], want[31] = x[0, 3], x[4, 3]
    assert np.array_equal(to_numpy_f16(v).reshape(-1, D), want)
    assert np.array_equal(to_numpy_f16(q), x[:, :Hq].reshape(T, -1).astype(np.float64))


def test_append_query_in_place_and_large_pool(bz):
    """The query heads rotated where they lie, and an entry beyond 2^31 elements of a pool."""
    import torch
    T, Hq, Hkv, D, page = 2, 8, 8, 256, 256
    pages = (1 << 32) // (Hkv * page * D) + 2  # 2^32 elements and a little
    pools = [torch.zeros((pages, Hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    x = np.random.default_rng(4).normal(0, 1, (T, Hq + 2 * Hkv, D)).astype(np.float16)
    one = torch.ones(Hkv, device="cuda")
    slots = np.array([pages * page - 1, (pages // 2 + 1) * page + 5], dtype=np.int64)
    freqs, pos = ref.frequencies(D, 1e6)[0], np.array([9, 70000], dtype=np.int32)
    xd = f16(x.reshape(T, -1))
    bz.bonsai_rope_append(xd, xd, *pools, one, one, dev(freqs), dev(pos), dev(slots), T, Hq, D,
                          ld_qkv=xd.shape[1], ld_q=xd.shape[1])
    want, slack = ref.rope(x[:, : Hq + Hkv], pos, freqs, D, 0, 1.0)
    got = to_numpy_f16(xd).reshape(T, -1, D)
    check(got[:, :Hq], want[:, :Hq], ref.f16_bound(want, slack)[:, :Hq])
    assert np.array_equal(got[:, Hq:], x[:, Hq:].astype(np.float64))
    for t in range(T):
        p, o = divmod(int(slots[t]), page)
        kb = ref.e4m3_values(pools[0][p, :, o].view(torch.uint8).cpu().numpy())
        check(kb, want[t, Hq:], ref.e4m3_bound(want[t, Hq:], slack[t, Hq:]))
    assert int((pools[1].view(torch.uint8) != 0).sum(dtype=torch.int64)) == int(
        sum((ref.e4m3_bound(0, 0) < np.abs(x[t, Hq + Hkv:].astype(np.float64))).sum() for t in range(T)))
