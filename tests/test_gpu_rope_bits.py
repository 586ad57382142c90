"""What rotary calls do not rotate keeps its bits, those of a NaN (sign, payload, signalling) too:
the rest of a head, all of it where R is 0, and the value heads of an append to an FP16 cache."""
import numpy as np
import pytest

from tests import layer_ref as ref
from tests.test_gpu_rope import bz, dev, f16, positions_of  # noqa: F401

pytestmark = pytest.mark.gpu


def bits_with_nans(rng, shape):
    """Random FP16 bit patterns, a third of them NaN."""
    b = rng.integers(0, 1 << 16, shape).astype(np.uint16)
    nan = rng.integers(1, 1 << 10, shape) | 0x7c00 | (rng.integers(0, 2, shape) << 15)
    return np.where(rng.random(shape) < 1 / 3, nan, b).astype(np.uint16)


def host_bits(t):
    import torch
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T,H,D,R", [(3, 2, 64, 0), (2, 3, 128, 64), (5, 2, 64, 38), (2, 3, 72, 70), (1, 1, 24, 2), (300, 5, 128, 96)])
def test_rope_keeps_the_bits_of_the_rest(bz, T, H, D, R, layout):  # noqa: F811
    import torch
    rng = np.random.default_rng(T + D + R)
    x = bits_with_nans(rng, (T, H, D))
    freqs, pos = ref.frequencies(R, 1e4)[0], positions_of(rng, T)
    xd, out = f16(x.view(np.float16)), torch.zeros((T, H * D), dtype=torch.float16, device="cuda")
    bz.bonsai_rope(xd, out, dev(freqs) if R else None, dev(pos), T, H, D, R, layout)
    assert np.array_equal(host_bits(out).reshape(T, H, D)[..., R:], x[..., R:])
    bz.bonsai_rope(xd, xd, dev(freqs) if R else None, dev(pos), T, H, D, R, layout)
    assert np.array_equal(host_bits(xd)[..., R:], x[..., R:])
    # rotated parts: a NaN in a pair makes both of it NaN
    a, b = (np.arange(R // 2), np.arange(R // 2) + R // 2) if layout == 0 else (np.arange(0, R, 2), np.arange(1, R, 2))
    v, got = x.view(np.float16), host_bits(out).reshape(T, H, D).view(np.float16)
    either = np.isnan(v[..., a]) | np.isnan(v[..., b])
    assert np.isnan(got[..., a][either]).all() and np.isnan(got[..., b][either]).all()


@pytest.mark.parametrize("layout,R", [(0, 64), (1, 64), (0, 38), (1, 38), (1, 0)])
def test_append_keeps_the_bits_of_values(bz, layout, R):  # noqa: F811
    import torch
    rng = np.random.default_rng(R + layout)
    T, Hq, Hkv, D, page = 21, 4, 2, 64, 16
    x = bits_with_nans(rng, (T, Hq + 2 * Hkv, D))
    freqs, pos = ref.frequencies(R, 1e4)[0], positions_of(rng, T)
    k, v = (torch.zeros((2, Hkv, page, D), dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros((T, Hq * D), dtype=torch.float16, device="cuda")
    bz.bonsai_rope_append(f16(x.view(np.float16)).view(T, -1), q, k, v, None, None, dev(freqs) if R else None, dev(pos),
                          dev(np.arange(T, dtype=np.int64)), T, Hq, R, layout)
    flat = [host_bits(p).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:T] for p in (k, v)]
    assert np.array_equal(flat[1], x[:, Hq + Hkv:])
    assert np.array_equal(flat[0][..., R:], x[:, Hq: Hq + Hkv, R:])
    assert np.array_equal(host_bits(q).reshape(T, Hq, D)[..., R:], x[:, :Hq, R:])
