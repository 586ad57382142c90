"""One decoded token through the calls that work in place on a fused projection's row."""
import numpy as np
import pytest

from tests import layer_ref as ref

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


@pytest.mark.parametrize("T", [1, 2, 3])
def test_query_and_key_columns_in_place(bz, T):
    """rope of qkv into its own query columns, and the append with q_out the same columns, give for
    any number of rows what they give into other buffers; the other columns keep their bits."""
    import torch
    rng = np.random.default_rng(T)
    Hq, Hkv, D, page = 6, 2, 64, 16
    w = Hq * D
    x = rng.normal(0, 1, (T, (Hq + 2 * Hkv) * D)).astype(np.float16)
    freqs = torch.from_numpy(ref.frequencies(D, 1e6)[0]).cuda()
    pos = torch.from_numpy(rng.integers(0, 9999, T).astype(np.int32)).cuda()
    slots = torch.arange(T, dtype=torch.int64, device="cuda") * 3
    want = torch.empty((T, w), dtype=torch.float16, device="cuda")
    bz.bonsai_rope(f16(x), want, freqs, pos, T, Hq, D, D)
    a = f16(x)
    bz.bonsai_rope(a, a[:, :w], freqs, pos, T, Hq, D, D)
    assert torch.equal(a[:, :w], want) and torch.equal(a[:, w:], f16(x)[:, w:])
    pools, b, pools2 = [], f16(x), []
    for p in (pools, pools2):
        p += [torch.zeros((2, Hkv, page, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    q = torch.empty((T, w), dtype=torch.float16, device="cuda")
    bz.bonsai_rope_append(f16(x), q, *pools, None, None, freqs, pos, slots, T, Hq, D)
    bz.bonsai_rope_append(b, b[:, :w], *pools2, None, None, freqs, pos, slots, T, Hq, D)
    assert torch.equal(q, want) and torch.equal(b[:, :w], want) and torch.equal(b[:, w:], f16(x)[:, w:])
    assert all(torch.equal(s, t) for s, t in zip(pools, pools2))
    # the attention reads its queries from those columns too
    table, n = torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.full((T,), 1, dtype=torch.int32, device="cuda")
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    bz.bonsai_paged_attention(b[:, :w], *pools2, None, None, table, n, out, T, Hq)
    bz.bonsai_paged_attention(q, *pools, None, None, table, n, out2, T, Hq)
    assert torch.equal(out, out2)
