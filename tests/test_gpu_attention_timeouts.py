"""The bounded waits of the paged attention, made to give up by the library's test hook: NaN
for every sequence with keys, the status bit, and nothing left behind for the calls that follow."""
import numpy as np
import pytest

from tests import layer_ref as ref
from tests.test_gpu_attention import bz, check, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("lengths,Hq,Hkv,D,page", [
    ([5], 1, 1, 64, 16),                       # one tile: the producer never waits for a stage
    ([70, 0, 300], 8, 2, 128, 16),             # a tile or two per CTA
    ([3000] * 40, 16, 8, 128, 64),             # more tiles than stages: the producer gives up too
    ([9000, 20], 16, 1, 256, 32)])             # one head over every CTA, joined in two levels
def test_forced_timeouts_nan_status_and_recovery(bz, lengths, Hq, Hkv, D, page, kv):  # noqa: F811
    rng = np.random.default_rng(sum(lengths) + kv)
    pool = ref.Pool(rng, lengths, Hkv, D, page, kv)
    d, q = pool.device(), rng.normal(0, 2, (len(lengths), Hq, D)).astype(np.float16)
    bz.bonsai_device_status(clear=True)
    first, first_lse = run(bz, q, d, Hq)
    assert bz.bonsai_device_status() == 0
    check(first, first_lse, q, pool, 0, D ** -0.5)
    for _ in range(2):
        bz.bonsai_debug_force_timeouts(True)
        try:
            got, lse = run(bz, q, d, Hq)
        finally:
            bz.bonsai_debug_force_timeouts(False)
        assert bz.bonsai_device_status(clear=True) == bz.BONSAI_DEVICE_ATTENTION_TIMEOUT
        some = np.array(lengths) > 0  # (a sequence without keys needs no copy: its zeros stand)
        assert np.isnan(got[some]).all() and (got[~some] == 0).all() and np.isnan(lse[some]).all()
        for _ in range(2):  # counters back at zero, partial results of the other call not taken
            again, again_lse = run(bz, q, d, Hq)
            assert np.array_equal(again, first) and np.array_equal(again_lse, first_lse)
        assert bz.bonsai_device_status() == 0
