"""Drafts written over and over into a page that holds committed tokens: what those lose beside an outlier, and no more."""
import numpy as np
import pytest

import step_ref as R
import workloads as W
from gpu_util import bf16_tensor, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held", [1, 5, 15])
@pytest.mark.parametrize("outlier", [1.0, 2.0 ** 5, 2.0 ** 9, 2.0 ** 14, 2.0 ** 30])
def test_committed_tokens_beside_an_outlier(lib, held, outlier):
    """A committed value is off by half a smallest step, 2^-10, of the page's largest scale so far at most, and by nothing
    where it is 2^-6 of that scale or more."""
    rng = np.random.default_rng(held)
    Hkv, n = 3, 4
    d = lib.attn_desc(1, n, Hkv, Hkv, 128, 3, 4)
    k, v = (dev(np.full((4, Hkv, 16, 128), 127, np.uint8)) for _ in range(2))
    s, t = dev(np.ones((4, Hkv, 2), np.float32)), dev(np.array([[2, 0, 3]], np.int32))
    value = lambda x, c: R.E4M3[host(x)[2, :, :held]] * host(s)[2, :, c, None, None].astype(np.float64)

    def write(new, at):
        lib.bdlm_write_kv8(d, len(new), None, 0, bf16_tensor(new), bf16_tensor(new), k, v, s, t, dev(np.array([at], np.int32)))

    write(W._normal_bf16(rng, (held, Hkv, 128), 1.0), 0)
    before = [value(x, c) for c, x in enumerate((k, v))]
    top = host(s)[2].astype(np.float64)
    for size in (1.0, outlier, 0.5, 1.0):
        draft = rng.normal(size=(n, Hkv, 128)).astype(np.float32)
        draft[1, :, 7] = 3 * size
        write(W.f32_to_bf16_bits(draft), held)
        top = np.maximum(top, host(s)[2])
    for c, x in enumerate((k, v)):
        was, now, most = before[c], value(x, c), top[:, c, None, None]
        assert np.all(np.abs(now - was) <= 2.0 ** -10 * most)
        kept = np.abs(was) >= 2.0 ** -6 * most
        assert np.array_equal(now[kept], was[kept])
        if held + 1 < 16:                                  # (the draft with the outlier is in the page)
            assert np.all(top[:, c] >= 3 * outlier / 448)
        # (the scale itself is the last draft's again)
        assert np.all(host(s)[2, :, c] <= 2.0 ** -5)
