"""The 4-bit attention at the ends of float32's range: scales of v down to 2^-126, scores next to the largest."""

import numpy as np
import pytest

from oracle import draft4 as o4
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_kv4 import _lib, attend, case, dev, f64  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

PAGE = 16


def words_of(pool, hkv, D):
    """(s, m) of K's and V's tokens: [pages][hkv][2][page][2], bf16 bits; and the way back into the pool's bytes."""
    at = pool.reshape(pool.shape[0], hkv, -1)[:, :, PAGE * D:PAGE * (D + 8)]
    return at.copy().view(np.uint16).reshape(pool.shape[0], hkv, 2, PAGE, 2)


def put(pool, hkv, D, words):
    pool.reshape(pool.shape[0], hkv, -1)[:, :, PAGE * D:PAGE * (D + 8)] = \
        words.view(np.uint8).reshape(pool.shape[0], hkv, -1)


@pytest.mark.parametrize("D,hq,K", [(64, 1, 0), (128, 4, 0), (128, 8, 0), (64, 4, 3), (128, 12, 1)])
@pytest.mark.parametrize("power", [-126, -124, -121, -119, -117, -110, -100, 120])
def test_scales_of_v_down_to_the_smallest_normal(D, hq, K, power):
    """Minima 0, so that the scales' part is all there is; one short sequence and one cut into parts."""
    r = np.random.default_rng(D + hq + 200 - power)
    lens, ks = [13, 3000], [K, 0]
    q, pool, table, _ = case(r, 2, K, hq, 1, D, PAGE, lens, ks)
    words = words_of(pool, 1, D)
    words[:, :, 1, :, 0] = o4.bf16_bits(o4.bf16(r.uniform(1, 2, words.shape[:2] + (PAGE,)) * 2.0 ** power))
    words[:, :, 1, :, 1] = 0
    put(pool, 1, D, words)
    out, lse, ws = attend(q.cuda(), dev(pool), dev(table), dev(np.int32(lens)), dev(np.int32(ks)), PAGE, D, 1, D ** -0.5)
    assert sb.sv_read_device_flags(ws) == 0
    for b in range(2):
        codes, s, m = o4.read_tokens(pool, table[b], PAGE, lens[b] + ks[b], 1, D)
        ref, _, coded, weight, spread = o4.attention(f64(q[b, :ks[b] + 1]), codes, s, m, lens[b], D ** -0.5)
        # the weights' fp16 (2^-11, 2^-32 of the largest below 2^-21 of it), scores' float32 sums, bf16's rounding and
        # smallest step, parts whose sums are rounded to float32's (2^-150 each, at most 188 of them)
        dz = (D + 8) * 2.0 ** -23 * spread + 2.0 ** -20
        bound = 2.0 ** -11 * coded + 2 * dz[..., None] * weight + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134 + 188 * 2.0 ** -150
        got = f64(out[b, :ks[b] + 1])
        # values beyond 2^96: a sum of 3000 weights of up to 2^8 times values of 2^124 is past float32's 2^128
        there = np.isfinite(got) if power == 120 else np.ones(got.shape, bool)
        assert np.all(np.abs(got - ref)[there] <= bound[there]), np.max((np.abs(got - ref) / bound)[there])
        assert np.any(got != 0)
