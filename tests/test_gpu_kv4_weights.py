"""The 4-bit attention's roundings to fp16, against the bounds that the header gives: weights far below a row's
largest, and values of q far below a row's largest."""

import numpy as np
import pytest

from oracle import draft4 as o4
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_kv4 import _lib, attend, bf, case, dev, f64  # noqa: F401
from tests.test_gpu_kv4_range import PAGE, put, words_of

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("D,hq", [(64, 1), (128, 8), (128, 12)])
@pytest.mark.parametrize("far", [8, 16, 20, 22, 24, 26, 28, 31])
@pytest.mark.parametrize("first", [True, False])
def test_weights_far_below_the_largest(D, hq, far, first):
    """One token of weight about 1 whose values are 0, among 2000 of about 2^-far each: 11 bits down to 2^-21 of the
    largest, then off by at most 2^-32 of it."""
    n = 2000
    r = np.random.default_rng(far)
    q, pool, table, _ = case(r, 1, 0, hq, 1, D, PAGE, [n], [0])
    q.zero_()
    q[..., 0] = 1.0
    words = words_of(pool, 1, D)
    words[:, :, :, :, 1] = 0
    words[:, :, 0, :, 0], words[:, :, 1, :, 0] = 0, o4.bf16_bits(1.0)     # keys are their minima; v = code
    words[:, :, 0, :, 1] = o4.bf16_bits(o4.bf16(r.uniform(-0.5, 0, words.shape[:2] + (PAGE,))))
    at = 0 if first else n - 1
    page, slot = table[0, at // PAGE], at % PAGE
    words[page, 0, 0, slot, 1] = o4.bf16_bits(o4.bf16(far * np.log(2)))
    put(pool, 1, D, words)
    pool.reshape(pool.shape[0], -1)[page, PAGE * D // 2 + slot * D // 2:PAGE * D // 2 + (slot + 1) * D // 2] = 0
    out, lse, ws = attend(q.cuda(), dev(pool), dev(table), dev(np.int32([n])), None, PAGE, D, 1, 1.0)
    assert sb.sv_read_device_flags(ws) == 0
    codes, s, m = o4.read_tokens(pool, table[0], PAGE, n, 1, D)
    z, v = m[0, :, 0], s[1, :, 0, None] * codes[1, :, 0]
    p = np.exp(z - z.max())
    ref = p @ v / p.sum()
    half = np.where(p >= 2.0 ** -21, 2.0 ** -11 * p, 2.0 ** -32)
    # float32 scores of up to 22 and their exponentials: 2^-20 relative; sums of 2000 weights: 2^-13 at the most; bf16
    # has a step of 2^-7 of the power of two below the value (7 bits behind the leading one), half of it is 2^-8
    bound = half @ v / p.sum() + (2.0 ** -20 + 2.0 ** -13 + 2.0 ** -8) * np.abs(ref)
    off = np.abs(f64(out)[0, 0] - ref)
    assert np.all(off <= bound), np.max(off / bound)
    assert np.all(np.abs(f64(lse)[0, 0] - (z.max() + np.log(p.sum()))) <= 2.0 ** -20 * 32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [20, 25, 27, 28, 30, 33, 36])
@pytest.mark.parametrize("largest", [1.0, 1.9921875, 2.0 ** -120, 2.0 ** 60])
def test_values_of_q_far_below_the_largest(D, far, largest):
    """One large value of q that meets codes of 0, and small ones at every other place: kept down to 2^-27 of the
    largest, then off by at most 2^-35 of it each (of any size where the largest is below 2^-106).  One token, so the
    scores are the logarithms that come back."""
    r = np.random.default_rng(far)
    B = 8
    q, pool, table, _ = case(r, B, 0, 2, 1, D, PAGE, [1] * B, [0] * B)
    x = (r.uniform(1, 2, (B, 2, D)) * largest * 2.0 ** -far).astype(np.float64)
    big = np.arange(B) * 7 % D
    for b in range(B):
        x[b, :, big[b]] = largest
    q = bf(x).reshape(B, 1, 2, D)
    words = words_of(pool, 1, D)
    words[:, :, 0, :, 1] = 0                                # keys s c
    put(pool, 1, D, words)
    flat = pool.reshape(pool.shape[0], -1)
    for b in range(B):
        byte = big[b] // 2
        flat[table[b, 0], byte] &= 0x0f if big[b] % 2 else 0xf0
    scale = float(2.0 ** min(far, 60) / largest) if 2.0 ** min(far, 60) / largest < 2.0 ** 63 else 2.0 ** 63
    out, lse, ws = attend(q.cuda(), dev(pool), dev(table), dev(np.int32([1] * B)), None, PAGE, D, 1, scale)
    assert sb.sv_read_device_flags(ws) == 0
    for b in range(B):
        codes, s, m = o4.read_tokens(pool, table[b], PAGE, 1, 1, D)
        key = s[0, 0, 0] * codes[0, 0, 0]
        assert key[big[b]] == 0
        f = f64(q[b, 0])
        z = scale * (f @ key)
        lost = 2.0 ** -35 * largest * scale * key.sum() if far > 26 and largest >= 2.0 ** -106 else 0
        bound = (D + 8) * 2.0 ** -23 * scale * (np.abs(f) @ key) + 2.0 ** -22 * np.abs(z) + lost
        assert np.all(np.abs(f64(lse)[b, 0] - z) <= bound)
