"""Rows of the 4-bit cache whose minimum is far below values on the borders of the codes: the codes
are those of exact arithmetic (fractions), whichever side of the border x - m lies on.  And values that
are read back as bf16: m + s c rounded once, wherever a sum in between might have been rounded too."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import draft4 as o4
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


def exact_codes(row, s):
    """round((x - min) / s), ties to even (Python's rounding of fractions), at most 15."""
    m, s = Fraction(float(min(row))), Fraction(float(s))
    return [min(round((Fraction(float(x)) - m) / s), 15) for x in row]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [0, -126 + 20, -62, 100])
def test_codes_next_to_borders(D, at):
    r = np.random.default_rng(D + at + 200)
    rows = []
    for far in (3, 10, 15, 17, 20, 22, 23, 24, 25, 26, 30, 40, 60, 100):
        for step in (1.0, 1.5, 1.25, 1.75):
            for sign in (1, -1):
                x = (r.integers(0, 15, D) + 0.5) * step                     # on borders, where 8 bits hold them
                x = np.where(r.uniform(size=D) < 0.2, r.integers(1, 16, D) * step, x)
                x[r.integers(0, D)] = 15 * step
                lowest = sign * 2.0 ** -far * r.choice([1, 1.5, 129 / 128])
                x = np.maximum(x, abs(lowest) * 2)
                x[r.integers(0, D // 2) + (0 if x[D // 2:].max() == 15 * step else D // 2)] = lowest
                rows.append(o4.bf16(x * 2.0 ** at))
    rows = np.array(rows)
    rows = rows[np.all(np.abs(rows) < 3e38, -1)]
    n = len(rows)
    x = torch.from_numpy(rows).to(torch.bfloat16).reshape(1, n, 1, D)
    assert np.array_equal(x.double().numpy().reshape(n, D), rows)
    pool = torch.zeros(1, sb.sv_kv4_page_bytes(1, D, n), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(4, dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")
    sb.sv_kv4_append(x.cuda(), (-x).cuda(), 0, 0, 0, sb.SV_BF16, pool, 1, n, i32(0).reshape(1, 1), 1, i32(0), None, 1, n, 1, D,
                     ws, 4)
    codes, s, m = o4.read_tokens(pool.cpu().numpy(), [0], n, n, 1, D)
    off, ties = [], 0
    for part, sign in enumerate((1, -1)):
        want_s, want_m = o4.quantise(sign * rows)[1:]
        assert np.array_equal(s[part, :, 0], want_s) and np.array_equal(m[part, :, 0], want_m)
        for t in range(n):
            want = exact_codes(sign * rows[t], s[part, t, 0])
            off += [(part, t, d) for d in range(D) if codes[part, t, 0, d] != want[d]]
            ties += sum(2 * (Fraction(float(v)) / Fraction(float(s[part, t, 0]))) % 2 == 1 for v in rows[t])
    assert not off, (len(off), off[:5])
    assert ties > 100  # values on borders but for the minimum


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [0, -100, 100])
def test_codes_of_values_next_to_zero(D, at):
    """Rows in which 0 lies on a border (a minimum of an odd number of half steps), with values so near to 0 that the
    difference to the minimum rounds onto the border: the side decides."""
    r = np.random.default_rng(D + at + 200)
    rows = []
    for odd in range(1, 30, 2):
        for step in (1.0, 1.25, 0.625, 1.375, 1.625, 129 / 128):
            low, high = -odd * 0.5 * step, (30 - odd) * 0.5 * step
            if o4.bf16(low) != low or o4.bf16(high) != high:
                continue
            x = r.uniform(low, high, D)
            tiny = r.choice([-1, 1], D) * r.integers(128, 256, D) / 128 * 2.0 ** -r.integers(10, 27, D).astype(float)
            x = np.where(r.uniform(size=D) < 0.4, tiny, x)
            x[:4] = 0.0, low, high, -2.0 ** -25
            rows.append(o4.bf16(r.permutation(x)) * 2.0 ** at)
    rows = np.array(rows)
    n = len(rows)
    assert n > 40
    x = torch.from_numpy(rows).to(torch.bfloat16).reshape(1, n, 1, D)
    pool = torch.zeros(1, sb.sv_kv4_page_bytes(1, D, n), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(4, dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")
    sb.sv_kv4_append(x.cuda(), (-x).cuda(), 0, 0, 0, sb.SV_BF16, pool, 1, n, i32(0).reshape(1, 1), 1, i32(0), None, 1, n, 1, D,
                     ws, 4)
    codes, s, m = o4.read_tokens(pool.cpu().numpy(), [0], n, n, 1, D)
    for part, sign in enumerate((1, -1)):
        want_s, want_m = o4.quantise(sign * rows)[1:]
        assert np.array_equal(s[part, :, 0], want_s) and np.array_equal(m[part, :, 0], want_m)
        for t in range(n):
            assert codes[part, t, 0].tolist() == exact_codes(sign * rows[t], s[part, t, 0]), (part, t)


def nearest_bf16(v):
    """The bf16 value nearest to a fraction, ties to even; 2^-133 is the smallest step."""
    if v == 0:
        return 0.0
    e = -126
    while abs(v) >= Fraction(2) ** (e + 1):
        e += 1
    step = Fraction(2) ** (e - 7)
    return float(round(v / step) * step)


def test_read_back_rounds_once():
    """Scales and minima any number of powers of two apart, products s c on the borders of bf16 among them."""
    r = np.random.default_rng(4)
    D, n = 64, 700
    pool = r.integers(0, 256, (1, o4.head_bytes(D, n))).astype(np.uint8)
    s = r.integers(128, 256, (2, n)) * 2.0 ** -7                             # every scale's 8 bits
    s = np.where(r.uniform(size=(2, n)) < 0.5, r.choice([131, 129, 171, 215], (2, n)) / 128, s)
    far = r.integers(-6, 60, (2, n))
    m = r.choice([-1.0, 1.0], (2, n)) * r.integers(128, 256, (2, n)) * 2.0 ** -7 * 2.0 ** -far.astype(float)
    base = 2.0 ** r.choice([-120, -30, 0, 90], (2, n))
    s, m = s * base, o4.bf16(m * base)
    pool[0, n * D:n * (D + 8)] = np.stack([o4.bf16_bits(s), o4.bf16_bits(m)], -1).astype(np.uint16).view(np.uint8).reshape(-1)
    codes, gs, gm = o4.read_tokens(pool, [0], n, n, 1, D)
    assert np.array_equal(gs[..., 0], s) and np.array_equal(gm[..., 0], m)
    out = torch.zeros(2, 1, n, 1, D, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(2, 1, n, 1, D, device="cuda")
    ws = torch.zeros(4, dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")
    for o, t in ((out, sb.SV_BF16), (wide, sb.SV_F32)):
        sb.sv_kv4_read(torch.from_numpy(pool).cuda(), 1, n, i32(0).reshape(1, 1), 1, i32(0), None, o[0], o[1], 0, 0, 0, t, 1, n,
                       1, D, ws, 4)
    got, wide = out.double().cpu().numpy(), wide.cpu().numpy()
    twice = 0
    for part in range(2):
        for t in range(n):
            for c in set(codes[part, t, 0].astype(int)):
                v = Fraction(float(m[part, t])) + Fraction(float(s[part, t])) * c
                want = nearest_bf16(v)
                here = got[part, 0, t, 0][codes[part, t, 0] == c]
                assert np.all(here == want), (part, t, c, float(v), want, here[0])
                w = wide[part, 0, t, 0][codes[part, t, 0] == c][0]
                assert w == np.float32(float(v)) or abs(Fraction(float(w)) - v) <= abs(v) * Fraction(1, 2 ** 24)
                twice += float(o4.bf16(float(w))) != want
    assert twice > 20  # a rounding by way of float32 gives another value there
