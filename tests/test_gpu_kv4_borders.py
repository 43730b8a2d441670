"""Rows of the 4-bit cache whose minimum is far below values on the borders of the codes: the codes
are those of exact arithmetic (fractions), whichever side of the border x - m lies on."""

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
