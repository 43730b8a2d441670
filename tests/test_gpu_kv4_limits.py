"""sv_kv4_append and sv_kv4_read with the largest T: room for 2^31 - 1 tokens a sequence, of which few are there."""

import numpy as np
import pytest

from oracle import draft4 as o4
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_kv4 import _lib, bf, dev, f64  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("T", [(1 << 31) - 1, (1 << 31) - 9, 1 << 30])
@pytest.mark.parametrize("H,D", [(1, 64), (2, 128)])
def test_the_largest_counts(T, H, D):
    r = np.random.default_rng(H)
    B, n, page = 3, np.int32([5, 0, 9]), 16
    k, v = bf(r.standard_normal((B, 9, H, D))).cuda(), bf(r.standard_normal((B, 9, H, D))).cuda()
    table, starts = dev(np.int32([[2], [1], [0]])), dev(np.int32([3, 0, 7]))
    pool = torch.zeros(B, sb.sv_kv4_page_bytes(H, D, page), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(4, dtype=torch.uint8, device="cuda")
    sb.sv_kv4_append(k, v, 9 * H * D, H * D, D, sb.SV_BF16, pool, B, page, table, 1, starts, dev(n), B, T, H, D, ws, 4)
    assert sb.sv_read_device_flags(ws) == 0
    want = np.zeros(pool.shape, np.uint8)
    for b in range(B):
        for i in range(n[b]):
            o4.write_token(want, 2 - b, [3, 0, 7][b] + i, page, f64(k[b, i]), f64(v[b, i]))
    assert np.array_equal(pool.cpu().numpy(), want)
    out = torch.full((2, B, 9, H, D), 7.0, device="cuda")
    sb.sv_kv4_read(pool, B, page, table, 1, starts, dev(n), out[0], out[1], 9 * H * D, H * D, D, sb.SV_F32, B, T, H, D, ws, 4)
    assert sb.sv_read_device_flags(ws) == 0
    for b in range(B):
        codes, s, m = o4.read_tokens(want, [2 - b], page, [3, 0, 7][b] + n[b], H, D)
        exact = (m[..., None] + s[..., None] * codes)[:, [3, 0, 7][b]:]
        assert np.allclose(out[:, b, :n[b]].cpu().numpy(), exact, rtol=2.0 ** -23, atol=0)
        assert torch.all(out[:, b, n[b]:] == 7.0)
