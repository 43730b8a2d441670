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


@pytest.mark.parametrize("B,T,H,D,page", [(2, 3, 96, 128, 5), (1, 2, 300, 64, 16), (3000, 2, 1, 64, 4), (1, 700, 20, 128, 32)])
def test_many_heads_and_many_sequences(B, T, H, D, page):
    """A token of more rows than a CTA takes at once, more sequences than rows of the grid."""
    r = np.random.default_rng(B + H)
    max_pages = -(-T // page) + 1
    starts = r.integers(0, page, B).astype(np.int32)
    n = r.integers(0, T + 1, B).astype(np.int32)
    n[0] = T
    table = r.permutation(B * max_pages).reshape(B, max_pages).astype(np.int32)
    k, v = bf(r.standard_normal((B, T, H, D))), bf(r.standard_normal((B, T, H, D)))
    pool = torch.zeros(B * max_pages, sb.sv_kv4_page_bytes(H, D, page), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(4, dtype=torch.uint8, device="cuda")
    args = (pool, B * max_pages, page, dev(table), max_pages, dev(starts), dev(n))
    sb.sv_kv4_append(k.cuda(), v.cuda(), 0, 0, 0, sb.SV_BF16, *args, B, T, H, D, ws, 4)
    assert sb.sv_read_device_flags(ws) == 0
    want = np.zeros(pool.shape, np.uint8)
    some = range(B) if B * T * H < 2000 else r.choice(B, min(B, 40), replace=False)
    kd, vd = f64(k), f64(v)
    for b in some:
        for i in range(n[b]) if T < 100 else sorted(r.choice(T, 30, replace=False)):
            t = starts[b] + i
            o4.write_token(want, table[b, t // page], t % page, page, kd[b, i], vd[b, i])
            h = (t % page) * D // 2
            got = pool[int(table[b, t // page])].cpu().numpy().reshape(H, -1)
            there = want[table[b, t // page]].reshape(H, -1)
            for part in range(2):
                at = part * page * D // 2 + h
                assert np.array_equal(got[:, at:at + D // 2], there[:, at:at + D // 2])
                at = page * D + part * page * 4 + (t % page) * 4
                assert np.array_equal(got[:, at:at + 4], there[:, at:at + 4])
    out = torch.full((2, B, T, H, D), 7.0, device="cuda")
    sb.sv_kv4_read(*args, out[0], out[1], 0, 0, 0, sb.SV_F32, B, T, H, D, ws, 4)
    x = torch.stack([k, v]).float().cuda()
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    there = (torch.arange(T, device="cuda")[None] < dev(n)[:, None])[None, :, :, None, None]
    # within half a step, and 15 roundings of the scale by 2^-8 where the largest codes are held at 15
    near = (out - x).abs() <= (high - low) / 15 * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -20
    assert torch.all(near | ~there) and torch.all((out == 7.0) | there)
