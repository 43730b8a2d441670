"""Bounded waits of the 4-bit attention and product that run out: the call ends, reports
SV_FLAG_TIMEOUT and leaves NaN; the next call is sound."""

import numpy as np
import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests import test_gpu_kv4 as kv
from tests import test_gpu_linear_w4 as w4
from tests.conftest import gpu_available
from tests.test_gpu_attention import _lib  # noqa: F401  (the fixture builds the library)
from tests.test_gpu_waits import no_patience

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("hq,K,L", [(4, 0, 300), (8, 1, 40), (16, 2, 5000)])
@pytest.mark.parametrize("D", [64, 128])
def test_kv4_attention(hq, K, L, D):
    r = np.random.default_rng(L)
    lens, ks = [L, 1, 0, L // 2], [K, 0, K, K // 2]
    q, pool, table, _ = kv.case(r, 4, K, hq, 2, D, 16, lens, ks)
    args = (q.cuda(), kv.dev(pool), kv.dev(table), kv.dev(np.int32(lens)), kv.dev(np.int32(ks)), 16, D, 2, 0.1)
    want = kv.attend(*args)
    with no_patience():
        out, lse, ws = kv.attend(*args)
    assert sb.sv_read_device_flags(ws) == sb.SV_FLAG_TIMEOUT
    for b in range(4):
        assert torch.isnan(out[b, :ks[b] + 1]).all() and torch.isnan(lse[b, :ks[b] + 1]).all()
        assert (out[b, ks[b] + 1:] == 7.0).all()
    ws[:4] = 0
    again = kv.attend(*args, ws=ws)  # the workspace is ready for the next call
    assert sb.sv_read_device_flags(ws) == 0
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("M,N,K,group", [(9, 200, 128, 32), (16, 8192, 8192, 64), (33, 300, 4096, 128), (70, 20000, 256, 64)])
def test_linear_w4(M, N, K, group):
    s = w4.inputs(M, M, N, K, group, True, True, False, torch.bfloat16)
    d = {k: None if v is None else v.cuda() for k, v in s.items()}
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(sb.sv_linear_w4_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    call = lambda: sb.sv_linear_w4(d["x"], 0, d["W"], 0, d["scales"], d["zeros"], group, d["bias"], None, 0, sb.SV_ACT_RELU,
                                   out, 0, sb.SV_BF16, M, N, K, ws, ws.numel())
    with no_patience():
        call()
    assert sb.sv_read_device_flags(ws) == sb.SV_FLAG_TIMEOUT and torch.isnan(out).all()
    ws.zero_()
    call()
    assert sb.sv_read_device_flags(ws) == 0
    w4.check(s, out, sb.SV_ACT_RELU, torch.bfloat16, group)
