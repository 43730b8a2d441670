"""sv_prefix_attention at the edge of its sizes."""

import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_attention import SENTINEL, _lib  # noqa: F401  (the fixture builds the library)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


def test_a_bad_sequence_of_more_than_two_to_the_31_values():
    """One query of 2^24 heads of 128: every value of a sequence that fails is NaN."""
    hq, hkv, D = 1 << 24, 1 << 18, 128
    need = sb.sv_prefix_attention_workspace_size(1, 0, hq, hkv, D, 0, 4)
    if torch.cuda.mem_get_info()[0] < need + 4 * hq * D + (1 << 30):
        pytest.skip("needs 27 GB")
    q = torch.zeros(hq, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full((hq, D), SENTINEL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq,), SENTINEL, device="cuda")
    pool = torch.zeros(1, 4, hkv, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    table = torch.zeros(1, dtype=torch.int32, device="cuda")
    for length in (-1, 3):
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        sb.sv_prefix_attention(q, 0, 0, 0, pool, pool, 0, 0, 0, 1, 4, None, 0, table, 1, lens, None, 1.0, out, 0, 0, 0,
                               lse, sb.SV_BF16, 1, 0, hq, hkv, D, ws, ws.numel())
        flags = sb.sv_read_device_flags(ws)
        if length < 0:
            assert flags == sb.SV_FLAG_BAD_N
            assert torch.isnan(lse).all() and all(torch.isnan(part).all() for part in out.split(1 << 21))
        else:  # (keys of zeros: three equal scores, values of zeros)
            assert flags == 0
            assert torch.allclose(lse, torch.full_like(lse, 3.0).log()) and not any(part.any() for part in out.split(1 << 21))
