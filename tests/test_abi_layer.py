"""Host-side argument checks of the layer operators' calls: nothing reaches a device."""

import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from speculative_decoding_verification_47_gb300 import build

P = 1 << 20  # an aligned dummy address; none of these calls reaches the device


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return sb.lib()


def refused(call, defaults, kw, status):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    with pytest.raises(sb.SVError) as e:
        call(**a, stream=0)
    assert e.value.status == status, (kw, str(e.value))


ATTN = dict(q=P, q_seq_stride=0, q_pos_stride=0, q_head_stride=0, k_pool=P, v_pool=P, page_stride=0,
            token_stride=0, head_stride=0, num_pages=10, page_size=16, prefix_pages=P, prefix_len=20,
            block_table=P, max_pages=4, seq_lens=P, k_per_row=None, scale=0.1, out=P,
            out_seq_stride=0, out_pos_stride=0, out_head_stride=0, lse=None, dtype=sb.SV_BF16, B=2,
            K=3, Hq=8, Hkv=2, D=128, workspace=P, workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=sb.SV_F32), sb.SV_ERR_DTYPE), (dict(dtype=sb.SV_E4M3), sb.SV_ERR_DTYPE),
    (dict(B=0), sb.SV_ERR_SHAPE), (dict(K=21), sb.SV_ERR_SHAPE), (dict(K=-1), sb.SV_ERR_SHAPE),
    (dict(Hq=0), sb.SV_ERR_SHAPE), (dict(Hq=7), sb.SV_ERR_SHAPE), (dict(Hkv=0), sb.SV_ERR_SHAPE),
    (dict(Hq=130, Hkv=2), sb.SV_ERR_SHAPE), (dict(D=96), sb.SV_ERR_SHAPE),
    (dict(D=256), sb.SV_ERR_SHAPE), (dict(page_size=0), sb.SV_ERR_SHAPE),
    (dict(max_pages=0), sb.SV_ERR_SHAPE), (dict(num_pages=0), sb.SV_ERR_SHAPE),
    (dict(prefix_len=-1), sb.SV_ERR_SHAPE), (dict(prefix_len=0x7fffffff - 10), sb.SV_ERR_SHAPE),
    (dict(max_pages=1 << 27), sb.SV_ERR_SHAPE), (dict(B=1 << 28), sb.SV_ERR_SHAPE),
    (dict(q=None), sb.SV_ERR_ARG), (dict(k_pool=None), sb.SV_ERR_ARG),
    (dict(v_pool=None), sb.SV_ERR_ARG), (dict(block_table=None), sb.SV_ERR_ARG),
    (dict(seq_lens=None), sb.SV_ERR_ARG), (dict(out=None), sb.SV_ERR_ARG),
    (dict(prefix_pages=None), sb.SV_ERR_ARG), (dict(scale=float("nan")), sb.SV_ERR_ARG),
    (dict(scale=float("inf")), sb.SV_ERR_ARG), (dict(q=P + 8), sb.SV_ERR_ARG),
    (dict(out=P + 2), sb.SV_ERR_ARG), (dict(lse=P + 2), sb.SV_ERR_ARG),
    (dict(q_pos_stride=1028), sb.SV_ERR_SHAPE), (dict(token_stride=-8), sb.SV_ERR_SHAPE),
    (dict(out_head_stride=64), sb.SV_ERR_SHAPE), (dict(workspace=None), sb.SV_ERR_WORKSPACE),
    (dict(workspace=P + 16), sb.SV_ERR_WORKSPACE), (dict(workspace_bytes=255), sb.SV_ERR_WORKSPACE),
])
def test_prefix_attention_host_checks(kw, status):
    refused(sb.sv_prefix_attention, ATTN, kw, status)


def test_prefix_attention_workspace_size():
    size = sb.sv_prefix_attention_workspace_size
    assert size(2, 3, 8, 2, 128, 20, 64) >= 256
    for bad in [(0, 3, 8, 2, 128, 20, 64), (2, 21, 8, 2, 128, 20, 64), (2, 3, 8, 3, 128, 20, 64),
                (2, 3, 8, 2, 96, 20, 64), (2, 3, 8, 2, 128, -1, 64), (2, 3, 8, 2, 128, 20, 0)]:
        assert size(*bad) == 0, bad
    w = size(256, 8, 32, 8, 128, 16384, 4112)
    refused(sb.sv_prefix_attention, {**ATTN, "B": 256, "K": 8, "Hq": 32, "Hkv": 8, "prefix_len": 16384,
                                     "max_pages": 257}, dict(workspace_bytes=w - 1),
            sb.SV_ERR_WORKSPACE)


NORM = dict(x=P, ldx=0, residual=2 * P, ldr=0, norm_w=3 * P, eps=1e-5, residual_out=4 * P, ldro=0,
            dtype=sb.SV_BF16, out=5 * P, ldo=0, out_dtype=sb.SV_E4M3, out_scale=6 * P, M=4, H=64)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=sb.SV_E4M3), sb.SV_ERR_DTYPE), (dict(dtype=9), sb.SV_ERR_DTYPE),
    (dict(out_dtype=sb.SV_F32), sb.SV_ERR_DTYPE), (dict(M=0), sb.SV_ERR_SHAPE),
    (dict(H=0), sb.SV_ERR_SHAPE), (dict(ldx=63), sb.SV_ERR_SHAPE), (dict(ldr=-64), sb.SV_ERR_SHAPE),
    (dict(ldro=1), sb.SV_ERR_SHAPE), (dict(ldo=63), sb.SV_ERR_SHAPE), (dict(x=None), sb.SV_ERR_ARG),
    (dict(norm_w=None), sb.SV_ERR_ARG), (dict(out=None), sb.SV_ERR_ARG),
    (dict(out_scale=None), sb.SV_ERR_ARG), (dict(eps=-1.0), sb.SV_ERR_ARG),
    (dict(eps=float("nan")), sb.SV_ERR_ARG), (dict(x=P + 1), sb.SV_ERR_ARG),
    (dict(dtype=sb.SV_F32, x=P + 2), sb.SV_ERR_ARG), (dict(out_scale=6 * P + 2), sb.SV_ERR_ARG),
    (dict(residual_out=2 * P, ldro=128), sb.SV_ERR_ARG), (dict(out=P), sb.SV_ERR_ARG),
    (dict(out=4 * P), sb.SV_ERR_ARG),
])
def test_rmsnorm_residual_host_checks(kw, status):
    refused(sb.sv_rmsnorm_residual, NORM, kw, status)


LINEAR = dict(x=P, ldx=0, x_scale=None, W=2 * P, ldw=0, w_scale=None, in_dtype=sb.SV_BF16, bias=None,
              residual=None, ldr=0, act=sb.SV_ACT_NONE, out=3 * P, ldo=0, out_dtype=sb.SV_BF16, M=4,
              N=32, K=64, workspace=P, workspace_bytes=256)


@pytest.mark.parametrize("kw,status", [
    (dict(in_dtype=sb.SV_F32), sb.SV_ERR_DTYPE), (dict(out_dtype=sb.SV_E4M3), sb.SV_ERR_DTYPE),
    (dict(M=0), sb.SV_ERR_SHAPE), (dict(N=0), sb.SV_ERR_SHAPE), (dict(K=0), sb.SV_ERR_SHAPE),
    (dict(K=63), sb.SV_ERR_SHAPE), (dict(ldx=68), sb.SV_ERR_SHAPE), (dict(ldw=32), sb.SV_ERR_SHAPE),
    (dict(ldo=31), sb.SV_ERR_SHAPE), (dict(ldx=-64), sb.SV_ERR_SHAPE),
    (dict(in_dtype=sb.SV_E4M3, ldx=72), sb.SV_ERR_SHAPE), (dict(ldw=1 << 39), sb.SV_ERR_SHAPE),
    (dict(act=5), sb.SV_ERR_ARG), (dict(act=-1), sb.SV_ERR_ARG), (dict(x=None), sb.SV_ERR_ARG),
    (dict(W=None), sb.SV_ERR_ARG), (dict(out=None), sb.SV_ERR_ARG), (dict(x=P + 2), sb.SV_ERR_ARG),
    (dict(W=P + 8), sb.SV_ERR_ARG), (dict(bias=P + 1), sb.SV_ERR_ARG),
    (dict(x_scale=P + 2), sb.SV_ERR_ARG), (dict(out=3 * P + 1), sb.SV_ERR_ARG),
    (dict(residual=3 * P, ldr=64), sb.SV_ERR_ARG), (dict(out=P), sb.SV_ERR_ARG),
    (dict(workspace=None), sb.SV_ERR_WORKSPACE), (dict(workspace=P + 4), sb.SV_ERR_WORKSPACE),
    (dict(workspace_bytes=4), sb.SV_ERR_WORKSPACE),
])
def test_linear_host_checks(kw, status):
    refused(sb.sv_linear, LINEAR, kw, status)


def test_linear_workspace_size():
    assert sb.sv_linear_workspace_size(4, 32, 64) >= 4
    assert sb.sv_linear_workspace_size(0, 32, 64) == 0


def test_other_calls_refuse_the_8_bit_type():
    assert sb.sv_workspace_size(4, 2, 10, sb.SV_E4M3) == 0
    with pytest.raises(sb.SVError) as e:
        sb.sv_draft_sample(P, 0, 0, sb.SV_E4M3, 4, 3, 100, None, None, 1.0, P, None, P, P, 256, 0)
    assert e.value.status == sb.SV_ERR_DTYPE
    with pytest.raises(sb.SVError) as e:
        sb.sv_lmhead_rmsnorm(P, P, 1e-5, P, P, sb.SV_E4M3, 4, 128, 128, P, 1 << 30, 0)
    assert e.value.status == sb.SV_ERR_DTYPE
