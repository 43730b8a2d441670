"""Host-side argument checks of the 4-bit draft's calls: nothing reaches a device."""

import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests.test_abi_layer import P, lib, refused  # noqa: F401  (the fixture builds the library)

BIG = 1 << 40

APPEND = dict(k=P, v=2 * P, seq_stride=0, pos_stride=0, head_stride=0, dtype=sb.SV_BF16, pool=3 * P, num_pages=10,
              page_size=16, block_table=P, max_pages=4, starts=P, n_per_row=None, B=2, T=3, Hkv=2, D=128, workspace=P,
              workspace_bytes=256)
READ = {("k_out" if k == "k" else "v_out" if k == "v" else k): v for k, v in APPEND.items()}
ROWS = [
    (dict(dtype=sb.SV_E4M3), sb.SV_ERR_DTYPE), (dict(B=0), sb.SV_ERR_SHAPE), (dict(T=0), sb.SV_ERR_SHAPE),
    (dict(Hkv=0), sb.SV_ERR_SHAPE), (dict(D=96), sb.SV_ERR_SHAPE), (dict(page_size=0), sb.SV_ERR_SHAPE),
    (dict(num_pages=0), sb.SV_ERR_SHAPE), (dict(max_pages=0), sb.SV_ERR_SHAPE),
    (dict(max_pages=1 << 27), sb.SV_ERR_SHAPE), (dict(Hkv=1 << 20, page_size=64), sb.SV_ERR_SHAPE),
    (dict(B=1 << 30, T=1 << 30), sb.SV_ERR_SHAPE), (dict(pos_stride=260), sb.SV_ERR_SHAPE),
    (dict(seq_stride=-8), sb.SV_ERR_SHAPE), (dict(pool=None), sb.SV_ERR_ARG), (dict(block_table=None), sb.SV_ERR_ARG),
    (dict(starts=None), sb.SV_ERR_ARG), (dict(pool=P + 8), sb.SV_ERR_ARG), (dict(starts=P + 2), sb.SV_ERR_ARG),
    (dict(n_per_row=P + 1), sb.SV_ERR_ARG), (dict(block_table=P + 2), sb.SV_ERR_ARG),
    (dict(workspace=None), sb.SV_ERR_WORKSPACE), (dict(workspace=P + 2), sb.SV_ERR_WORKSPACE),
    (dict(workspace_bytes=3), sb.SV_ERR_WORKSPACE),
]


@pytest.mark.parametrize("kw,status", ROWS + [
    (dict(dtype=sb.SV_F32), sb.SV_ERR_DTYPE), (dict(k=None), sb.SV_ERR_ARG), (dict(v=None), sb.SV_ERR_ARG),
    (dict(k=P + 8), sb.SV_ERR_ARG), (dict(v=P + 2), sb.SV_ERR_ARG)])
def test_kv4_append_host_checks(kw, status):
    refused(sb.sv_kv4_append, APPEND, kw, status)


@pytest.mark.parametrize("kw,status", ROWS + [
    (dict(k_out=None), sb.SV_ERR_ARG), (dict(v_out=None), sb.SV_ERR_ARG), (dict(v_out=P + 8), sb.SV_ERR_ARG),
    (dict(head_stride=64), sb.SV_ERR_SHAPE), (dict(v_out=P), sb.SV_ERR_SHAPE)])
def test_kv4_read_host_checks(kw, status):
    refused(sb.sv_kv4_read, READ, kw, status)


def test_kv4_sizes():
    assert sb.sv_kv4_page_bytes(8, 128, 16) == 8 * 16 * 136
    assert sb.sv_kv4_page_bytes(3, 64, 7) == 3 * 512  # 504 bytes a head, rounded up to 16
    assert sb.sv_kv4_page_bytes(1, 128, 1) == 144
    for bad in [(0, 128, 16), (8, 96, 16), (8, 128, 0), (1 << 20, 128, 64)]:
        assert sb.sv_kv4_page_bytes(*bad) == 0, bad
    size = sb.sv_kv4_attention_workspace_size
    assert size(2, 3, 8, 2, 128) >= 256
    for bad in [(0, 3, 8, 2, 128), (2, 21, 8, 2, 128), (2, 3, 8, 3, 128), (2, 3, 8, 2, 96), (2, 3, 130, 2, 128)]:
        assert size(*bad) == 0, bad
    assert sb.sv_linear_w4_workspace_size(4, 32, 64) >= 4 and sb.sv_linear_w4_workspace_size(4, 32, 0) == 0
    assert sb.sv_kv_pages_workspace_size(100, 0) >= 16
    for bad in [(0, 1), (10, -1), (10, (1 << 24) + 1)]:
        assert sb.sv_kv_pages_workspace_size(*bad) == 0, bad


ATTN = dict(q=P, q_seq_stride=0, q_pos_stride=0, q_head_stride=0, pool=2 * P, num_pages=10, page_size=16,
            block_table=P, max_pages=4, seq_lens=P, k_per_row=None, window=0, sinks=0, scale=0.1, out=3 * P,
            out_seq_stride=0, out_pos_stride=0, out_head_stride=0, lse=None, dtype=sb.SV_BF16, B=2, K=3, Hq=8, Hkv=2,
            D=128, workspace=P, workspace_bytes=BIG)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=sb.SV_F32), sb.SV_ERR_DTYPE), (dict(B=0), sb.SV_ERR_SHAPE), (dict(K=21), sb.SV_ERR_SHAPE),
    (dict(K=-1), sb.SV_ERR_SHAPE), (dict(Hq=7), sb.SV_ERR_SHAPE), (dict(Hkv=0), sb.SV_ERR_SHAPE),
    (dict(Hq=130), sb.SV_ERR_SHAPE), (dict(D=96), sb.SV_ERR_SHAPE), (dict(page_size=0), sb.SV_ERR_SHAPE),
    (dict(max_pages=0), sb.SV_ERR_SHAPE), (dict(num_pages=0), sb.SV_ERR_SHAPE), (dict(window=-1), sb.SV_ERR_SHAPE),
    (dict(sinks=-1), sb.SV_ERR_SHAPE), (dict(max_pages=1 << 27), sb.SV_ERR_SHAPE), (dict(B=1 << 28), sb.SV_ERR_SHAPE),
    (dict(q_pos_stride=1028), sb.SV_ERR_SHAPE), (dict(out_seq_stride=-8), sb.SV_ERR_SHAPE),
    (dict(out_head_stride=64), sb.SV_ERR_SHAPE), (dict(q=None), sb.SV_ERR_ARG), (dict(pool=None), sb.SV_ERR_ARG),
    (dict(block_table=None), sb.SV_ERR_ARG), (dict(seq_lens=None), sb.SV_ERR_ARG), (dict(out=None), sb.SV_ERR_ARG),
    (dict(scale=float("nan")), sb.SV_ERR_ARG), (dict(scale=2.0 ** 64), sb.SV_ERR_ARG),
    (dict(scale=float("-inf")), sb.SV_ERR_ARG), (dict(q=P + 8), sb.SV_ERR_ARG), (dict(pool=P + 4), sb.SV_ERR_ARG),
    (dict(out=P + 2), sb.SV_ERR_ARG), (dict(lse=P + 2), sb.SV_ERR_ARG), (dict(seq_lens=P + 2), sb.SV_ERR_ARG),
    (dict(k_per_row=P + 1), sb.SV_ERR_ARG), (dict(block_table=P + 3), sb.SV_ERR_ARG),
    (dict(workspace=None), sb.SV_ERR_WORKSPACE), (dict(workspace=P + 16), sb.SV_ERR_WORKSPACE),
    (dict(workspace_bytes=255), sb.SV_ERR_WORKSPACE),
])
def test_kv4_attention_host_checks(kw, status):
    refused(sb.sv_kv4_attention, ATTN, kw, status)


LINEAR = dict(x=P, ldx=0, W=2 * P, ldw=0, scales=P, zeros=None, group=64, bias=None, residual=None, ldr=0,
              act=sb.SV_ACT_NONE, out=3 * P, ldo=0, out_dtype=sb.SV_BF16, M=4, N=32, K=128, workspace=P,
              workspace_bytes=BIG)


@pytest.mark.parametrize("kw,status", [
    (dict(out_dtype=sb.SV_E4M3), sb.SV_ERR_DTYPE), (dict(M=0), sb.SV_ERR_SHAPE), (dict(N=0), sb.SV_ERR_SHAPE),
    (dict(K=0), sb.SV_ERR_SHAPE), (dict(K=(1 << 30) + 64), sb.SV_ERR_SHAPE), (dict(group=16), sb.SV_ERR_SHAPE),
    (dict(group=256, K=256), sb.SV_ERR_SHAPE), (dict(K=96), sb.SV_ERR_SHAPE), (dict(ldx=120), sb.SV_ERR_SHAPE),
    (dict(ldx=132), sb.SV_ERR_SHAPE), (dict(ldw=63), sb.SV_ERR_SHAPE), (dict(ldw=72), sb.SV_ERR_SHAPE),
    (dict(ldo=31), sb.SV_ERR_SHAPE), (dict(ldr=-32), sb.SV_ERR_SHAPE), (dict(act=5), sb.SV_ERR_ARG),
    (dict(x=None), sb.SV_ERR_ARG), (dict(W=None), sb.SV_ERR_ARG), (dict(scales=None), sb.SV_ERR_ARG),
    (dict(out=None), sb.SV_ERR_ARG), (dict(x=P + 8), sb.SV_ERR_ARG), (dict(W=P + 4), sb.SV_ERR_ARG),
    (dict(scales=P + 1), sb.SV_ERR_ARG), (dict(bias=P + 1), sb.SV_ERR_ARG), (dict(out=P), sb.SV_ERR_ARG),
    (dict(residual=3 * P, ldr=64), sb.SV_ERR_ARG), (dict(out=3 * P + 1), sb.SV_ERR_ARG),
    (dict(workspace=None), sb.SV_ERR_WORKSPACE), (dict(workspace=P + 4), sb.SV_ERR_WORKSPACE),
    (dict(workspace_bytes=4), sb.SV_ERR_WORKSPACE), (dict(N=1 << 30, K=256, out=1 << 45), sb.SV_ERR_SHAPE),
    (dict(ldw=1 << 38), sb.SV_ERR_SHAPE), (dict(ldx=1 << 38), sb.SV_ERR_SHAPE),
])
def test_linear_w4_host_checks(kw, status):
    refused(sb.sv_linear_w4, LINEAR, kw, status)


POOLS = dict(pools=[P, 2 * P], page_bytes=[512, 1024], num_pools=2, num_pages=100)
COPY = dict(**POOLS, src=P, dst=P, n=5, workspace=P, workspace_bytes=BIG)
TABLE = dict(block_table=P, max_pages=4, seq_lens=P, shares=P)
FORK = dict(**POOLS, page_size=16, **TABLE, free_pages=P, free_top=P, src=P, dst=P, F=3, B=8, workspace=P,
            workspace_bytes=BIG)
FREE = dict(**TABLE, num_pages=100, free_pages=P, free_top=P, free_capacity=100, seqs=P, n=3, B=8, workspace=P,
            workspace_bytes=BIG)
COMPACT = dict(**POOLS, block_table=P, max_pages=4, B=8, prefix_pages=P, prefix_count=2, shares=P, free_pages=P,
               free_top=P, free_capacity=100, workspace=P, workspace_bytes=BIG)
OF_POOLS = [
    (dict(pools=[P, None]), sb.SV_ERR_ARG), (dict(pools=[P, P + 8]), sb.SV_ERR_ARG), (dict(pools=None), sb.SV_ERR_ARG),
    (dict(page_bytes=None), sb.SV_ERR_ARG), (dict(page_bytes=[512, 1000]), sb.SV_ERR_SHAPE),
    (dict(page_bytes=[0, 512]), sb.SV_ERR_SHAPE), (dict(page_bytes=[512, 1 << 31]), sb.SV_ERR_SHAPE),
    (dict(pools=[], page_bytes=[], num_pools=0), sb.SV_ERR_SHAPE),
    (dict(pools=[P] * 257, page_bytes=[16] * 257, num_pools=257), sb.SV_ERR_SHAPE)]
OF_ALL = [(dict(num_pages=0), sb.SV_ERR_SHAPE), (dict(workspace=None), sb.SV_ERR_WORKSPACE),
          (dict(workspace=P + 8), sb.SV_ERR_WORKSPACE), (dict(workspace_bytes=15), sb.SV_ERR_WORKSPACE)]
OF_TABLE = [(dict(B=0), sb.SV_ERR_SHAPE), (dict(max_pages=0), sb.SV_ERR_SHAPE), (dict(block_table=None), sb.SV_ERR_ARG),
            (dict(block_table=P + 2), sb.SV_ERR_ARG), (dict(shares=None), sb.SV_ERR_ARG), (dict(free_top=P + 1), sb.SV_ERR_ARG),
            (dict(free_pages=None), sb.SV_ERR_ARG), (dict(max_pages=0x7fffffff), sb.SV_ERR_SHAPE)]


@pytest.mark.parametrize("kw,status", OF_POOLS + OF_ALL + [
    (dict(n=0), sb.SV_ERR_SHAPE), (dict(n=(1 << 24) + 1), sb.SV_ERR_SHAPE), (dict(src=None), sb.SV_ERR_ARG),
    (dict(dst=P + 2), sb.SV_ERR_ARG)])
def test_copy_pages_host_checks(kw, status):
    refused(sb.sv_kv_copy_pages, COPY, kw, status)


@pytest.mark.parametrize("kw,status", OF_POOLS + OF_ALL + OF_TABLE + [
    (dict(F=0), sb.SV_ERR_SHAPE), (dict(F=4097), sb.SV_ERR_SHAPE), (dict(page_size=0), sb.SV_ERR_SHAPE),
    (dict(max_pages=1 << 27), sb.SV_ERR_SHAPE), (dict(seq_lens=None), sb.SV_ERR_ARG), (dict(src=None), sb.SV_ERR_ARG),
    (dict(dst=None), sb.SV_ERR_ARG)])
def test_fork_host_checks(kw, status):
    refused(sb.sv_kv_fork, FORK, kw, status)


@pytest.mark.parametrize("kw,status", OF_ALL + OF_TABLE + [
    (dict(n=0), sb.SV_ERR_SHAPE), (dict(n=4097), sb.SV_ERR_SHAPE), (dict(free_capacity=99), sb.SV_ERR_SHAPE),
    (dict(seqs=None), sb.SV_ERR_ARG), (dict(seq_lens=P + 2), sb.SV_ERR_ARG)])
def test_free_host_checks(kw, status):
    refused(sb.sv_kv_free, FREE, kw, status)


@pytest.mark.parametrize("kw,status", OF_POOLS + OF_ALL + OF_TABLE + [
    (dict(free_capacity=99), sb.SV_ERR_SHAPE), (dict(prefix_count=-1), sb.SV_ERR_ARG),
    (dict(prefix_pages=None), sb.SV_ERR_ARG), (dict(prefix_pages=P + 1), sb.SV_ERR_ARG)])
def test_compact_host_checks(kw, status):
    refused(sb.sv_kv_compact, COMPACT, kw, status)


def test_pools_must_match_their_number():
    with pytest.raises(ValueError):
        sb.sv_kv_copy_pages([P], [512, 512], 2, 100, P, P, 5, P, BIG, 0)
