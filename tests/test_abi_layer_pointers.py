"""Calls that the host refuses because the device could not answer them: misaligned index
arrays, which would be a fault there, and scales whose product with log2(e) is infinite."""

import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests.test_abi_layer import ATTN, P, lib, refused  # noqa: F401  (the fixture builds the library)


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("name", ["prefix_pages", "block_table", "seq_lens", "k_per_row"])
def test_prefix_attention_index_arrays(name, off):
    refused(sb.sv_prefix_attention, ATTN, {name: P + off}, sb.SV_ERR_ARG)


@pytest.mark.parametrize("scale", [2.5e38, -2.5e38, 3.4e38])
def test_prefix_attention_scales(scale):
    refused(sb.sv_prefix_attention, ATTN, dict(scale=scale), sb.SV_ERR_ARG)
