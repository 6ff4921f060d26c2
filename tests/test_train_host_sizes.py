"""Sizes that do not fit the C ABI's ints are refused by the training pass's binding."""
import os

import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import _native, api, build

BIG = 2 ** 32 + 64  # cut to 32 bits it would be 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(_native.LIB_PATH):
        build.build()


@pytest.mark.parametrize("call", [
    lambda: api.la_rotary_frequencies(BIG),
    lambda: api.la_chunk_bwd_workspace_bytes(BIG, 1, 64, 64, 64),
    lambda: api.la_chunk_bwd_workspace_bytes(1, 1, BIG, 64, 64),
    lambda: api.la_chunk_bwd_workspace_bytes(1, 1, 64, 64, 64, chunk=BIG),
    lambda: api.la_gated_norm_bwd_workspace_bytes(1, BIG, 64, 64),
    lambda: api.la_gated_norm_bwd_workspace_bytes(1, 1, 64, 64, BIG),
    lambda: api.la_residual_norm_bwd_workspace_bytes(64, BIG),
    lambda: api.la_chunk_bwd(*[torch.zeros(1, 1, 4, 64)] * 4, chunk=BIG),
])
def test_sizes_past_32_bits(call):
    with pytest.raises(ValueError, match="2\\^31"):
        call()
