"""Sizes at the ends of 32 bits in the training pass's calls.  Needs a GB300."""
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api

pytestmark = pytest.mark.gpu


def test_gated_norm_of_two_sequences_of_almost_2_31_tokens():
    """A team steps from the first sequence's last tokens into the second: its token index passes
    2^31 on the way.  Rows of one value, whose gradients have a closed form: n = x rho, dx =
    rho dy (1 - n^2) with rho = 1 / sqrt(x^2 + 1)."""
    B, L = 2, 2 ** 31 - 100
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(B, 1, L, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dy = torch.empty(B, L, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dx = torch.full_like(x, 7.0)
    api.la_gated_norm_bwd(dy, x, eps=1.0, dx=dx)
    api.la_device_status()
    n = 1 << 18
    for b in range(B):
        for part in (slice(0, n), slice(L // 2, L // 2 + n), slice(L - n, L)):
            X, Y = x[b, 0, part, 0].double(), dy[b, part, 0].double()
            want = Y / (X * X + 1) ** 1.5
            # half a step of bf16, and a dozen fp32 roundings of what cancels in 1 - n^2
            tol = want.abs() * 2.0 ** -8 + 12 * 2.0 ** -24 * Y.abs()
            assert ((dx[b, 0, part, 0].double() - want).abs() <= tol).all()
    for b in range(B):  # nothing left out (7.0 is above any gradient: |dy| stays below 7)
        assert not (dx[b] == 7.0).any()
