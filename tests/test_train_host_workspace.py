"""The workspace of the attention's backward pass: what a call's own parts come to, and no more."""
import os

import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import _native, api, build

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(_native.LIB_PATH):
        build.build()
    yield
    api.la_set_feature_map("identity")


def parts(B, H, L, dk, dv, dtype, phi, kind, ddecay, dS0):
    """Bytes of a call's parts without the states between segments, and those of one cut."""
    wide = max(dk, dv) > 64
    full = dtype == "f32" or (phi == "elu1" and (ddecay or dS0))  # inputs as three planes
    tc = not full and not (L <= 64 and not wide and B * H > 152)
    C = 128 if tc else 32 if full else 64
    seqs, chunks = B * H, -(-L // C)
    n = 0
    if kind != "none":
        n += 8 * seqs * chunks * C                       # log decays, two floats a token
    if ddecay:
        n += 4 * seqs * L * (5 if tc else 3)             # shares
        state = (128 if wide else 64) ** 2 if tc else dk * dv
        n += 4 * seqs * (chunks - 1) * (state + 16)      # kept states, <G, S> of them
        n += seqs * chunks * (9 if tc else 1)            # pairs around blocks, strong decays
    return n, 8 * seqs * dk * dv


CASES = [(1, 1, 1, 16, 16), (1, 1, 300, 16, 64), (4, 16, 4096, 64, 64), (2, 32, 8192, 128, 128),
         (1, 16, 32768, 128, 128), (3, 5, 777, 64, 128), (64, 32, 64, 64, 64), (1, 1, 1 << 20, 64, 64),
         (1, 4, 1 << 18, 32, 32), (8, 64, 512, 128, 128)]


@pytest.mark.parametrize("kind,ddecay,dS0", [("none", False, False), ("none", False, True),
                                             ("head", False, False), ("head", True, False),
                                             ("token", True, True), ("logit", False, True)])
@pytest.mark.parametrize("dtype,phi", [("bf16", "identity"), ("bf16", "elu1"), ("f32", "identity")])
@pytest.mark.parametrize("B,H,L,dk,dv", CASES)
def test_need_is_the_sum_of_its_parts(B, H, L, dk, dv, dtype, phi, kind, ddecay, dS0):
    api.la_set_feature_map(phi)
    need = api.la_chunk_bwd_workspace_bytes_for(B, H, L, dk, dv, 64, DT[dtype], kind, ddecay, dS0)
    least, cut = parts(B, H, L, dk, dv, dtype, phi, kind, ddecay, dS0)
    # parts start on 256 bytes; a sequence is cut until its pieces are about five waves of blocks, three
    # to an SM at most, and a piece holds 512 chunks at most
    cuts = max(1 + 5 * 3 * 152 // (B * H), -(-L // (512 * 32)))
    assert max(least, 256) <= need <= least + cuts * (cut + 8 * B * H) + 20 * 256
    if L <= 32:
        assert need <= least + 20 * 256  # one chunk: no cut
    most = api.la_chunk_bwd_workspace_bytes(B, H, L, dk, dv, 64, DT[dtype])
    assert need <= most
    if ddecay and (phi == "elu1" or dtype == "f32"):
        assert most <= 2 * need


def test_query_refuses_what_the_call_does():
    lib = _native.load()
    ask = lib.la_chunk_bwd_workspace_bytes_for
    assert ask(1, 1, 64, 64, 64, 64, 1, 0, 0, 0) > 0
    for bad in ((0, 1, 64, 64, 64, 64, 1, 0, 0, 0), (1, 1, 0, 64, 64, 64, 1, 0, 0, 0),
                (1, 1, 64, 48, 64, 64, 1, 0, 0, 0), (1, 1, 64, 64, 64, 65, 1, 0, 0, 0),
                (1, 1, 64, 64, 64, 64, 3, 0, 0, 0), (1, 1, 2 ** 30 + 1, 64, 64, 64, 1, 0, 0, 0),
                (2 ** 20, 2 ** 12, 64, 64, 64, 64, 1, 0, 0, 0), (1, 1, 64, 64, 64, 64, 1, 4, 0, 0),
                (1, 1, 64, 64, 64, 64, 1, -1, 0, 0), (1, 1, 64, 64, 64, 64, 1, 0, 1, 0)):
        assert ask(*bad) == 0
