"""Long sequences in the attention backward: slow per-head decays, whose gradient is one number a
head, summed over every token, in which errors that stay from chunk to chunk would add up; and
head widths that are padded on the way, cut into segments; and many short sequences.  Needs a
GB300."""
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api
from tests.test_gpu_train import check_attn

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _identity():
    api.la_set_feature_map("identity")
    yield
    api.la_set_feature_map("identity")


def head_decay_grad(q, k, v, dO, decay):
    """In 64 bits: dlog gamma_h, the sum over tokens t of the pairs (i < t <= j), which is the sum
    over j >= t of q_j dq_j less that over i >= t of k_i dk_i.  Chunk by chunk."""
    B, H, L, _ = q.shape
    C = 128
    a = decay.double().view(1, H, 1, 1)
    n = torch.arange(C, device="cuda").double()
    D = torch.where(n[:, None] >= n, torch.exp(a * (n[:, None] - n).clamp(min=0)), 0.0)
    head, tail, whole = (torch.exp(a * m.view(1, 1, -1, 1)) for m in (n + 1, C - 1 - n, n[:1] + C))
    S = torch.zeros(B, H, q.shape[-1], v.shape[-1], device="cuda", dtype=torch.float64)
    G = torch.zeros_like(S)
    net = torch.zeros(B, H, L, device="cuda", dtype=torch.float64)
    chunks = [[t[:, :, c:c + C].double() for t in (q, k, v, dO)] for c in range(0, L, C)]
    for c, (Q, K, V, O) in enumerate(chunks):
        pairs = (Q @ K.mT) * (O @ V.mT) * D
        net[:, :, c * C:(c + 1) * C] += (
            pairs.sum(-1) - pairs.sum(-2) + ((O @ S.mT) * head * Q).sum(-1))
        S = whole * S + (tail * K).mT @ V
    for c in reversed(range(len(chunks))):
        Q, K, V, O = chunks[c]
        net[:, :, c * C:(c + 1) * C] -= ((V @ G.mT) * tail * K).sum(-1)
        G = whole * G + (head * Q).mT @ O
    return net.flip(-1).cumsum(-1).sum((0, 2))


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 64, 64), ("bf16", 64, 32), ("f32", 64, 64)])
def test_slow_head_decays(dtype, dk, dv):
    """The pairs around a chunk follow from those around the next one by two sums, and are
    formed anew every 512 tokens: at most 4 chunks of 128 tokens (more smaller ones, with as
    many tokens) follow one another.  A sum's products are cut, not rounded, 8 times (64 values in
    steps of 16, in two products): 8 U of its size.  8 such sums with independent signs: 23 U, and
    what the gradient's own sums are off: 32 U, 2e-6 of its size.  As many sequences as there are SMs, so that they run whole."""
    B, H, L = 4, 38, 8192
    g = torch.Generator("cuda").manual_seed(5)
    q, k = (torch.randn(B, H, L, dk, generator=g, device="cuda").mul_(0.2).to(DT[dtype])
            for _ in range(2))
    v, dO = (torch.randn(B, H, L, dv, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    decay = torch.log1p(-2.0 ** -torch.linspace(5, 13, H, device="cuda", dtype=torch.float64)).float()
    got = api.la_chunk_bwd(q, k, v, dO, decay_kind="head", decay=decay)[3].double()
    api.la_device_status()
    want = head_decay_grad(q, k, v, dO, decay)
    assert (got - want).norm() <= 32 * 2.0 ** -24 * want.norm()


@pytest.mark.parametrize("phi,kind,dk,dv", [
    ("identity", "token", 16, 64), ("identity", "logit", 32, 16), ("identity", "head", 128, 64),
    ("identity", "token", 64, 128), ("elu1", "none", 16, 32), ("elu1", "token", 32, 128)])
def test_unequal_heads_in_segments(phi, kind, dk, dv):
    """Widths that are padded on the way, in sequences that are cut; odd lengths."""
    check_attn(1, 3, 3001, dk, dv, "bf16", phi, kind, states=True, seed=dk + dv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 32), (64, 64), (128, 16)])
def test_nothing_is_written_past_the_gradients(dtype, dk, dv):
    B, H, L = 2, 3, 133
    g = torch.Generator("cuda").manual_seed(9)
    q, k = (torch.randn(B, H, L, dk, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    v, dO = (torch.randn(B, H, L, dv, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    decay = -0.1 * torch.rand(B, H, L, generator=g, device="cuda")
    S0 = torch.randn(B, H, dk, dv, generator=g, device="cuda")
    want = api.la_chunk_bwd(q, k, v, dO, decay_kind="token", decay=decay, S0=S0)
    pads, outs = [], []
    for t in want:
        pad = torch.full((t.numel() + 128,), 7.0, dtype=t.dtype, device="cuda")
        pads.append(pad)
        outs.append(pad[64:-64].view(t.shape))
    dq, dk_, dv_, dd, ds = outs
    api.la_chunk_bwd(q, k, v, dO, decay_kind="token", decay=decay, S0=S0, dq=dq, dk=dk_, dv=dv_,
                     ddecay=dd, dS0=ds)
    api.la_device_status()
    for t, out, pad in zip(want, outs, pads):
        assert torch.equal(t, out)
        assert (pad[:64] == 7).all() and (pad[-64:] == 7).all()


@pytest.mark.parametrize("phi,kind", [("identity", "token"), ("identity", "none"), ("elu1", "head"),
                                      ("identity", "logit")])
@pytest.mark.parametrize("L,dk,dv", [(1, 64, 64), (5, 16, 32), (63, 64, 64), (64, 32, 64), (65, 64, 16)])
def test_many_short_sequences(L, dk, dv, phi, kind):
    """More sequences than SMs, of one chunk and just above it."""
    B, H = 5, 32
    check_attn(B, H, L, dk, dv, "bf16", phi, kind, states=L % 2 == 1)
    check_attn(B, H, L, dk, dv, "bf16", phi, kind, states=False, want_decay_grad=False)
