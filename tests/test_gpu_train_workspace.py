"""The attention's backward pass in a workspace of just the bytes that its call needs.  Needs a GB300."""
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _identity():
    api.la_set_feature_map("identity")
    yield
    api.la_set_feature_map("identity")


@pytest.mark.parametrize("kind,ddecay,dS0", [("none", False, False), ("none", False, True),
                                             ("head", False, False), ("head", True, False),
                                             ("token", True, True), ("logit", False, True)])
@pytest.mark.parametrize("dtype,phi", [("bf16", "identity"), ("bf16", "elu1"), ("f32", "identity")])
@pytest.mark.parametrize("B,H,L,dk,dv", [(1, 1, 1, 16, 16), (2, 3, 700, 64, 32), (1, 2, 3000, 128, 128),
                                         (5, 32, 60, 64, 64), (1, 1, 129, 16, 128)])
def test_exact_workspace(B, H, L, dk, dv, dtype, phi, kind, ddecay, dS0):
    """Nothing behind it is written, and what lies in it or behind it before does not matter."""
    api.la_set_feature_map(phi)
    g = torch.Generator("cuda").manual_seed(L)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k = (rand(B, H, L, dk).mul_(0.3).to(DT[dtype]) for _ in range(2))
    v, dO = (rand(B, H, L, dv).to(DT[dtype]) for _ in range(2))
    decay = {"none": None, "head": -0.1 * torch.rand(H, generator=g, device="cuda"),
             "token": -2 * torch.rand(B, H, L, generator=g, device="cuda"),
             "logit": 2 * rand(B, H, L)}[kind]
    if kind == "token":
        decay[..., ::50] = -8.0  # strong ones, whose chunks keep their states
    S0, dSf = rand(B, H, dk, dv), rand(B, H, dk, dv)
    need = api.la_chunk_bwd_workspace_bytes_for(B, H, L, dk, dv, 64, DT[dtype], kind, ddecay, dS0)
    most = api.la_chunk_bwd_workspace_bytes(B, H, L, dk, dv, 64, DT[dtype])
    call = lambda ws: api.la_chunk_bwd(  # noqa: E731
        q, k, v, dO, decay_kind=kind, decay=decay, S0=S0, dS_final=dSf, want_decay_grad=ddecay,
        want_state_grad=dS0, workspace=ws)
    want = call(torch.zeros(most, dtype=torch.uint8, device="cuda"))
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")  # NaNs
    got = call(ws[:need])
    api.la_device_status()
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    assert (got[3] is not None) == ddecay and (got[4] is not None) == dS0
    assert (ws[need:] == 255).all()
    with pytest.raises(api.LAError):
        call(ws[:need - 1])


def test_a_call_without_fp32_gradients_allocates_little():
    """No kept states, no shares: segment states alone."""
    B, H, L, d = 2, 32, 8192, 128
    q, k, v, dO = (torch.randn(B, H, L, d, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    outs = [torch.empty_like(q) for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    api.la_chunk_bwd(q, k, v, dO, dq=outs[0], dk=outs[1], dv=outs[2])
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < 32 << 20


@pytest.mark.parametrize("kind", ["head", "token", "logit"])
@pytest.mark.parametrize("dtype,phi,dk,dv", [("bf16", "identity", 64, 64), ("bf16", "identity", 128, 128),
                                             ("bf16", "identity", 32, 128), ("bf16", "elu1", 64, 64),
                                             ("f32", "identity", 128, 64)])
def test_state_gradient_without_the_decays(dtype, phi, dk, dv, kind):
    """dS0 alone is formed as beside ddecay: the same bits, of dq, dk and dv too."""
    api.la_set_feature_map(phi)
    g = torch.Generator("cuda").manual_seed(dk)
    B, H, L = 2, 3, 900
    q, k, v, dO = (torch.randn(B, H, L, d, generator=g, device="cuda").mul_(0.4).to(DT[dtype])
                   for d in (dk, dk, dv, dv))
    decay = torch.randn(B, H, L, generator=g, device="cuda")
    decay = {"head": -0.01 * decay[0, :, 0].abs(), "token": -decay.abs(), "logit": decay}[kind]
    S0, dSf = (torch.randn(B, H, dk, dv, generator=g, device="cuda") for _ in range(2))
    call = lambda ddecay: api.la_chunk_bwd(  # noqa: E731
        q, k, v, dO, decay_kind=kind, decay=decay.contiguous(), S0=S0, dS_final=dSf, want_decay_grad=ddecay)
    alone, both = call(False), call(True)
    api.la_device_status()
    assert alone[3] is None and both[3] is not None
    for i in (0, 1, 2, 4):
        assert torch.equal(alone[i], both[i])
