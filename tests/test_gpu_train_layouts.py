"""The training pass's calls on the parts of packed projections: every order of the axes, in place,
into a packed gradient, at full length and on a prefix of a longer batch.  Needs a GB300."""
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api

pytestmark = pytest.mark.gpu

B, H, L, D = 3, 4, 9, 64
# where the axes b, p (the parts), l, h of the packed tensor end up, its last axis being d
ORDERS = ["bplh", "bphl", "blph", "blhp", "lbph", "pblh", "bhpl", "lbhp"]


def parts(order, longer, dtype, seed, fill=None):
    """The packed tensor and its three parts as [B,H,L,d] views of the first L tokens."""
    n = {"b": B, "p": 3, "l": L + longer, "h": H}
    g = torch.Generator("cuda").manual_seed(seed)
    t = torch.randn(*(n[a] for a in order), D, generator=g, device="cuda").to(dtype)
    if fill is not None:
        t.fill_(fill)
    at = [order.index(a) for a in "pbhl"] + [4]
    return t, [p[:, :, :L] for p in t.permute(at)]


def outside(t, order, longer, touched):
    """The elements of a packed tensor that the given parts (tokens before L) do not hold."""
    keep = torch.ones_like(t, dtype=torch.bool)
    at = [order.index(a) for a in "pbhl"] + [4]
    view = keep.permute(at)
    for p in touched:
        view[p][:, :, :L] = False
    return keep


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("longer", [0, 5])
@pytest.mark.parametrize("order", ORDERS)
def test_rotary_between_parts(order, longer, dtype):
    t, (q, k, _) = parts(order, longer, dtype, 1)
    t0 = t.clone()
    f = api.la_rotary_frequencies(D)[0].cuda()
    off = torch.tensor([0, 3, 1000], dtype=torch.int32, device="cuda")
    for call in (api.la_rotary_fwd, api.la_rotary_bwd):
        want = call(q.contiguous(), k.contiguous(), f, offsets=off)
        # into a packed tensor, from dense ones and from another packed one
        for x, y in ((q, k), (q.contiguous(), k.contiguous())):
            out, (qo, ko, _) = parts(order, longer, dtype, 2, fill=7.0)
            call(x, y, f, offsets=off, q_out=qo, k_out=ko)
            assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
            assert (out[outside(out, order, longer, (0, 1))] == 7).all()
        # in place
        call(q, k, f, offsets=off, q_out=q, k_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        rest = outside(t, order, longer, (0, 1))
        assert torch.equal(t[rest], t0[rest])


@pytest.mark.parametrize("longer", [0, 5])
@pytest.mark.parametrize("order", ORDERS)
def test_gated_norm_between_parts(order, longer):
    """x and its gradient as two parts of one tensor, and x's gradient over x."""
    t, (x, dx, _) = parts(order, longer, torch.bfloat16, 3)
    t0 = t.clone()
    g = torch.Generator("cuda").manual_seed(4)
    dy, gate = (torch.randn(B, L, H * D, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.rand(D, generator=g, device="cuda")
    want = api.la_gated_norm_bwd(dy, x.contiguous(), gate, w)
    got = api.la_gated_norm_bwd(dy, x, gate, w, dx=dx)
    for a, b in zip(got[:3], want):
        assert torch.equal(a, b)
    api.la_gated_norm_bwd(dy, x, gate, w, dx=x)
    assert torch.equal(x, want[0])
    rest = outside(t, order, longer, (0, 1))
    assert torch.equal(t[rest], t0[rest])


def test_gated_norm_forward_between_parts():
    """y into the rows of a packed tensor whose other part is x."""
    t, (x, _, _) = parts("blph", 0, torch.bfloat16, 5)
    t0 = t.clone()
    want = api.la_gated_norm_fwd(x.contiguous())
    y = t.view(B, L, 3 * H * D)[..., H * D:2 * H * D]
    api.la_gated_norm_fwd(x, y=y)
    assert torch.equal(y, want)
    assert torch.equal(t[:, :, 0], t0[:, :, 0]) and torch.equal(t[:, :, 2], t0[:, :, 2])
