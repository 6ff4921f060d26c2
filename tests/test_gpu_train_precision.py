"""How far bf16 gradients are off beside the rounding of the outputs themselves.  Needs a GB300."""
import numpy as np
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api
from tests import train_reference as T

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _identity():
    api.la_set_feature_map("identity")
    yield
    api.la_set_feature_map("identity")


def exact(q, k, v, dO, phi, la):
    q, k, v, dO = map(T.f64, (q, k, v, dO))
    q1, k1 = np.ones_like(q), np.ones_like(k)
    if phi == "elu1":
        q1, k1 = (np.where(x > 0, 1.0, np.exp(np.minimum(x, 0))) for x in (q, k))
        q, k = (np.where(x > 0, x + 1, np.exp(np.minimum(x, 0))) for x in (q, k))
    out = [np.empty_like(x) for x in (q, k, v)]
    for at in np.ndindex(*q.shape[:2]):
        for o, x in zip(out, T._walk(q[at], k[at], v[at], dO[at], la[at], None, None)):
            o[at] = x
    return out[0] * q1, out[1] * k1, out[2]


@pytest.mark.parametrize("phi", ["identity", "elu1"])
@pytest.mark.parametrize("kind", ["none", "token"])
@pytest.mark.parametrize("B,H,L,dk,dv", [(1, 2, 900, 64, 64), (1, 2, 900, 128, 128), (1, 2, 600, 16, 32),
                                         (1, 2, 500, 64, 128), (1, 2, 60, 64, 64), (5, 32, 60, 64, 64)])
def test_roundings_of_bf16_gradients(B, H, L, dk, dv, kind, phi):
    """The outputs' rounding, and that of one operand of every product (a score, or the state): of
    equal size and independent, so 1.42 times the outputs' alone; a decayed key or query is one
    more, 1.74 times.  phi's own would be another."""
    g = torch.Generator().manual_seed(L + dk)
    q, k = (torch.randn(B, H, L, dk, generator=g).bfloat16() for _ in range(2))
    v, dO = (torch.randn(B, H, L, dv, generator=g).bfloat16() for _ in range(2))
    decay = -0.02 * torch.rand(B, H, L, generator=g) if kind == "token" else None
    la = T.log_decay(kind, decay, B, H, L)[0]
    api.la_set_feature_map(phi)
    got = api.la_chunk_bwd(*(t.cuda() for t in (q, k, v, dO)), decay_kind=kind,
                           decay=None if decay is None else decay.cuda(), want_decay_grad=False)
    api.la_device_status()
    most = 1.5 if kind == "none" else 1.8
    for name, x, want in zip(("dq", "dk", "dv"), got, exact(q, k, v, dO, phi, la)):
        rounded = torch.from_numpy(want).bfloat16().double().numpy()
        off, alone = (np.linalg.norm(y - want) for y in (T.f64(x), rounded))
        assert off <= most * alone, (name, off / alone)
