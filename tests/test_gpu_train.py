"""The training pass's operators on the GPU, element by element against the 64-bit references and
their bounds, and run together as a layer.  Needs a GB300."""
import numpy as np
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api
from tests import ssm_reference as R
from tests import train_reference as T
from tests.test_gpu_ssm_limits import run_together

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _identity():
    api.la_set_feature_map("identity")
    yield
    api.la_set_feature_map("identity")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _compare(got, ref, live=None):
    for name, g in got.items():
        if g is not None:
            R.check(g, ref[name], name, live)


# ---------------------------------------------------------------- rotary positions
def rotary_inputs(B, Hq, Hk, L, d, rot, dtype, packed=True, seed=0):
    """q and k as slices of a projection's token-major output, with a few elements between."""
    g = _gen(seed)
    if packed:
        x = torch.randn(B, L, (Hq + Hk) * d + 8, generator=g).to(DT[dtype]).cuda()
        q = x[..., :Hq * d].unflatten(-1, (Hq, d)).permute(0, 2, 1, 3)
        k = x[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d)).permute(0, 2, 1, 3)
    else:
        q, k = (torch.randn(B, h, L, d, generator=g).to(DT[dtype]).cuda() for h in (Hq, Hk))
    f, _ = api.la_rotary_frequencies(rot)
    return q, k, f.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,L,d,rot,packed", [
    (1, 1, 1, 1, 2, 2, False),
    (3, 4, 4, 1, 64, 64, True),
    (2, 3, 1, 5, 64, 32, True),      # fewer heads of k, half of each head turned
    (2, 9, 17, 3, 128, 128, True),   # heads in several groups
    (1, 2, 2, 130, 80, 40, True),
    (2, 1, 2, 7, 16, 6, False),      # no vector divides the turned half
    (1, 3, 2, 9, 33, 32, False),     # an odd head size
    (1, 1, 1, 4, 40, 38, True),
    (300, 2, 2, 1, 256, 256, False),
    (1, 8, 8, 1500, 64, 64, True),
])
def test_rotary(B, Hq, Hk, L, d, rot, packed, backward, interleaved, dtype):
    q, k, f = rotary_inputs(B, Hq, Hk, L, d, rot, dtype, packed)
    offsets = torch.randint(0, 100000, (B,), generator=_gen(1), dtype=torch.int32)
    call = api.la_rotary_bwd if backward else api.la_rotary_fwd
    qo, ko = call(q, k, f, offsets=offsets.cuda(), interleaved=interleaved, scale=1.25)
    assert qo.is_contiguous() and ko.is_contiguous()
    pos = offsets[:, None].long() + torch.arange(L)
    for x, y in ((q, qo), (k, ko)):
        R.check(y, T.rotary(x, f, pos, 1.25, interleaved, backward, dtype), "rotary")
        if rot < d:  # what is not turned is copied as it is
            assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotary_positions_lengths_and_outputs_in_slices(dtype):
    B, H, L, d = 4, 3, 11, 64
    q, k, f = rotary_inputs(B, H, H, L, d, 64, dtype)
    g = _gen(2)
    pos = torch.randint(-50, 2 ** 20, (B, L), generator=g, dtype=torch.int32)
    off = torch.tensor([0, 7, -20, 2 ** 20], dtype=torch.int32)
    n = torch.tensor([0, 1, L + 5, -3], dtype=torch.int32)
    out = torch.full((B, L, 2 * H * d + 16), 7.0, dtype=DT[dtype], device="cuda")
    qo = out[..., :H * d].unflatten(-1, (H, d)).permute(0, 2, 1, 3)
    ko = out[..., H * d:2 * H * d].unflatten(-1, (H, d)).permute(0, 2, 1, 3)
    api.la_rotary_fwd(q, k, f, positions=pos.cuda(), offsets=off.cuda(), lengths=n.cuda(),
                      q_out=qo, k_out=ko)
    where = pos.long() + off[:, None].long()
    live = np.arange(L)[None] < np.clip(n.numpy(), 0, L)[:, None]
    rows = np.broadcast_to(live[:, None], (B, H, L))
    for x, y in ((q, qo), (k, ko)):
        R.check(y, T.rotary(x, f, where, 1.0, False, False, dtype), "rotary", rows)
    assert (out.float().cpu().numpy()[~live] == 7.0).all()
    assert (out[..., 2 * H * d:] == 7.0).all()
    made, _ = api.la_rotary_fwd(q, None, f, lengths=n.cuda())
    assert (made.cpu().transpose(1, 2)[torch.from_numpy(~live)] == 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_in_place_and_back(interleaved):
    q, k, f = rotary_inputs(2, 4, 4, 50, 64, 64, "f32", packed=False)
    q0, k0 = q.clone(), k.clone()
    want, _ = api.la_rotary_fwd(q, k, f, interleaved=interleaved)
    api.la_rotary_fwd(q, k, f, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, want)
    api.la_rotary_bwd(q, k, f, interleaved=interleaved, q_out=q, k_out=k)
    # two turns of at most 2^-21 each, of pairs no longer than the row's largest
    for a, b in ((q, q0), (k, k0)):
        assert (a - b).abs().max() <= 2.0 ** -19 * b.abs().max()


@pytest.mark.parametrize("pos", [0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31])
def test_rotary_angles_of_far_positions(pos):
    """The largest positions, with frequencies that are no short fractions of a turn."""
    f = torch.tensor([1.0, 0.3333333, 6.2831855, 100.25, 1e-30, 2.0 ** -126, 3e9, 0.0])
    x = torch.ones(1, 1, 1, 16, device="cuda")
    y, _ = api.la_rotary_fwd(x, None, f.cuda(), offsets=torch.tensor([pos], dtype=torch.int32).cuda())
    import math
    from fractions import Fraction
    # pi to 60 digits: the turns of pos * f as a fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    for i, w in enumerate(f.tolist()):
        turns = Fraction(pos) * Fraction(w) / (2 * pi)
        a = float((turns - math.floor(turns)) * 2 * pi)
        got = y[0, 0, 0, i].item(), y[0, 0, 0, i + 8].item()
        want = math.cos(a) - math.sin(a), math.sin(a) + math.cos(a)
        # pos * 2^-64 turns of the angle, sine and cosine to 2^-22, two sums
        tol = 2.0 ** -20 + abs(pos) * max(1.0, abs(w)) * 2.0 ** -60
        assert max(abs(p - q) for p, q in zip(got, want)) <= tol, (w, got, want)


def test_rotary_non_finite_inputs_stay_in_their_pairs():
    q, _, f = rotary_inputs(1, 2, 1, 6, 32, 16, "f32", packed=False)
    q[0, 0, 2, 3], q[0, 1, 4, 20] = NAN, INF
    y, _ = api.la_rotary_fwd(q, None, f)
    bad = ~torch.isfinite(y[0]).cpu()
    want = torch.zeros(2, 6, 32, dtype=torch.bool)
    want[0, 2, 3] = want[0, 2, 11] = want[1, 4, 20] = True
    assert torch.equal(bad, want)


def test_rotary_offsets_past_32_bits():
    """The last tokens of a tensor of more than 2^31 elements, and a stride that passes them."""
    L = (1 << 31) // 64 + 3
    x = torch.zeros(1, 1, L, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, -5:] = torch.randn(5, 64, generator=_gen(3)).bfloat16().cuda()
    f = api.la_rotary_frequencies(64)[0].cuda()
    y, _ = api.la_rotary_fwd(x, None, f)
    tail = x[:, :, -5:].contiguous()
    at = torch.tensor([L - 5], dtype=torch.int32).cuda()
    want, _ = api.la_rotary_fwd(tail, None, f, offsets=at)
    assert torch.equal(y[:, :, -5:], want)


# ---------------------------------------------------------------- norms
def gated_inputs(B, H, L, d, dtype, shared, bias, gate, head_major, seed=0):
    g = _gen(seed)
    dt = DT[dtype]
    x = torch.randn(B, H, L, d, generator=g).to(dt).cuda() if head_major else \
        torch.randn(B, L, H, d, generator=g).to(dt).cuda().permute(0, 2, 1, 3)
    z = torch.randn(B, L, H * d, generator=g).to(dt).cuda() if gate else None
    dy = torch.randn(B, L, H * d + 3, generator=g).to(dt).cuda()[..., 1:1 + H * d] if d % 2 else \
        torch.randn(B, L, H * d, generator=g).to(dt).cuda()
    n = d if shared else H * d
    w = (1 + 0.1 * torch.randn(n, generator=g)).cuda()
    b = torch.randn(n, generator=g).cuda() if bias else None
    return dy, x, z, w, b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm,activation,gate_first", [
    ("rms", "silu", False), ("layer", "silu", True), ("rms", "sigmoid", True),
    ("layer", "sigmoid", False), ("layer", "none", False)])
@pytest.mark.parametrize("B,H,L,d,shared,bias,gate,head_major", [
    (1, 1, 1, 1, True, False, True, True),
    (2, 3, 5, 64, True, True, True, True),
    (2, 3, 5, 64, False, True, True, False),
    (3, 2, 70, 16, True, False, True, True),
    (1, 4, 33, 128, False, False, True, True),
    (2, 2, 9, 80, True, True, False, True),
    (1, 2, 600, 256, True, True, True, False),
    (1, 1, 5, 520, True, True, True, True),     # a block to a row
    (2, 1, 3, 4096, True, False, True, True),
    (1, 1, 2, 16384, False, True, True, True),
    (2, 2, 4, 33, True, True, True, True),      # no vector divides the rows
    (1, 2, 3, 1001, False, True, True, False),
    (1, 1, 2, 9999, True, True, True, True),
])
def test_gated_norm_bwd(B, H, L, d, shared, bias, gate, head_major, norm, activation, gate_first,
                        dtype):
    dy, x, z, w, b = gated_inputs(B, H, L, d, dtype, shared, bias, gate, head_major)
    got = api.la_gated_norm_bwd(dy, x, z, w, b, norm=norm, activation=activation,
                                gate_first=gate_first)
    ref = T.gated_norm_back(dy, x, z, w, b, norm, activation, gate_first, 1e-5, dtype)
    _compare(dict(zip(("dx", "dgate", "dweight", "dbias"), got)), ref)
    assert (got[1] is None) == (z is None) and (got[3] is None) == (b is None)


def test_gated_norm_bwd_in_place_slices_and_optional_outputs():
    dy, x, z, w, b = gated_inputs(2, 4, 40, 64, "bf16", True, True, True, True)
    want = api.la_gated_norm_bwd(dy, x, z, w, b)
    dx, dz, dw, db = api.la_gated_norm_bwd(dy, x, z, w, b, want_param_grads=False)
    assert dw is None and db is None and torch.equal(dx, want[0]) and torch.equal(dz, want[1])
    wide = torch.full((2, 40, 3 * 256), 7.0, dtype=torch.bfloat16, device="cuda")
    token_major = wide[..., 256:512].unflatten(-1, (4, 64)).permute(0, 2, 1, 3)
    api.la_gated_norm_bwd(dy, x, z, w, b, dx=token_major, dgate=wide[..., :256])
    assert torch.equal(token_major, want[0]) and torch.equal(wide[..., :256], want[1])
    assert (wide[..., 512:] == 7.0).all()
    x2, z2, dy2 = x.clone(), z.clone(), dy.clone()
    got = api.la_gated_norm_bwd(dy, x2, z2, w, b, dx=x2, dgate=z2)
    assert got[0] is x2 and all(torch.equal(a, c) for a, c in zip(got, want))
    got = api.la_gated_norm_bwd(dy2, x, z, w, b, dgate=dy2)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    with pytest.raises(api.LAError):
        api.la_gated_norm_bwd(dy, x, z, w, b, dx=z.view(2, 4, 40, 64))


@pytest.mark.parametrize("heads", [1, 5])
def test_gated_norm_bwd_many_rows(heads):
    """More rows than the card holds teams: several rows to each, partial last rounds."""
    dy, x, z, w, b = gated_inputs(3, 5, 4111, 64, "f32", heads == 1, True, True, True)
    got = api.la_gated_norm_bwd(dy, x, z, w, b)
    ref = T.gated_norm_back(dy, x, z, w, b, "rms", "silu", False, 1e-5, "f32")
    _compare(dict(zip(("dx", "dgate", "dweight", "dbias"), got)), ref)


def test_gated_norm_bwd_empty_and_zero_rows():
    w, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    x = torch.zeros(2, 3, 0, 64, device="cuda")
    z = torch.zeros(2, 0, 192, device="cuda")
    dx, dz, dw, db = api.la_gated_norm_bwd(z, x, z, w, b)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()
    # rows of zeros: the norm is flat there, and its gradient finite
    dy, x, z, w, b = gated_inputs(1, 2, 3, 64, "f32", True, True, True, True)
    x[0, 0, 1] = 0
    got = api.la_gated_norm_bwd(dy, x, z, w, b)
    ref = T.gated_norm_back(dy, x, z, w, b, "rms", "silu", False, 1e-5, "f32")
    _compare(dict(zip(("dx", "dgate", "dweight", "dbias"), got)), ref)


def resid_inputs(rows, D, dtype, res_dtype, post, scaled, dr=True, seed=0):
    g = _gen(seed)
    dt, rd = DT[dtype], DT[res_dtype]
    r = (2 * torch.randn(rows, D, generator=g) + 0.25).to(rd).cuda()
    dy, x = (torch.randn(rows, D, generator=g).to(dt).cuda() for _ in range(2))
    drr = torch.randn(rows, D, generator=g).to(rd).cuda() if dr else None
    w, p, s = ((1 + 0.1 * torch.randn(D, generator=g)).cuda() for _ in range(3))
    return dy, r, drr, x, w, p if post else None, s if scaled else None


NAMES = ("dx", "dresidual", "dweight", "dbias", "dpost_weight", "dscale")


@pytest.mark.parametrize("dtype,res_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("rows,D,post,scaled,dr", [
    (1, 1, True, True, True), (3, 64, False, False, True), (5, 64, True, True, False),
    (70, 16, True, False, True), (33, 128, False, True, True), (9, 512, True, True, True),
    (4, 1024, False, False, False), (3, 4096, True, True, True), (2, 16384, True, True, True),
    (7, 33, True, True, True), (5, 619, True, False, True), (3, 3723, False, True, True),
    (1000, 200, True, True, True), (2, 10001, True, True, True),
])
def test_residual_norm_bwd(rows, D, post, scaled, dr, norm, dtype, res_dtype):
    dy, r, drr, x, w, p, s = resid_inputs(rows, D, dtype, res_dtype, post, scaled, dr)
    got = api.la_residual_norm_bwd(dy, r, w, dr=drr, x=x, post_weight=p, scale=s, alpha=0.75,
                                   norm=norm, want_dbias=True)
    ref = T.residual_norm_back(dy, r, w, drr, x, p, s, 0.75, norm, 1e-5, dtype, res_dtype)
    _compare(dict(zip(NAMES, got)), ref)
    assert (got[4] is None) == (not post) and (got[5] is None) == (not scaled)


def test_residual_norm_bwd_in_place_and_optional_outputs():
    dy, r, dr, x, w, p, s = resid_inputs(300, 256, "bf16", "f32", True, True)
    want = api.la_residual_norm_bwd(dy, r, w, dr=dr, x=x, post_weight=p, scale=s)
    some = api.la_residual_norm_bwd(dy, r, w, dr=dr, x=x, post_weight=p, scale=s,
                                    want_dresidual=False, want_param_grads=False)
    assert some[1:] == (None,) * 5 and torch.equal(some[0], want[0])
    for same in (dy, x):  # dx over dy, and over x
        dy2, x2, dr2 = dy.clone(), x.clone(), dr.clone()
        got = api.la_residual_norm_bwd(dy2, r, w, dr=dr2, x=x2, post_weight=p, scale=s,
                                       dx=dy2 if same is dy else x2, dresidual=dr2)
        assert all(torch.equal(a, b) for a, b in zip(got, want) if b is not None)
    with pytest.raises(api.LAError):
        api.la_residual_norm_bwd(dy, r, w, dr=dr, x=x, post_weight=p, scale=s, dresidual=r)
    with pytest.raises(api.LAError):  # a post norm needs x
        api.la_residual_norm_bwd(dy, r, w, post_weight=p)


def test_residual_norm_bwd_misaligned_and_empty():
    """Tensors that start off a 16-byte boundary, and no rows."""
    dy, r, dr, x, w, p, s = resid_inputs(20, 64, "bf16", "f32", True, True)
    want = api.la_residual_norm_bwd(dy, r, w, dr=dr, x=x, post_weight=p, scale=s, want_dbias=True)
    off = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    got = api.la_residual_norm_bwd(off(dy), off(r), w, dr=off(dr), x=off(x), post_weight=p, scale=s,
                                   want_dbias=True)
    ref = T.residual_norm_back(dy, r, w, dr, x, p, s, 1.0, "rms", 1e-5, "bf16", "f32")
    _compare(dict(zip(NAMES, got)), ref)
    _compare(dict(zip(NAMES, want)), ref)
    e = torch.zeros(0, 64, device="cuda")
    got = api.la_residual_norm_bwd(e, e, torch.ones(64, device="cuda"), want_dbias=True)
    assert got[0].shape == (0, 64) and (got[2] == 0).all() and (got[3] == 0).all()


# ---------------------------------------------------------------- attention
def attn_inputs(B, H, L, dk, dv, dtype, phi, kind, states, seed=0):
    g = _gen(seed)
    unit = 1.0 if phi == "elu1" else dk ** -0.5
    dt = DT[dtype]
    q, k = ((unit * torch.randn(B, H, L, dk, generator=g)).to(dt).cuda() for _ in range(2))
    v, dO = (torch.randn(B, H, L, dv, generator=g).to(dt).cuda() for _ in range(2))
    decay = {"none": lambda: None, "head": lambda: -0.2 * torch.rand(H, generator=g),
             "token": lambda: -0.3 * torch.rand(B, H, L, generator=g),
             "logit": lambda: torch.randn(B, H, L, generator=g)}[kind]()
    decay = None if decay is None else decay.cuda()
    S0, dSf = (0.3 * torch.randn(B, H, dk, dv, generator=g).cuda() if states else None
               for _ in range(2))
    return q, k, v, dO, decay, S0, dSf


ATTN = ("dq", "dk", "dv", "ddecay", "dS0")


def check_attn(B, H, L, dk, dv, dtype, phi, kind, states, seed=0, edit=None, **kw):
    q, k, v, dO, decay, S0, dSf = attn_inputs(B, H, L, dk, dv, dtype, phi, kind, states, seed)
    if edit is not None:
        edit(q, k, v, dO, decay)
    api.la_set_feature_map(phi)
    got = api.la_chunk_bwd(q, k, v, dO, decay_kind=kind, decay=decay, S0=S0, dS_final=dSf, **kw)
    api.la_device_status()
    ref = T.chunk_back(q, k, v, dO, phi, kind, decay, S0, dSf, dtype,
                       want_f32=got[3] is not None or got[4] is not None)
    _compare(dict(zip(ATTN, got)), ref)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("phi", ["identity", "elu1"])
@pytest.mark.parametrize("kind", ["none", "head", "token", "logit"])
@pytest.mark.parametrize("L", [1, 2, 31, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_bwd_square_heads(d, L, kind, phi, dtype):
    check_attn(1, 2, L, d, d, dtype, phi, kind, states=L % 2 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (32, 64), (64, 32), (128, 64), (64, 128)])
@pytest.mark.parametrize("kind", ["none", "logit"])
@pytest.mark.parametrize("phi", ["identity", "elu1"])
def test_chunk_bwd_other_heads(dk, dv, kind, phi, dtype):
    check_attn(2, 2, 77, dk, dv, dtype, phi, kind, states=True)
    check_attn(2, 1, 161, dk, dv, dtype, phi, kind, states=False)


@pytest.mark.parametrize("phi", ["identity", "elu1"])
@pytest.mark.parametrize("kind", ["none", "head", "token"])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_bwd_bf16_without_f32_outputs(d, kind, phi):
    """dq, dk and dv alone: the states enter the products as one bf16 plane."""
    got = check_attn(1, 3, 290, d, d, "bf16", phi, kind, True, want_decay_grad=False,
                     want_state_grad=False)
    assert got[3] is None and got[4] is None


@pytest.mark.parametrize("dtype,d,L", [("bf16", 64, 3000), ("bf16", 128, 1500), ("f32", 64, 900),
                                       ("f32", 32, 2000)])
@pytest.mark.parametrize("kind", ["head", "logit"])
def test_chunk_bwd_in_segments(kind, dtype, d, L):
    """One long sequence, cut into many segments."""
    check_attn(1, 1, L, d, d, dtype, "identity", kind, True)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 32), ("f32", 64)])
@pytest.mark.parametrize("what", ["strong", "mixed", "ends", "none"])
def test_chunk_bwd_extreme_decays(what, dtype, d):
    """Decays of e^-3 a token (past the factors of a block), sudden resets among slow tokens, decays of
    zero (a log of minus infinity, the type's lowest value), and logs of zero."""
    def edit(q, k, v, dO, decay):
        if what == "strong":
            decay.fill_(-3.0)
        elif what == "mixed":
            decay.fill_(-0.001)
            decay[:, :, ::7] = -30.0
        elif what == "ends":
            decay.fill_(-0.05)
            decay[:, :, 5] = -INF
            decay[:, :, 64] = torch.finfo(torch.float32).min
            decay[:, :, 100] = -1000.0
        else:
            decay.zero_()
    # the reference's exp of the same logs: below -200 a decay is zero in either
    check_attn(1, 2, 150, d, d, dtype, "identity", "token", True, edit=edit)


@pytest.mark.parametrize("d", [32, 64])
def test_chunk_bwd_gate_logits_at_the_ends(d):
    def edit(q, k, v, dO, decay):
        decay[:, :, 3], decay[:, :, 40], decay[:, :, 90] = 1e30, -1e30, 90.0
        decay[:, :, 91], decay[:, :, 92] = -90.0, 0.0
    check_attn(1, 2, 140, d, d, "bf16", "identity", "logit", True, edit=edit)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("bf16", 32), ("f32", 64)])
def test_chunk_bwd_non_finite_inputs_stay_in_their_sequence(dtype, d):
    q, k, v, dO, decay, S0, dSf = attn_inputs(2, 3, 200, d, d, dtype, "identity", "token", True)
    clean = api.la_chunk_bwd(q, k, v, dO, decay_kind="token", decay=decay, S0=S0, dS_final=dSf)
    q[0, 1, 150, 3], v[1, 2, 10, 0], dO[1, 2, 190, 5] = NAN, INF, -INF
    got = api.la_chunk_bwd(q, k, v, dO, decay_kind="token", decay=decay, S0=S0, dS_final=dSf)
    for a, b in zip(got, clean):
        for at in ((0, 0), (0, 2), (1, 0), (1, 1)):
            assert torch.equal(a[at], b[at])
    # behind the last token that a NaN in q reaches, dk and dv are as before: G runs backward
    assert torch.isnan(got[1][0, 1, 100].float()).any()
    assert torch.equal(got[2][0, 1, 151:], clean[2][0, 1, 151:])


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("bf16", 16)])
def test_chunk_bwd_pieces_chained_are_the_whole(dtype, d):
    """A sequence in two pieces, back to front, each handing its dS0 on."""
    q, k, v, dO, decay, S0, dSf = attn_inputs(1, 2, 256, d, d, dtype, "identity", "logit", True)
    whole = api.la_chunk_bwd(q, k, v, dO, decay_kind="logit", decay=decay, S0=S0, dS_final=dSf)
    cut = lambda t, s: t[:, :, s].contiguous()  # noqa: E731
    first, second = slice(0, 100), slice(100, 256)
    _, S1 = api.la_chunk_fwd(*(cut(t.float(), first) for t in (q, k, v)), 64, "logit",
                             cut(decay, first), S0)
    back = api.la_chunk_bwd(*(cut(t, second) for t in (q, k, v, dO)), decay_kind="logit",
                            decay=cut(decay, second), S0=S1, dS_final=dSf)
    front = api.la_chunk_bwd(*(cut(t, first) for t in (q, k, v, dO)), decay_kind="logit",
                             decay=cut(decay, first), S0=S0, dS_final=back[4])
    ref = T.chunk_back(q, k, v, dO, "identity", "logit", decay, S0, dSf, dtype)
    joined = [torch.cat([a, b], 2) for a, b in zip(front[:4], back[:4])] + [front[4]]
    _compare(dict(zip(ATTN, joined)), ref)
    _compare(dict(zip(ATTN, whole)), ref)


def test_chunk_bwd_empty():
    q = torch.zeros(2, 3, 0, 64, device="cuda")
    dSf = torch.randn(2, 3, 64, 64, generator=_gen(0)).cuda()
    d = torch.zeros(3, device="cuda")
    got = api.la_chunk_bwd(q, q, q, q, decay_kind="head", decay=d, dS_final=dSf, want_state_grad=True)
    assert torch.equal(got[4], dSf) and (got[3] == 0).all() and got[0].shape == q.shape
    got = api.la_chunk_bwd(q, q, q, q, want_state_grad=True)
    assert (got[4] == 0).all()
    e = torch.zeros(0, 3, 5, 64, device="cuda")
    assert api.la_chunk_bwd(e, e, e, e)[0].shape == e.shape


@pytest.mark.parametrize("chunk", [1, 16, 64])
def test_chunk_bwd_does_not_depend_on_chunk(chunk):
    q, k, v, dO, decay, *_ = attn_inputs(1, 2, 200, 64, 64, "bf16", "identity", "token", False)
    want = api.la_chunk_bwd(q, k, v, dO, decay_kind="token", decay=decay)
    got = api.la_chunk_bwd(q, k, v, dO, chunk=chunk, decay_kind="token", decay=decay)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], want[:4]))


def test_chunk_bwd_many_sequences():
    """More sequences than a grid's y axis holds, one token each; and of 32768 the last ones."""
    B, H, d = 1, 70000, 16
    q, k, v, dO, decay, S0, dSf = attn_inputs(B, H, 2, d, d, "f32", "identity", "token", True)
    got = api.la_chunk_bwd(q, k, v, dO, decay_kind="token", decay=decay, S0=S0, dS_final=dSf)
    api.la_device_status()
    at = slice(69990, 70000)
    ref = T.chunk_back(*(t[:, at] for t in (q, k, v, dO)), "identity", "token", decay[:, at],
                       S0[:, at], dSf[:, at], "f32")
    _compare({n: g[:, at] for n, g in zip(ATTN, got)}, ref)


def test_chunk_bwd_repeats_its_bits_whatever_the_workspace_holds():
    q, k, v, dO, decay, S0, dSf = attn_inputs(1, 4, 2000, 128, 128, "bf16", "identity", "logit", True)
    args = dict(decay_kind="logit", decay=decay, S0=S0, dS_final=dSf)
    want = api.la_chunk_bwd(q, k, v, dO, **args)
    need = api.la_chunk_bwd_workspace_bytes(1, 4, 2000, 128, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaNs
    guard = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    got = api.la_chunk_bwd(q, k, v, dO, workspace=ws, **args)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    api.la_chunk_bwd(q, k, v, dO, workspace=guard[:need], **args)
    assert (guard[need:] == 255).all()


# ---------------------------------------------------------------- streams, threads, graphs
def _calls():
    q, k, v, dO, decay, S0, dSf = attn_inputs(1, 4, 1024, 64, 64, "bf16", "identity", "logit", True)
    dy, x, z, w, b = gated_inputs(1, 4, 1024, 64, "bf16", True, True, True, True)
    rdy, r, dr, rx, rw, p, s = resid_inputs(1024, 256, "bf16", "f32", True, True)
    rq, rk, f = rotary_inputs(1, 4, 4, 1024, 64, 64, "bf16")
    return {
        "la_chunk_bwd": lambda **kw: api.la_chunk_bwd(q, k, v, dO, decay_kind="logit", decay=decay,
                                                      S0=S0, dS_final=dSf, **kw),
        "la_gated_norm_bwd": lambda **kw: api.la_gated_norm_bwd(dy, x, z, w, b, **kw),
        "la_residual_norm_bwd": lambda **kw: api.la_residual_norm_bwd(
            rdy, r, rw, dr=dr, x=rx, post_weight=p, scale=s, want_dbias=True, **kw),
        "la_rotary_fwd": lambda **kw: api.la_rotary_fwd(rq, rk, f, **kw),
        "la_rotary_bwd": lambda **kw: api.la_rotary_bwd(rq, rk, f, **kw),
    }


NAMED = ["la_chunk_bwd", "la_gated_norm_bwd", "la_residual_norm_bwd", "la_rotary_fwd",
         "la_rotary_bwd"]


@pytest.mark.parametrize("name", NAMED)
def test_another_stream_and_two_graphs(name):
    """On a stream that is not the current one; captured twice, replayed side by side with eager
    calls in between."""
    call = _calls()[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    runs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        runs.append((graph, out, torch.cuda.Stream()))
    for _ in range(3):
        for graph, _, stream in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        call()
    torch.cuda.synchronize()
    for _, out, _ in runs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("name", ["la_chunk_bwd", "la_gated_norm_bwd", "la_residual_norm_bwd"])
def test_two_threads_on_one_stream(name, monkeypatch):
    call = _calls()[name]
    want = call()
    got = run_together(monkeypatch, name, -3, [call, call])
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


# ---------------------------------------------------------------- together
def _layer(qkv, gate, logits, S0, wn, res, wr, f):
    """A linear attention layer on 64-bit leaves: rotary positions, gated attention, norm and gate
    per head, the residual step with the next norm.  [B,L,3*H*d] -> y, r, S."""
    B, L, width = qkv.shape
    H, d = logits.shape[1], wn.numel()
    q, k, v = (t.unflatten(-1, (H, d)).transpose(1, 2) for t in qkv.split(H * d, -1))
    a = torch.arange(L).double()[:, None] * f.double()
    c, s = torch.cos(a), torch.sin(a)

    def turned(x):
        p, r = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([p * c - r * s, p * s + r * c], -1)

    q, k = turned(q), turned(k)
    S, O = S0, []
    for t in range(L):
        S = torch.sigmoid(-logits[:, :, t])[..., None, None] * S + k[:, :, t, :, None] * v[:, :, t, None]
        O.append((q[:, :, t, :, None] * S).sum(-2))
    O = torch.stack(O, 2).transpose(1, 2)
    n = O / torch.sqrt((O * O).mean(-1, keepdim=True) + 1e-5) * wn
    u = n.flatten(2) * torch.nn.functional.silu(gate)
    r = res + u
    m = r - r.mean(-1, keepdim=True)
    return m / torch.sqrt((m * m).mean(-1, keepdim=True) + 1e-5) * wr, r, S


def test_a_layers_training_pass():
    """Forward and backward through the library's calls, fp32, against autograd in 64 bits.  Every
    call's own error is below 2^-16 of its result's size (their tests' bounds at these sizes); six
    follow one another, each passing the errors on by factors of order one: 2^-12 of a gradient's
    norm."""
    B, H, L, d = 2, 3, 150, 64
    g = _gen(9)
    rand = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
    qkv, gate, res = 0.5 * rand(B, L, 3 * H * d), rand(B, L, H * d), rand(B, L, H * d)
    logits, S0 = rand(B, H, L), 0.1 * rand(B, H, d, d)
    wn, wr = 1 + 0.1 * rand(d), 1 + 0.1 * rand(H * d)
    dy, dr, dSf = rand(B, L, H * d), rand(B, L, H * d), 0.1 * rand(B, H, d, d)
    f, _ = api.la_rotary_frequencies(d)
    names = ("qkv", "gate", "logits", "S0", "wn", "res", "wr")
    leaves = [t.double().requires_grad_(True) for t in (qkv, gate, logits, S0, wn, res, wr)]
    y, r, S = _layer(*leaves[:4], leaves[4], *leaves[5:], f)
    want = dict(zip(names, torch.autograd.grad((y, r, S), leaves,
                                               (dy.double(), dr.double(), dSf.double()))))

    qkv, gate, res, logits, S0, wn, wr, dy, dr, dSf, f = (
        t.cuda() for t in (qkv, gate, res, logits, S0, wn, wr, dy, dr, dSf, f))
    q, k, v = (t.unflatten(-1, (H, d)).transpose(1, 2) for t in qkv.split(H * d, -1))
    q, k = api.la_rotary_fwd(q, k, f)
    v = v.contiguous()
    O, _ = api.la_chunk_fwd(q, k, v, 64, "logit", logits, S0)
    u = api.la_gated_norm_fwd(O, gate, wn)
    y2, r2 = api.la_residual_norm_fwd(u, res, wr, norm="layer")
    near = lambda a, b: ((a.cpu().double() - b).norm() / b.norm()).item() < 2.0 ** -12  # noqa: E731
    assert near(y2, y.detach()) and near(r2, r.detach())

    got = {}
    du, got["res"], got["wr"], *_ = api.la_residual_norm_bwd(dy, r2, wr, dr=dr, norm="layer")
    dO, got["gate"], got["wn"], _ = api.la_gated_norm_bwd(du, O, gate, wn)
    dq, dk, dv, got["logits"], got["S0"] = api.la_chunk_bwd(
        q, k, v, dO, decay_kind="logit", decay=logits, S0=S0, dS_final=dSf)
    dqkv = torch.empty_like(qkv)
    views = [t.unflatten(-1, (H, d)).transpose(1, 2) for t in dqkv.split(H * d, -1)]
    api.la_rotary_bwd(dq, dk, f, q_out=views[0], k_out=views[1])
    views[2].copy_(dv)
    got["qkv"] = dqkv
    for name in names:
        assert near(got[name], want[name]), name
