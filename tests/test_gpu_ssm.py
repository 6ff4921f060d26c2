"""The state space block's operators on the GPU, element by element against the
64-bit references and their bounds, and run together as a block.  Needs a GB300."""
import numpy as np
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api
from causal_linear_attention_chunkwise_gb300 import workloads as W
from tests import ssm_reference as R
from tests.gpu_helpers import to_dev

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rows(g, B, L, D, dtype, packed):
    """[B,L,D] on the GPU: its own tensor, or the middle of rows 2D + 3 wide."""
    if packed:
        return torch.randn(B, L, 2 * D + 3, generator=g).to(DT[dtype]).cuda()[..., 2:2 + D]
    return torch.randn(B, L, D, generator=g).to(DT[dtype]).cuda()


def _lengths(B, L):
    """One empty sequence, one of a token, one full, one past L, one below 0."""
    return torch.tensor([0, 1, L, L + 5, -2, max(L - 3, 0)][:B], dtype=torch.int32).cuda()


def _live(lengths, B, L):
    if lengths is None:
        return np.ones((B, L), bool)
    return np.arange(L)[None] < np.clip(lengths.cpu().numpy(), 0, L)[:, None]


def _poison(t, live):
    """NaN in the rows that no sequence owns."""
    t = t.clone() if t.is_contiguous() else t
    t[torch.from_numpy(~live).cuda()] = NAN
    return t


# ---------------------------------------------------------------- convolution
def conv_inputs(B, L, D, Wd, dtype, packed=False, state=True, ragged=False, seed=0):
    g = _gen(seed)
    x = _rows(g, B, L, D, dtype, packed)
    weight, bias = torch.randn(D, Wd, generator=g).cuda(), torch.randn(D, generator=g).cuda()
    st = torch.randn(B, Wd - 1, D, generator=g).to(DT[dtype]).cuda() if state else None
    n = _lengths(B, L) if ragged else None
    if ragged:
        x = _poison(x, _live(n, B, L))
    return x, weight, bias, st, n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,D,Wd,act,packed,state,ragged", [
    (1, 1, 1, 2, "silu", False, False, False),
    (3, 1, 64, 4, "silu", False, True, False),
    (2, 2, 72, 4, "none", False, True, False),     # fewer tokens than the state has rows
    (2, 3, 40, 8, "silu", True, True, False),
    (2, 100, 256, 4, "silu", False, False, False),
    (6, 67, 48, 3, "silu", False, True, True),
    (6, 33, 51, 4, "none", True, True, True),       # no vector divides D
    (6, 5, 136, 5, "silu", True, False, True),
    (1, 1100, 520, 2, "silu", False, True, False),
    (2, 300, 24, 6, "silu", False, True, False),
    (2, 129, 33, 7, "silu", False, True, False),
    (3, 50, 30, 4, "silu", False, True, False),      # pairs of channels, not fours
    (2, 4100, 1024, 4, "silu", True, True, False),   # runs of several batches of tokens
    (5, 1500, 516, 3, "silu", False, True, True),
])
def test_conv(B, L, D, Wd, act, packed, state, ragged, dtype):
    x, weight, bias, st, n = conv_inputs(B, L, D, Wd, dtype, packed, state, ragged)
    y = torch.full((B, L, D), 7.0, dtype=x.dtype, device="cuda")
    y, sf = api.la_causal_conv_fwd(x, weight, bias, activation=act, state0=st, lengths=n, y=y)
    ref, last = R.causal_conv(x, weight, bias, act, st, n, dtype)
    live = _live(n, B, L)
    R.check(y, ref, "y", live)
    assert (y.float().cpu().numpy()[~live] == 7.0).all()  # rows behind a length stay as they were
    assert np.array_equal(R.f64(sf), last)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_token_by_token_in_place_is_the_prompt(dtype):
    B, L, D, Wd = 3, 9, 72, 4
    x, weight, bias, st, _ = conv_inputs(B, L, D, Wd, dtype)
    y, sf = api.la_causal_conv_fwd(x, weight, bias, state0=st)
    s = st.clone()
    steps = [api.la_causal_conv_fwd(x[:, t:t + 1].contiguous(), weight, bias, state0=s,
                                    state_final=s)[0] for t in range(L)]
    assert torch.equal(torch.cat(steps, 1), y)
    assert torch.equal(s, sf)


def test_conv_state_in_place_over_a_prompt():
    x, weight, bias, st, _ = conv_inputs(2, 200, 64, 4, "bf16")
    y, sf = api.la_causal_conv_fwd(x, weight, bias, state0=st)
    y2, sf2 = api.la_causal_conv_fwd(x, weight, bias, state0=st, state_final=st)
    assert sf2 is st and torch.equal(sf2, sf) and torch.equal(y2, y)


def test_conv_non_finite_inputs_stay_in_their_windows():
    x, weight, bias, st, _ = conv_inputs(1, 40, 16, 4, "f32", state=False)
    x[0, 10, 3], x[0, 20, 4], x[0, 30, 5] = NAN, float("inf"), -float("inf")
    y, _ = api.la_causal_conv_fwd(x, weight, bias, activation="none")
    bad = ~torch.isfinite(y[0]).cpu()
    want = torch.zeros(40, 16, dtype=torch.bool)
    want[10:14, 3] = want[20:24, 4] = want[30:34, 5] = True
    assert torch.equal(bad, want)


def test_conv_empty():
    x, weight, bias, st, _ = conv_inputs(2, 0, 16, 4, "bf16")
    y, sf = api.la_causal_conv_fwd(x, weight, bias, state0=st)
    assert y.shape == (2, 0, 16) and torch.equal(sf, st)
    _, sf = api.la_causal_conv_fwd(x, weight, bias)
    assert (sf == 0).all()


# ---------------------------------------------------------------- selective scan
def scan_inputs(B, L, ch, N, G, dtype, packed=False, gate=True, state=True, ragged=False,
                seed=0, skip=True):
    g = _gen(seed)
    i = dict(x=_rows(g, B, L, ch, dtype, packed), dt=_rows(g, B, L, ch, dtype, packed),
             z=_rows(g, B, L, ch, dtype, packed) if gate else None)
    bc = torch.randn(B, L, 2, G, N, generator=g).to(DT[dtype]).cuda()
    i["Bm"], i["Cm"] = bc[:, :, 0], bc[:, :, 1]
    if G == 1 and not packed:
        i["Bm"], i["Cm"] = (t[:, :, 0].contiguous() for t in (i["Bm"], i["Cm"]))
    i["A"] = -(torch.arange(1, N + 1) * (0.5 + torch.rand(ch, N, generator=g))).cuda()
    step = torch.exp(np.log(1e-3) + torch.rand(ch, generator=g) * np.log(100.0))
    i["dt_bias"] = (step + torch.log(-torch.expm1(-step))).cuda()
    i["D"] = torch.randn(ch, generator=g).cuda() if skip else None
    i["h0"] = torch.randn(B, ch, N, generator=g).cuda() if state else None
    i["lengths"] = _lengths(B, L) if ragged else None
    if ragged:
        live = _live(i["lengths"], B, L)
        for k in ("x", "dt", "z", "Bm", "Cm"):
            if i[k] is not None:
                i[k] = _poison(i[k], live)
    return i


def scan(i, **kw):
    a = dict(i)
    return api.la_selective_scan_fwd(a.pop("x"), a.pop("dt"), a.pop("A"), a.pop("Bm"),
                                     a.pop("Cm"), **a, **kw)


def scan_reference(i, dtype, softplus=True):
    return R.selective_scan(softplus=softplus, dtype=dtype, **i)


SCANS = [  # B, L, ch, N, G, packed, gate, state, ragged
    (1, 1, 1, 1, 1, False, False, False, False),
    (4, 1, 96, 16, 1, True, True, True, False),
    (3, 1, 70, 24, 2, False, True, True, False),
    (6, 1, 33, 16, 1, False, True, True, True),
    (2, 2, 64, 16, 1, False, True, True, False),
    (2, 31, 40, 4, 1, False, True, False, False),
    (2, 65, 34, 7, 2, True, True, True, False),
    (1, 130, 100, 16, 1, True, False, True, False),
    (2, 100, 30, 17, 1, False, True, True, False),
    (2, 64, 20, 33, 2, True, True, False, False),
    (1, 70, 9, 64, 1, False, True, True, False),
    (1, 40, 12, 100, 3, False, False, True, False),
    (1, 33, 5, 128, 1, True, True, True, False),
    (1, 20, 3, 256, 1, False, True, True, False),
    (1, 20, 3, 129, 1, False, True, True, False),
    (6, 67, 24, 16, 2, False, True, True, True),
    (6, 200, 51, 16, 1, True, True, True, True),
    (6, 37, 18, 24, 1, True, False, False, True),
    (1, 1500, 64, 16, 1, True, True, True, False),  # long enough for several segments
    (6, 900, 24, 16, 1, True, True, True, True),
    (1, 1111, 40, 24, 2, False, True, True, False),
    (1, 700, 6, 128, 1, False, True, True, False),
    (2, 65, 34, 6, 1, False, True, True, False),     # bf16 rows aligned to 4 bytes only
    (1, 300, 70, 10, 1, False, True, True, False),
    (130, 1, 1300, 16, 1, False, True, True, False),  # several sequences to a thread
    (131, 3, 650, 16, 2, True, True, True, False),
    (301, 1, 1030, 7, 1, False, True, True, False),
    (70, 2, 300, 128, 1, False, True, False, False),
    (600, 1, 520, 3, 1, False, False, True, False),
    (6, 8, 7000, 16, 1, False, True, True, True),
    (9, 9, 24, 16, 1, False, True, True, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ch,N,L", [(70, 13, 50), (70, 3, 1200), (5, 20, 33), (130, 16, 20)])
def test_scan_aligned_rows_of_uneven_width(ch, N, L, dtype):
    """Rows that start on 16-byte boundaries although no vector divides the width or N."""
    i = scan_inputs(2, L, ch, N, 1, dtype)
    for k in ("x", "dt", "z", "Bm", "Cm"):
        v = i[k]
        wide = torch.full((2, L, (v.shape[-1] + 15) // 8 * 8), NAN, dtype=v.dtype, device="cuda")
        wide[..., :v.shape[-1]] = v
        i[k] = wide[..., :v.shape[-1]]
    wide = torch.full((2, L, (ch + 15) // 8 * 8), 5.0, dtype=DT[dtype], device="cuda")
    y, h = scan(i, y=wide[..., :ch])
    ref, href = scan_reference(i, dtype)
    R.check(y, ref, "y")
    R.check(h, href, "h_final")
    assert (wide[..., ch:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,ch,N,G,packed,gate,state,ragged", SCANS)
def test_scan(B, L, ch, N, G, packed, gate, state, ragged, dtype):
    i = scan_inputs(B, L, ch, N, G, dtype, packed, gate, state, ragged)
    y = torch.full((B, L, ch), 7.0, dtype=DT[dtype], device="cuda")
    y, h = scan(i, y=y)
    ref, href = scan_reference(i, dtype)
    live = _live(i["lengths"], B, L)
    R.check(y, ref, "y", live)
    assert (y.float().cpu().numpy()[~live] == 7.0).all()
    R.check(h, href, "h_final")


def test_scan_many_sequences_with_lengths_and_states_in_place():
    B, L, ch, N = 140, 4, 1200, 16
    i = scan_inputs(B, L, ch, N, 1, "bf16")
    i["lengths"] = (torch.arange(B, dtype=torch.int32) % (L + 1)).cuda()
    live = _live(i["lengths"], B, L)
    for k in ("x", "dt", "z", "Bm", "Cm"):
        i[k] = _poison(i[k], live)
    ref, href = scan_reference(i, "bf16")
    h = i["h0"].clone()
    y = torch.full((B, L, ch), 7.0, dtype=torch.bfloat16, device="cuda")
    scan(dict(i, h0=h), y=y, h_final=h)
    R.check(y, ref, "y", live)
    assert (y.float().cpu().numpy()[~live] == 7.0).all()
    R.check(h, href, "h_final")


@pytest.mark.parametrize("segments", [True, False])
def test_scan_state_in_place_and_without_segments(segments):
    i = scan_inputs(2, 800, 48, 16, 1, "f32")
    y, h = scan(i)
    h0 = i["h0"].clone()
    y2, h2 = scan(dict(i, h0=h0), h_final=h0, segments=segments)
    ref, href = scan_reference(i, "f32")
    assert h2 is h0
    R.check(y2, ref, "y")
    R.check(h2, href, "h_final")
    if segments:
        assert torch.equal(y2, y) and torch.equal(h2, h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_token_by_token_in_place(dtype):
    B, L, ch, N = 3, 20, 70, 16
    i = scan_inputs(B, L, ch, N, 1, dtype)
    (ref, tol), (href, htol) = scan_reference(i, dtype)
    h = i["h0"].clone()
    outs = []
    for t in range(L):
        s = {k: (v[:, t:t + 1].contiguous() if k in ("x", "dt", "z", "Bm", "Cm") else v)
             for k, v in i.items()}
        outs.append(scan(dict(s, h0=h), h_final=h)[0])
    R.check(torch.cat(outs, 1), (ref, tol), "y")
    R.check(h, (href, htol), "h_final")


def test_scan_resumes():
    i = scan_inputs(2, 300, 64, 16, 1, "f32")
    cut = 113
    part = lambda a, b: {k: (v[:, a:b].contiguous() if k in ("x", "dt", "z", "Bm", "Cm") else v)  # noqa: E731
                         for k, v in i.items()}
    y1, h = scan(part(0, cut))
    y2, h = scan(dict(part(cut, 300), h0=h))
    ref, href = scan_reference(i, "f32")
    R.check(torch.cat([y1, y2], 1), ref, "y")
    R.check(h, href, "h_final")


@pytest.mark.parametrize("L", [1, 6, 500])
def test_scan_plain_steps(L):
    """No softplus, no bias, no skip, no gate, no state; a step of zero keeps the state, a
    negative step and a growing state are as the formula has them."""
    i = scan_inputs(2, L, 40, 16, 1, "f32", gate=False, state=False, skip=False)
    i["dt_bias"] = None
    i["dt"] = 0.01 * i["dt"]
    i["dt"][:, ::3] = 0
    i["A"][::2] = 0.1 * i["A"][::2].abs()
    y, h = scan(i, dt_softplus=False)
    ref, href = scan_reference(i, "f32", softplus=False)
    R.check(y, ref, "y")
    R.check(h, href, "h_final")


@pytest.mark.parametrize("L", [3, 600])
def test_scan_extreme_steps(L):
    """Steps from far below to far above one: decays of 1 and of 0, and gates at both ends."""
    i = scan_inputs(1, L, 64, 16, 1, "f32")
    i["dt"] = 12 * i["dt"]
    i["dt"][:, 1::5] = -60.0
    i["dt"][:, 2::5] = 40.0
    i["z"] = 30 * i["z"]
    y, h = scan(i)
    ref, href = scan_reference(i, "f32")
    R.check(y, ref, "y")
    R.check(h, href, "h_final")


@pytest.mark.parametrize("L", [5, 700])
def test_scan_non_finite_inputs_stay_in_their_channel_and_after_their_token(L):
    i = scan_inputs(2, L, 40, 16, 1, "f32", gate=False)
    t = L // 2
    i["x"][0, t, 7] = NAN
    i["dt"][1, t, 9] = NAN
    y, h = scan(i)
    bad = torch.isnan(y).cpu()
    want = torch.zeros_like(bad)
    want[0, t:, 7] = want[1, t:, 9] = True
    assert torch.equal(bad, want)
    hb = torch.isnan(h).cpu().any(-1)
    assert hb[0].nonzero().flatten().tolist() == [7] and hb[1].nonzero().flatten().tolist() == [9]


def test_scan_empty():
    i = scan_inputs(2, 0, 16, 8, 1, "bf16")
    y, h = scan(i)
    assert y.shape == (2, 0, 16) and torch.equal(h, i["h0"])
    _, h = scan(dict(i, h0=None))
    assert (h == 0).all()


def test_scan_same_bits_every_run():
    i = scan_inputs(1, 3000, 256, 16, 1, "bf16")
    y, h = scan(i)
    for _ in range(3):
        y2, h2 = scan(i)
        assert torch.equal(y, y2) and torch.equal(h, h2)


@pytest.mark.parametrize("L", [2, 40, 1000])
def test_outputs_in_slices_and_no_final_states(L):
    """The halves of one wider tensor: x and z read from it, y written over what was x's
    neighbour; no final states asked for."""
    ch = 48
    i = scan_inputs(2, L, ch, 16, 1, "bf16")
    wide = torch.full((2, L, 3 * ch), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[..., :ch], wide[..., 2 * ch:] = i["x"], i["z"]
    y, h = scan(dict(i, x=wide[..., :ch], z=wide[..., 2 * ch:]), y=wide[..., ch:2 * ch],
                want_final_state=False)
    assert h is None
    ref, _ = scan_reference(i, "bf16")
    R.check(wide[..., ch:2 * ch], ref, "y")
    assert torch.equal(wide[..., :ch], i["x"]) and torch.equal(wide[..., 2 * ch:], i["z"])
    weight = torch.randn(ch, 4, generator=_gen(30)).cuda()
    y, sf = api.la_causal_conv_fwd(wide[..., :ch], weight, y=wide[..., ch:2 * ch],
                                   want_final_state=False)
    assert sf is None
    ref, _ = R.causal_conv(i["x"], weight, None, "silu", None, None, "bf16")
    R.check(wide[..., ch:2 * ch], ref, "conv")
    assert torch.equal(wide[..., :ch], i["x"]) and torch.equal(wide[..., 2 * ch:], i["z"])
    api.la_gated_norm_fwd(wide[:, None, :, :ch], wide[..., 2 * ch:], y=wide[..., ch:2 * ch])
    ref = R.gated_norm(i["x"][:, None], i["z"], None, None, "rms", "silu", False, 1e-5, "bf16")
    R.check(wide[..., ch:2 * ch], ref, "gated")
    assert torch.equal(wide[..., :ch], i["x"]) and torch.equal(wide[..., 2 * ch:], i["z"])


def test_one_token_taken_out_of_a_prompt():
    """x[:, t:t+1] of longer tensors as it lies: rows a whole sequence apart."""
    i = scan_inputs(5, 9, 72, 16, 1, "bf16")
    cut = lambda v: v[:, 4:5]  # noqa: E731
    part = {k: (cut(v) if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in i.items()}
    dense = {k: (v.contiguous() if k in ("x", "dt", "z", "Bm", "Cm") else v)
             for k, v in part.items()}
    y = torch.full((5, 9, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    _, h = scan(part, y=cut(y))
    want = scan(dense)
    assert torch.equal(cut(y), want[0]) and torch.equal(h, want[1])
    w = torch.randn(72, 4, generator=_gen(32)).cuda()
    st = torch.randn(5, 3, 72, generator=_gen(33)).bfloat16().cuda()
    _, sf = api.la_causal_conv_fwd(part["x"], w, state0=st, y=cut(y))
    want = api.la_causal_conv_fwd(dense["x"], w, state0=st)
    assert torch.equal(cut(y), want[0]) and torch.equal(sf, want[1])
    api.la_gated_norm_fwd(part["x"][:, None], part["z"], y=cut(y))
    assert torch.equal(cut(y), api.la_gated_norm_fwd(dense["x"][:, None], dense["z"]))
    rest = torch.ones(9, dtype=torch.bool)
    rest[4] = False
    assert (y[:, rest.cuda()] == 5).all()


def test_many_sequences_of_one_token():
    i = scan_inputs(70000, 1, 8, 4, 1, "f32")
    ref, href = scan_reference({k: (v[-300:] if k in ("x", "dt", "z", "Bm", "Cm", "h0") else v)
                                for k, v in i.items()}, "f32")
    y, h = scan(i)
    R.check(y[-300:], ref, "y")
    R.check(h[-300:], href, "h_final")
    x, weight, bias, st, _ = conv_inputs(70000, 1, 8, 4, "f32")
    y, _ = api.la_causal_conv_fwd(x, weight, bias, state0=st)
    ref, _ = R.causal_conv(x[-300:], weight, bias, "silu", st[-300:], None, "f32")
    R.check(y[-300:], ref, "conv")


def test_scan_ragged_segments_in_place():
    i = scan_inputs(6, 900, 64, 16, 1, "f32", ragged=True)
    assert api.la_selective_scan_fwd_workspace_bytes(6, 900, 64, 16) > 0
    ref, href = scan_reference(i, "f32")
    h = i["h0"].clone()
    y, _ = scan(dict(i, h0=h), h_final=h)
    live = _live(i["lengths"], 6, 900)
    R.check(y, ref, "y", live)
    assert (y.cpu().numpy()[~live] == 0).all()
    R.check(h, href, "h_final")


# ---------------------------------------------------------------- norms
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,L,d,norm,act,first,heads,head_major,bias", [
    (1, 1, 1, 1, "rms", "silu", False, False, True, False),
    (2, 3, 5, 64, "rms", "silu", False, False, True, False),
    (2, 4, 37, 128, "layer", "sigmoid", False, True, True, True),
    (3, 2, 7, 80, "rms", "silu", True, False, False, False),
    (2, 5, 3, 33, "layer", "silu", True, True, False, True),
    (1, 2, 9, 256, "rms", "none", False, True, True, False),
    (2, 1, 5, 1000, "layer", "silu", False, False, False, False),
    (1, 1, 3, 4096, "rms", "silu", True, False, False, True),
    (1, 2, 2, 5003, "rms", "sigmoid", False, True, False, False),
    (1, 1, 2, 16384, "layer", "silu", True, False, False, True),
    (2, 16, 130, 16, "rms", "silu", False, False, True, False),
    (64, 8, 1, 128, "rms", "silu", False, False, True, False),
    (2, 3, 5, 66, "layer", "silu", False, True, True, True),     # pairs of elements
    (1, 2, 3, 1030, "layer", "silu", True, False, True, False),
    (1, 2, 3, 515, "rms", "silu", False, True, True, False),     # single elements
    (1, 1, 2, 16383, "layer", "sigmoid", False, False, True, True),
    (1, 3, 2, 512, "layer", "silu", False, False, True, False),
])
def test_gated_norm(B, H, L, d, norm, act, first, heads, head_major, bias, dtype):
    g = _gen(3)
    x = (1 + torch.randn(B, H, L, d, generator=g)).to(DT[dtype]).cuda()
    if not head_major:
        x = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    gate = _rows(g, B, L, H * d, dtype, not head_major)
    n = H * d if heads else d
    w = torch.randn(n, generator=g).cuda()
    b = torch.randn(n, generator=g).cuda() if bias else None
    y = api.la_gated_norm_fwd(x, gate, w, b, norm=norm, activation=act, gate_first=first)
    R.check(y, R.gated_norm(x, gate, w, b, norm, act, first, 1e-5, dtype), "y")


@pytest.mark.parametrize("d", [64, 100])
def test_gated_norm_optional_arguments_and_slices(d):
    g = _gen(4)
    x = torch.randn(2, 3, 6, d, generator=g).cuda()
    y = api.la_gated_norm_fwd(x, norm="layer", eps=1e-3)
    R.check(y, R.gated_norm(x, None, None, None, "layer", "silu", False, np.float32(1e-3), "f32"), "y")
    wide = torch.full((2, 6, 3 * d + 8), 5.0).cuda()  # written into the middle of wider rows
    gate = torch.randn(2, 6, 3 * d, generator=g).cuda()
    api.la_gated_norm_fwd(x, gate, y=wide[..., 4:4 + 3 * d])
    R.check(wide[..., 4:4 + 3 * d], R.gated_norm(x, gate, None, None, "rms", "silu", False, 1e-5, "f32"), "y")
    assert (wide[..., :4] == 5).all() and (wide[..., 4 + 3 * d:] == 5).all()
    ref = R.gated_norm(x, gate, None, None, "rms", "silu", True, 1e-5, "f32")
    y = api.la_gated_norm_fwd(x, gate, gate_first=True, y=gate)  # over the gate itself
    assert y is gate
    R.check(y, ref, "y over gate")
    # one head's row for every head, by a stride of zero
    one = torch.randn(2, 1, 6, d, generator=g).cuda().expand(2, 3, 6, d)
    R.check(api.la_gated_norm_fwd(one), R.gated_norm(one, None, None, None, "rms", "silu", False, 1e-5, "f32"), "y")


def test_gated_norm_rows_of_zeros_and_non_finite_rows():
    x = torch.randn(1, 2, 8, 64, generator=_gen(5)).cuda()
    x[0, 0, 1] = 0
    x[0, 1, 2, 5] = NAN
    x[0, 0, 3, 6] = float("inf")
    y = api.la_gated_norm_fwd(x).view(8, 2, 64)
    assert (y[1, 0] == 0).all()
    assert torch.isnan(y[2, 1]).all()
    assert (y[3, 0, :6] == 0).all() and torch.isnan(y[3, 0, 6])  # finite / inf, inf / inf
    rest = torch.ones(8, 2, dtype=torch.bool)
    rest[2, 1] = rest[3, 0] = False
    assert torch.isfinite(y[rest.cuda()]).all()


@pytest.mark.parametrize("dtype,rd", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("R_,D,post,scale,norm,bias", [
    (1, 1, False, False, "rms", False),
    (5, 64, True, True, "rms", False),
    (7, 100, False, True, "layer", True),
    (32, 2048, False, False, "rms", False),
    (3, 4096, True, True, "layer", True),
    (9, 1001, True, False, "rms", False),
    (2, 16384, True, True, "rms", False),
    (2, 9001, True, True, "layer", True),
    (700, 520, True, True, "rms", False),
    (3, 8192, False, False, "layer", False),
    (11, 66, True, True, "layer", True),
    (5, 3150, True, True, "rms", False),
    (4, 515, True, False, "layer", True),
    (2, 16383, True, True, "rms", False),
    (5000, 24, True, True, "rms", False),      # teams of a warp with several rows each
    (1500, 2056, True, True, "layer", False),  # blocks with several rows each
    (1301, 1027, True, True, "layer", True),   # and the same where rows start in mid-vector
    (3001, 77, True, True, "rms", False),
    (21001, 13, False, True, "layer", False),
    (701, 9001, True, True, "rms", False),
    (3, 16377, True, False, "layer", True),
    (4, 16378, False, False, "rms", False),
    (4, 16381, True, True, "rms", False),
])
def test_residual_norm(R_, D, post, scale, norm, bias, dtype, rd):
    g = _gen(6)
    x = torch.randn(R_, D, generator=g).to(DT[dtype]).cuda()
    res = (3 * torch.randn(R_, D, generator=g)).to(DT[rd]).cuda()
    p = lambda on: torch.randn(D, generator=g).cuda() if on else None  # noqa: E731
    pw, sc, w, b = p(post), p(scale), p(True), p(bias)
    y, r = api.la_residual_norm_fwd(x, res, w, b, post_weight=pw, scale=sc, alpha=0.7, norm=norm)
    ry, rr = R.residual_norm(x, res, pw, sc, 0.7, w, b, norm, 1e-5, dtype, rd)
    R.check(r, rr, "residual_out")
    R.check(y, ry, "y")
    # in place over both inputs, between rows that stay as they are
    xw, rw = (torch.full(((R_ + 16) * D,), 3.0, dtype=v.dtype, device="cuda") for v in (x, res))
    x2, res2 = (w[8 * D:(8 + R_) * D].view(R_, D) for w in (xw, rw))
    x2.copy_(x), res2.copy_(res)
    y2, r2 = api.la_residual_norm_fwd(x2, res2, w, b, post_weight=pw, scale=sc, alpha=0.7,
                                      norm=norm, y=x2, residual_out=res2)
    assert y2 is x2 and r2 is res2 and torch.equal(y2, y) and torch.equal(r2, r)
    for w in (xw, rw):
        assert (w[:8 * D] == 3).all() and (w[(8 + R_) * D:] == 3).all()


def test_residual_norm_first_block_and_shapes():
    g = _gen(7)
    x = torch.randn(2, 3, 96, generator=g).cuda()
    y, r = api.la_residual_norm_fwd(x)
    ry, rr = R.residual_norm(x, None, None, None, 1.0, None, None, "rms", 1e-5, "f32", "f32")
    R.check(y, ry, "y")
    assert torch.equal(r, x)
    y, r = api.la_residual_norm_fwd(x.bfloat16(), residual_dtype=torch.float32)
    assert r.dtype == torch.float32 and torch.equal(r, x.bfloat16().float())
    y, r = api.la_residual_norm_fwd(torch.zeros(0, 96).cuda())
    assert y.shape == (0, 96)


def test_residual_norm_post_normed_row_of_zeros():
    x = torch.zeros(2, 64).cuda()
    res = torch.randn(2, 64, generator=_gen(8)).cuda()
    y, r = api.la_residual_norm_fwd(x, res, post_weight=torch.ones(64).cuda())
    assert torch.equal(r, res) and torch.isfinite(y).all()


# ---------------------------------------------------------------- together
def block_params(Dm, ch, N, Wd, rank, seed=0):
    g = _gen(seed)
    r = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).cuda()  # noqa: E731
    step = torch.exp(np.log(1e-3) + torch.rand(ch, generator=g) * np.log(100.0))
    return dict(w_in=r(2 * ch, Dm), conv=r(ch, Wd), conv_b=0.1 * r(ch, 1)[:, 0],
                w_x=r(rank + 2 * N, ch), w_dt=r(ch, rank),
                dt_bias=(step + torch.log(-torch.expm1(-step))).cuda(),
                A=-(torch.arange(1, N + 1).float().repeat(ch, 1)).cuda(), D=torch.ones(ch).cuda(),
                w_out=r(Dm, ch), norm=(1 + r(Dm, 1)[:, 0]), onorm=(1 + r(ch, 1)[:, 0]))


def block(p, x, residual, conv_state, h, Wd, rank, N, lengths=None):
    """A state space block as a user composes it: residual norm, input projection, convolution,
    scan, gated norm, output projection; the states in place.  x, residual [B,L,Dm]."""
    u, residual = api.la_residual_norm_fwd(x, residual, p["norm"])
    xz = u @ p["w_in"].T.to(u.dtype)
    ch = p["A"].shape[0]
    xi, z = xz[..., :ch], xz[..., ch:]
    c, _ = api.la_causal_conv_fwd(xi, p["conv"], p["conv_b"], state0=conv_state, lengths=lengths,
                                  state_final=conv_state)
    xd = c @ p["w_x"].T.to(u.dtype)
    dt = xd[..., :rank] @ p["w_dt"].T.to(u.dtype)
    y, _ = api.la_selective_scan_fwd(c, dt, p["A"], xd[..., rank:rank + N], xd[..., rank + N:],
                                     D=p["D"], dt_bias=p["dt_bias"], h0=h, h_final=h,
                                     lengths=lengths)
    o = api.la_gated_norm_fwd(y[:, None], z, p["onorm"])
    return o @ p["w_out"].T.to(u.dtype), residual


DIMS = dict(Dm=96, ch=192, N=16, Wd=4, rank=6)


def _states(B):
    return (torch.zeros(B, DIMS["Wd"] - 1, DIMS["ch"]).cuda(),
            torch.zeros(B, DIMS["ch"], DIMS["N"]).cuda())


def test_block_prompt_then_tokens_is_the_whole_prompt():
    """The prompt in one call, and a shorter prompt followed by single tokens, in fp32.  Both
    compute the same sums in another order: some 1e-6 of the values' size at 40 tokens."""
    p = block_params(**DIMS)
    B, L, cut = 2, 40, 33
    x = torch.randn(B, L, DIMS["Dm"], generator=_gen(9)).cuda()
    res = torch.randn(B, L, DIMS["Dm"], generator=_gen(10)).cuda()
    args = (DIMS["Wd"], DIMS["rank"], DIMS["N"])
    cs, h = _states(B)
    y, r = block(p, x, res, cs, h, *args)
    cs2, h2 = _states(B)
    parts = [(0, cut)] + [(t, t + 1) for t in range(cut, L)]
    outs = [block(p, x[:, a:b].contiguous(), res[:, a:b].contiguous(), cs2, h2, *args)
            for a, b in parts]
    for got, want in ((torch.cat([o[0] for o in outs], 1), y), (cs2, cs), (h2, h),
                      (torch.cat([o[1] for o in outs], 1), r)):
        assert (got - want).abs().max() <= 2e-5 * want.abs().max()


def test_block_padded_batch_is_each_sequence_alone():
    p = block_params(**DIMS)
    B, L = 4, 50
    x = torch.randn(B, L, DIMS["Dm"], generator=_gen(11)).cuda()
    res = torch.randn(B, L, DIMS["Dm"], generator=_gen(12)).cuda()
    n = torch.tensor([50, 0, 17, 1], dtype=torch.int32).cuda()
    args = (DIMS["Wd"], DIMS["rank"], DIMS["N"])
    cs, h = _states(B)
    y, _ = block(p, x, res, cs, h, *args, lengths=n)
    for b, m in enumerate(n.tolist()):
        cs1, h1 = _states(1)
        if m:
            y1, _ = block(p, x[b:b + 1, :m].contiguous(), res[b:b + 1, :m].contiguous(), cs1, h1,
                          *args)
            assert (y[b, :m] - y1[0]).abs().max() <= 2e-5 * y1.abs().max()
        assert (h[b] - h1[0]).abs().max() <= 2e-5 * max(1.0, float(h1.abs().max()))
        assert (cs[b] - cs1[0]).abs().max() <= 2e-5 * max(1.0, float(cs1.abs().max()))


def test_attention_output_through_gated_and_residual_norm():
    """O of la_chunk_fwd straight into the gated norm, then the residual step."""
    B, H, L, d = 2, 4, 150, 64
    w = W.small_prefill(B, H, L, d, d, "bf16", "identity", "logit", 64)
    inp = W.make_prefill_inputs(w, seed=5)
    api.la_set_feature_map("identity")
    O, _ = api.la_chunk_fwd(*(to_dev(inp[k]) for k in "qkv"), 64, "logit", to_dev(inp["decay"]))
    g = _gen(13)
    gate = torch.randn(B, L, H * d, generator=g).bfloat16().cuda()
    nw = torch.randn(d, generator=g).cuda()
    y = api.la_gated_norm_fwd(O, gate, nw)
    R.check(y, R.gated_norm(O, gate, nw, None, "rms", "silu", False, 1e-5, "bf16"), "y")
    res = torch.randn(B, L, H * d, generator=g).cuda()
    out, r = api.la_residual_norm_fwd(y, res, alpha=0.5)
    ro, rr = R.residual_norm(y, res, None, None, 0.5, None, None, "rms", 1e-5, "bf16", "f32")
    R.check(out, ro, "out")
    R.check(r, rr, "residual")
    api.la_device_status()


def test_block_decode_step_captured_and_replayed():
    """A decode step of the block in a CUDA graph, states in place: replays advance it as eager
    calls do, bit for bit."""
    p = block_params(**DIMS)
    B, steps = 3, 5
    args = (DIMS["Wd"], DIMS["rank"], DIMS["N"])
    toks = torch.randn(steps, B, 1, DIMS["Dm"], generator=_gen(14)).cuda()
    res = torch.randn(B, 1, DIMS["Dm"], generator=_gen(15)).cuda()
    cs, h = _states(B)
    eager = [block(p, toks[t], res, cs, h, *args)[0].clone() for t in range(steps)]
    cs2, h2 = _states(B)
    x = toks[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(p, x, res, cs2, h2, *args)
    torch.cuda.current_stream().wait_stream(side)
    cs2.zero_(), h2.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = block(p, x, res, cs2, h2, *args)
    for t in range(steps):
        x.copy_(toks[t])
        graph.replay()
        assert torch.equal(y, eager[t])
    assert torch.equal(h2, h) and torch.equal(cs2, cs)


def test_two_captured_prompts_replay_side_by_side():
    """Two graphs of long scans captured on one stream keep workspaces of their own."""
    runs = []
    for seed in (20, 21):
        i = scan_inputs(1, 3000, 256, 16, 1, "bf16", seed=seed)
        want = scan(i)
        y, h = torch.empty_like(want[0]), torch.empty_like(want[1])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            scan(i, y=y, h_final=h)
        runs.append((i, want, y, h, graph, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for *_, graph, stream in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, want, y, h, *_ in runs:
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])


def test_calls_on_two_streams_at_once():
    runs = []
    for seed in (22, 23):
        i = scan_inputs(1, 2500, 256, 16, 1, "f32", seed=seed)
        runs.append((i, scan(i), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[scan(i, stream=s) for i, _, s in runs] for _ in range(3)]
    torch.cuda.synchronize()
    for rep in got:
        for (y, h), (_, want, _) in zip(rep, runs):
            assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    s = torch.cuda.Stream()
    x = torch.randn(2, 3, 4, 64).cuda()
    torch.cuda.synchronize()
    a = api.la_gated_norm_fwd(x, stream=s)
    b = api.la_residual_norm_fwd(x, stream=s)[0]
    c = api.la_causal_conv_fwd(x[0], torch.ones(64, 2).cuda(), stream=s)[0]
    s.synchronize()
    assert torch.equal(a, api.la_gated_norm_fwd(x))
    assert torch.equal(b, api.la_residual_norm_fwd(x)[0])
    assert torch.equal(c, api.la_causal_conv_fwd(x[0], torch.ones(64, 2).cuda())[0])


def test_offsets_past_32_bits():
    """The last sequence of tensors with more than 2^31 elements."""
    B, L, D = 2, 1 << 18, 1 << 13  # 2 * 2^31 elements of bf16
    x = torch.zeros(B, L, D, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    x[1, -64:] = torch.randn(64, D, generator=_gen(24)).bfloat16().cuda()
    weight, bias = torch.randn(D, 4, generator=_gen(25)).cuda(), None
    _, sf = api.la_causal_conv_fwd(x, weight, bias, y=y)
    ref, _ = R.causal_conv(x[1:, -66:], weight, bias, "silu", None, None, "bf16")
    assert torch.equal(sf, x[:, -3:])
    R.check(y[1:, -60:], (ref[0][:, -60:], ref[1][:, -60:]), "conv")
    o = api.la_gated_norm_fwd(x.view(B, L, 64, 128).permute(0, 2, 1, 3), y=y)
    ref = R.gated_norm(x[1:, -8:].reshape(1, 8, 64, 128).permute(0, 2, 1, 3), None, None, None,
                       "rms", "silu", False, 1e-5, "bf16")
    R.check(o[1:, -8:], ref, "gated")
    del o
    out, r = api.la_residual_norm_fwd(x, y=y, residual_out=torch.empty_like(x))
    ro, _ = R.residual_norm(x[1, -8:], None, None, None, 1.0, None, None, "rms", 1e-5, "bf16",
                            "bf16")
    R.check(out[1, -8:], ro, "residual")
    assert torch.equal(r[1, -8:], x[1, -8:])
