"""The state space block's operators on the GPU at the ends of their ranges: masks and
infinities among the steps, states that grow, the largest sizes, calls side by side."""
import threading

import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import _native, api
from tests import ssm_reference as R
from tests.test_gpu_ssm import DT, _live, scan, scan_inputs, scan_reference

pytestmark = pytest.mark.gpu

INF = float("inf")


# ---------------------------------------------------------------- steps
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mask", ["-inf", "lowest", "-2.4e38"])
@pytest.mark.parametrize("L", [1, 6, 40, 700])
def test_scan_masked_steps_keep_the_state(L, mask, dtype):
    """softplus(-200) is below every fp32 number, so its step is 0, and so are those of the
    values that a mask writes: the same bits."""
    i = scan_inputs(2, L, 40, 16, 1, dtype)
    at = (torch.arange(L) % 3 != 1).cuda()
    fill = torch.finfo(DT[dtype]).min if mask == "lowest" else float(mask)
    got, want = (dict(i, dt=i["dt"].clone()) for _ in range(2))
    got["dt"][:, at], want["dt"][:, at] = fill, -200.0
    (y, h), (y2, h2) = scan(got), scan(want)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    ref, href = scan_reference(want, dtype)
    R.check(y, ref, "y")
    R.check(h, href, "h_final")
    if L == 1:
        assert torch.equal(h, i["h0"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 5, 40, 700])
def test_scan_largest_finite_step_forgets_the_state(L, dtype):
    """delta of the type's largest value: every decay is 0, and with x = 0 so is the write."""
    i = scan_inputs(2, L, 40, 16, 1, dtype, gate=False)
    t = L // 2
    i["dt"][:, t], i["x"][:, t] = torch.finfo(DT[dtype]).max, 0
    y, h = scan(i)
    assert (y[:, t] == 0).all() and torch.isfinite(y).all() and torch.isfinite(h).all()
    if t == L - 1:
        assert (h == 0).all()


@pytest.mark.parametrize("L", [5, 40, 700])
def test_scan_infinite_steps_stay_in_their_channel(L):
    i = scan_inputs(2, L, 40, 16, 1, "f32", gate=False)
    t = L // 2
    i["dt"][0, t, 7], i["dt"][1, t, 9] = INF, -INF
    y, h = scan(i)
    want = torch.zeros(2, L, 40, dtype=torch.bool)
    want[0, t:, 7] = True
    assert torch.equal(~torch.isfinite(y).cpu(), want)
    assert (~torch.isfinite(h)).any(-1).nonzero().tolist() == [[0, 7]]


def test_gates_at_the_ends_of_their_range_touch_their_element_alone():
    """A gate of the lowest value is a factor of 0, a NaN or an infinity leaves one element."""
    i = scan_inputs(1, 20, 40, 16, 1, "f32")
    y0, h0 = scan(i)
    z = i["z"].clone()
    z[0, 3, 1], z[0, 4, 2], z[0, 5, 3] = torch.finfo(torch.float32).min, float("nan"), INF
    y, h = scan(dict(i, z=z))
    assert y[0, 3, 1] == 0 and torch.isnan(y[0, 4, 2]) and not torch.isfinite(y[0, 5, 3])
    o0 = api.la_gated_norm_fwd(i["x"][:, None], i["z"])
    o = api.la_gated_norm_fwd(i["x"][:, None], z)
    assert o[0, 3, 1] == 0 and torch.isnan(o[0, 4, 2]) and not torch.isfinite(o[0, 5, 3])
    rest = torch.ones(20, 40, dtype=torch.bool, device="cuda")
    rest[3, 1] = rest[4, 2] = rest[5, 3] = False
    assert torch.equal(y[0, rest], y0[0, rest]) and torch.equal(h, h0)
    assert torch.equal(o[0, rest], o0[0, rest])


# ---------------------------------------------------------------- groups
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,L,ch,N,G,packed,ragged", [
    (2, 40, 272, 16, 2, False, False),    # 136 channels a group: three blocks, 16-byte rows
    (2, 40, 150, 24, 2, False, False),    # 75: no vector divides it
    (2, 40, 300, 10, 2, True, False),     # 150: rows on 4-byte boundaries at best
    (2, 33, 520, 4, 2, False, False),
    (2, 20, 120, 128, 3, False, False),
    (1, 18, 99, 256, 3, False, False),
    (6, 1200, 400, 16, 4, False, True),   # segments too
    (1, 900, 264, 32, 3, True, False),
])
def test_scan_groups_of_several_blocks(B, L, ch, N, G, packed, ragged, dtype):
    i = scan_inputs(B, L, ch, N, G, dtype, packed, ragged=ragged)
    if L > 100:
        assert api.la_selective_scan_fwd_workspace_bytes(B, L, ch, N, G) > 0
    y, h = scan(i)
    ref, href = scan_reference(i, dtype)
    R.check(y, ref, "y", _live(i["lengths"], B, L))
    R.check(h, href, "h_final")


# ---------------------------------------------------------------- growth over segments
def _segment(B, L, ch, N):
    """Tokens in a segment of the scan's plan, from the size of its workspace."""
    need = api.la_selective_scan_fwd_workspace_bytes(B, L, ch, N)
    nseg = need // (4 * B * ch * (N + 1)) + 1
    assert nseg > 3
    return ((L + nseg - 1) // nseg + 15) // 16 * 16


def test_scan_states_that_grow_over_a_segment():
    """exp(delta A) over a whole segment passes fp32's range although every state stays in it:
    66 steps of exponent 1.5 take 1e-30 to 1e13 in the third segment.  Tokens and states of zeros
    stay zeros."""
    B, L, ch, N = 1, 1500, 24, 16
    seg = _segment(B, L, ch, N)
    assert seg >= 66
    i = scan_inputs(B, L, ch, N, 1, "f32", gate=False, skip=False)
    i["dt_bias"] = None
    i["dt"][:] = 0
    i["dt"][:, 2 * seg:2 * seg + 66] = 0.25
    i["x"][:] = 0
    i["A"][:] = 6.0
    i["h0"][:] = 1e-30 * i["h0"]
    i["h0"][:, ::2] = 0
    y, h = scan(i, dt_softplus=False)
    ref, href = scan_reference(i, "f32", softplus=False)
    assert href[0].max() > 1e12
    R.check(y, ref, "y")
    R.check(h, href, "h_final")
    assert (y[..., ::2] == 0).all() and (h[:, ::2] == 0).all()


def test_scan_sum_of_steps_past_fp32():
    """The steps of a segment sum to infinity: a decaying state ends at 0, one that does not
    decay (A = 0) stays."""
    B, L, ch, N = 1, 1500, 24, 16
    seg = _segment(B, L, ch, N)
    i = scan_inputs(B, L, ch, N, 1, "f32", gate=False, skip=False)
    i["x"][:] = 0
    i["dt"][:, 2 * seg + 3:2 * seg + 6] = torch.finfo(torch.float32).max
    i["A"][::2] = 0
    y, h = scan(i)
    assert torch.equal(h[:, ::2], i["h0"][:, ::2]) and (h[:, 1::2] == 0).all()
    assert torch.isfinite(y).all() and (y[:, 3 * seg:, 1::2] == 0).all()


# ---------------------------------------------------------------- sizes
def test_scan_token_of_more_channels_than_32_bits_of_lanes():
    """2^27 + 64 channels of 65 states, 32 lanes to a channel; the states in place.  With A = 0,
    delta = 1/2, B = 1 and sum C = 1 every value is exact: h = x / 2 and y = x / 2."""
    ch, N = (1 << 27) + 64, 65
    torch.cuda.empty_cache()
    x = torch.randn(1, 1, ch, device="cuda", dtype=torch.bfloat16)
    u = 0.5 * x
    bc = torch.ones(2, 1, 1, N, dtype=torch.bfloat16, device="cuda")
    bc[1] = 1 / 64
    bc[1, ..., 64] = 0
    A = torch.zeros(ch, N, device="cuda")
    h = torch.zeros(1, ch, N, device="cuda")
    y = torch.full_like(x, 7.0)
    api.la_selective_scan_fwd(x, torch.full_like(x, 0.5), A, bc[0], bc[1], dt_softplus=False,
                              h0=h, h_final=h, y=y)
    assert torch.equal(y, u)
    del A
    for part, want in zip(h.split(1 << 24, 1), u[0, 0].float().split(1 << 24)):
        assert (part[0] == want[:, None]).all()
    del h, part
    torch.cuda.empty_cache()


def test_scan_offsets_past_32_bits():
    """The last tokens of the last sequence, behind 2^31 elements; a step of 1e30 in front of them
    leaves nothing of the tokens before."""
    B, L, ch, N, last = 2, 1 << 18, 1 << 13, 4, 40
    torch.cuda.empty_cache()
    tail = scan_inputs(1, last, ch, N, 1, "bf16", gate=False, state=False)
    x = torch.zeros(B, L, ch, dtype=torch.bfloat16, device="cuda")
    dt, bc = torch.zeros_like(x), torch.zeros(B, L, 2, N, dtype=torch.bfloat16, device="cuda")
    dt[:, -last - 1] = 1e30
    x[1, -last:], dt[1, -last:] = tail["x"][0], tail["dt"][0]
    bc[1, -last:, 0], bc[1, -last:, 1] = tail["Bm"][0], tail["Cm"][0]
    y = torch.zeros_like(x)
    args = dict(tail, x=x, dt=dt, Bm=bc[:, :, 0], Cm=bc[:, :, 1])
    ref, href = scan_reference(tail, "bf16")
    for segments in (True, False):
        _, h = scan(args, y=y, segments=segments)
        R.check(y[1:, -last:], ref, "y")
        R.check(h[1:], href, "h_final")
        y.zero_()
    del x, dt, y, args
    torch.cuda.empty_cache()


def test_tokens_of_more_sequences_than_32_bits_of_elements():
    """One token for each of 2^19 sequences of 2^13 channels: 2^32 states, in place."""
    B, ch, k = 1 << 19, 1 << 13, 3
    torch.cuda.empty_cache()
    tail = scan_inputs(k, 1, ch, 1, 1, "bf16")
    grow = lambda t: torch.zeros(B, *t.shape[1:], dtype=t.dtype, device="cuda")  # noqa: E731
    full = dict(tail)
    for name in ("x", "dt", "z", "Bm", "Cm", "h0"):
        full[name] = grow(tail[name])
        full[name][-k:] = tail[name]
    y = grow(tail["x"])
    ref, href = scan_reference(tail, "bf16")
    scan(full, y=y, h_final=full["h0"])
    R.check(y[-k:], ref, "y")
    R.check(full["h0"][-k:], href, "h_final")
    x = full["x"]
    del full
    weight = torch.randn(ch, 2, generator=torch.Generator().manual_seed(50)).cuda()
    state = torch.zeros(B, 1, ch, dtype=torch.bfloat16, device="cuda")
    state[-k:] = tail["z"]
    api.la_causal_conv_fwd(x, weight, state0=state, state_final=state, y=y)
    ref, _ = R.causal_conv(tail["x"], weight, None, "silu", tail["z"], None, "bf16")
    R.check(y[-k:], ref, "conv")
    assert torch.equal(state[-k:], tail["x"])
    del x, y, state
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- side by side
class _Meeting:
    """The library, with one entry point that two threads enter together: both have their
    workspaces before either launches.  Keeps the workspaces' addresses."""

    def __init__(self, name, workspace_at):
        self.lib, self.name, self.at = _native.load(), name, workspace_at
        self.both, self.seen = threading.Barrier(2), []

    def __getattr__(self, name):
        fn = getattr(self.lib, name)
        if name != self.name:
            return fn

        def call(*args):
            self.seen.append(args[self.at])
            self.both.wait(timeout=60)
            return fn(*args)
        return call


def run_together(monkeypatch, name, workspace_at, calls):
    """What the two calls give in two threads at once, on one stream; they may share no workspace."""
    lib = _Meeting(name, workspace_at)
    got, errors = [None, None], []

    def work(k):
        try:
            got[k] = calls[k]()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    with monkeypatch.context() as m:
        m.setattr(_native, "load", lambda: lib)
        threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(lib.seen) and lib.seen[0] != lib.seen[1]
    return got


def test_scans_of_two_threads_on_one_stream(monkeypatch):
    """Each of the two launches of a segmented scan may have one of another thread in front of it."""
    runs = [scan_inputs(1, 2500, 256, 16, 1, "bf16", seed=s) for s in (40, 41)]
    want = [scan(i) for i in runs]
    got = run_together(monkeypatch, "la_selective_scan_fwd", -3,
                       [lambda i=i: scan(i) for i in runs])
    for (y, h), (y2, h2) in zip(got, want):
        assert torch.equal(y, y2) and torch.equal(h, h2)
