"""The state space block's operators on the GPU at the ends of their ranges: masks and
infinities among the steps, states that grow, the largest sizes, calls side by side."""
import threading

import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import _native, api
from tests import ssm_reference as R
from tests.test_gpu_ssm import DT, scan, scan_inputs, scan_reference

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
