"""Cases that measure the operators of a linear attention layer's training pass: rotary positions
(forward and backward), the backward pass of chunkwise linear attention, and the backward passes of
the gated output norm and of the residual norm.

Each case runs one operator.  ``own`` selects between the plain form (elementary torch operations
in 32 bits, angles and long sums of logarithms in 64) and the library's calls; ``exact`` evaluates
the definitions in 64 bits, written apart from the plain forms: the attention's gradients by the
recurrence, token by token, where the plain form works in chunks, and the norms' by differentiating
their definition.  All inputs are made from the seed; parameters, decays and states are fp32,
activations and their gradients bf16 or fp32.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
CHUNK = 64


# ---------------------------------------------------------------- the cases
def _rotary(name, B, Hq, Hk, L, d, rot, dtype, interleaved, backward, far):
    c = {"op": "rotary", "B": B, "Hq": Hq, "Hk": Hk, "L": L, "d": d, "rot": rot, "dtype": dtype,
         "interleaved": interleaved, "backward": backward, "far": far}
    return dict(c, name=name) if name else c


def _attn(name, B, H, L, dk, dv, dtype, phi, decay, states):
    c = {"op": "attn", "B": B, "H": H, "L": L, "dk": dk, "dv": dv, "dtype": dtype, "phi": phi,
         "decay": decay, "states": states}
    return dict(c, name=name) if name else c


def _gated(name, B, H, L, d, dtype, norm, gate_first, shared, head_major):
    c = {"op": "gated", "B": B, "H": H, "L": L, "d": d, "dtype": dtype, "norm": norm,
         "gate_first": gate_first, "shared": shared, "head_major": head_major}
    return dict(c, name=name) if name else c


def _resid(name, R, D, dtype, res_dtype, post, scale, norm):
    c = {"op": "resid", "R": R, "D": D, "dtype": dtype, "res_dtype": res_dtype, "post": post,
         "scale": scale, "norm": norm}
    return dict(c, name=name) if name else c


def listed():
    return [
        # One token of each of 64 sequences of 32 heads, each at a position of its own: decode.
        _rotary("rotary_token", 64, 32, 32, 1, 128, 128, "bf16", False, False, False),
        # Four prompts: q and k as slices of one projection, turned into the heads' layout.
        _rotary("rotary_prompt", 4, 16, 16, 4096, 64, 64, "bf16", False, False, False),
        # The gradients of one long fp32 sequence, far positions of a scaled context, half of
        # each head rotated, an odd length; written into the projection's gradient.
        _rotary("rotary_far_bwd", 1, 16, 16, 32767, 128, 64, "f32", True, True, True),
        # A short sequence of one narrow head: what a call costs.
        _attn("attn_bwd_short", 1, 1, 300, 16, 16, "f32", "identity", "none", False),
        # Four sequences of 16 heads with the positive feature map and no decay.
        _attn("attn_bwd_elu", 4, 16, 4096, 64, 64, "bf16", "elu1", "none", False),
        # Two sequences of 32 wide heads with a constant decay for each head.
        _attn("attn_bwd_head", 2, 32, 8192, 128, 128, "bf16", "identity", "head", False),
        # One long sequence with a gate for each token, carried on from a state: the gradients of
        # the gate's logits and of the state as well.
        _attn("attn_bwd_gate", 1, 16, 32768, 128, 128, "bf16", "identity", "logit", True),
        # An odd fp32 batch with values wider than keys and a decay for each token.
        _attn("attn_bwd_ragged", 3, 5, 777, 64, 128, "f32", "identity", "token", True),
        # The gradient of an attention layer's output norm and gate, per head.
        _gated("gated_bwd_heads", 4, 16, 4096, 64, "bf16", "rms", False, True, True),
        # The same over a state space block's whole width, fp32, an odd length.
        _gated("gated_bwd_wide", 2, 1, 2047, 4096, "f32", "rms", True, False, False),
        # Layer norm's backward pass for the last rows of a small batch.
        _resid("resid_bwd_rows", 32, 4096, "bf16", "bf16", False, False, "layer"),
        # A prompt batch with an fp32 residual stream, a norm after the block and a layer scale.
        _resid("resid_bwd_prompt", 16384, 4096, "bf16", "f32", True, True, "rms"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "attn", "attn", "gated", "resid"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "rotary":
        L = 1 if rng.random() < 0.3 else _log_int(rng, 2, 32768)
        d = rng.choice([16, 32, 64, 80, 128, 256])
        rot = rng.choice([d, d, d // 2, d // 2 - 2])
        Hq = _log_int(rng, 1, max(1, min(64, (64 << 20) // (2 * L * d))))
        Hk = rng.choice([Hq, Hq, _log_int(rng, 1, Hq)])
        B = _log_int(rng, 1, max(1, min(256, (64 << 20) // (2 * L * d * Hq))))
        return _rotary(None, B, Hq, Hk, L, d, rot, dtype, flag(), L > 1 and flag(), flag())
    if op == "attn":
        dk, dv = rng.choice([(64, 64), (64, 64), (128, 128), (128, 128), (32, 64), (16, 16),
                             (128, 64)])
        phi = rng.choice(["identity", "elu1"])
        decay = "none" if phi == "elu1" and flag() else rng.choice(["head", "token", "logit"])
        most = (64 << 20) if dtype == "bf16" else (16 << 20)
        L = _log_int(rng, 1, 16384)
        H = _log_int(rng, 1, max(1, min(32, most // (L * max(dk, dv)))))
        B = _log_int(rng, 1, max(1, min(16, most // (L * max(dk, dv) * H))))
        return _attn(None, B, H, L, dk, dv, dtype, phi, decay, flag())
    if op == "gated":
        L = _log_int(rng, 1, 16384)
        d = rng.choice([32, 64, 80, 128, 256, _log_int(rng, 16, 8192)])
        H = _log_int(rng, 1, max(1, min(64, 8192 // d)))
        B = _log_int(rng, 1, max(1, min(64, (16 << 20) // (L * H * d))))
        return _gated(None, B, H, L, d, dtype, rng.choice(["rms", "rms", "layer"]), flag(), flag(),
                      flag())
    R = _log_int(rng, 1, 16384)
    D = _log_int(rng, 64, min(16384, max(64, (32 << 20) // R)))
    return _resid(None, R, D, dtype, rng.choice([dtype, "f32"]), flag(), flag(),
                  rng.choice(["rms", "layer"]))


# ---------------------------------------------------------------- inputs
def _frequencies(rot):
    return torch.exp(torch.arange(rot // 2, dtype=torch.float64, device="cuda")
                     * (-2 / rot * math.log(10000.0))).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if case["op"] == "rotary":
        B, Hq, Hk, L, d = (case[k] for k in ("B", "Hq", "Hk", "L", "d"))
        zeros = lambda *n: torch.zeros(*n, device="cuda")  # noqa: E731
        # a projection's output [B,L,heads*d], read forward; backward its gradient, written
        source, target = (zeros, rand) if case["backward"] else (rand, zeros)
        packed = s["packed"] = source(B, L, (Hq + 2 * Hk) * d).to(dt)
        s["q"] = packed[..., :Hq * d].unflatten(-1, (Hq, d)).permute(0, 2, 1, 3)
        s["k"] = packed[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d)).permute(0, 2, 1, 3)
        s["q2"], s["k2"] = target(B, Hq, L, d).to(dt), target(B, Hk, L, d).to(dt)
        s["inv_freq"] = _frequencies(case["rot"])
        if case["far"]:
            s["inv_freq"] = s["inv_freq"] / 32  # positions of a context stretched by 32
        s["scale"] = 1.0 + 0.1 * math.log(32.0) if case["far"] else 1.0
        most = 1_000_000 if case["far"] else 32768
        s["offsets"] = torch.randint(0, most, (B,), generator=g, device="cuda", dtype=torch.int32)
    elif case["op"] == "attn":
        B, H, L, dk, dv = (case[k] for k in ("B", "H", "L", "dk", "dv"))
        unit = 1.0 if case["phi"] == "elu1" else dk ** -0.5
        s["q"], s["k"] = (unit * rand(B, H, L, dk)).to(dt), (unit * rand(B, H, L, dk)).to(dt)
        s["v"], s["dO"] = rand(B, H, L, dv).to(dt), rand(B, H, L, dv).to(dt)
        if case["decay"] == "head":
            s["decay"] = torch.log1p(-torch.exp2(-5 - 3 * torch.linspace(0, 1, H, device="cuda")))
        elif case["decay"] == "logit":
            s["decay"] = rand(B, H, L)
        elif case["decay"] == "token":
            s["decay"] = -0.2 * rand(B, H, L).abs()
        else:
            s["decay"] = None
        s["S0"] = 0.1 * rand(B, H, dk, dv) if case["states"] else None
        s["dSf"] = 0.1 * rand(B, H, dk, dv) if case["states"] else None
    elif case["op"] == "gated":
        B, H, L, d = (case[k] for k in ("B", "H", "L", "d"))
        if case["head_major"]:
            s["x"] = rand(B, H, L, d).to(dt)
        else:
            s["x"] = rand(B, L, H, d).to(dt).permute(0, 2, 1, 3)
        s["gate"] = rand(B, L, H * d).to(dt)
        s["dy"] = rand(B, L, H * d).to(dt)
        s["weight"] = 1 + 0.1 * rand(d if case["shared"] else H * d)
    else:
        R, D = case["R"], case["D"]
        rd = DTYPES[case["res_dtype"]]
        s["x"] = rand(R, D).to(dt)
        s["weight"] = 1 + 0.1 * rand(D)
        s["post_weight"] = 1 + 0.1 * rand(D) if case["post"] else None
        s["scale"] = 0.5 + 0.1 * rand(D) if case["scale"] else None
        s["r"] = (2 * rand(R, D) + 0.25).to(rd)   # the residual stream after the addition
        s["dy"] = rand(R, D).to(dt)
        s["dr"] = rand(R, D).to(rd)
    return s


# ---------------------------------------------------------------- plain forms
def _angles(s):
    """[B,1,L,rot/2] in 64 bits: far positions lose their angle in 32."""
    L = s["case"]["L"]
    pos = s["offsets"][:, None].double() + torch.arange(L, device="cuda")
    return (pos[..., None] * s["inv_freq"].double())[:, None]


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        out = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        out = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([out, rest], -1)


def _rotary_plain(s):
    c = s["case"]
    angle = _angles(s)
    cos = (torch.cos(angle) * s["scale"]).float()
    sin = (torch.sin(angle) * s["scale"]).float()
    dt = s["q"].dtype
    if not c["backward"]:
        return (_rotate(s["q"], cos, sin, c["rot"], c["interleaved"]).to(dt),
                _rotate(s["k"], cos, sin, c["rot"], c["interleaved"]).to(dt))
    dq = _rotate(s["q2"], cos, -sin, c["rot"], c["interleaved"])
    dk = _rotate(s["k2"], cos, -sin, c["rot"], c["interleaved"])
    s["q"].copy_(dq)
    s["k"].copy_(dk)
    return s["packed"]


def _silu(x):
    return x / (1 + torch.exp(-x))


def _phi(x, kind):
    """phi(x) and its derivative."""
    if kind == "identity":
        return x, torch.ones_like(x)
    e = torch.exp(torch.clamp(x, max=0.0))
    return torch.where(x > 0, x + 1, e), e


def _chunks(x):
    """[B,H,L,d] -> [B,H,chunks,CHUNK,d] in fp32, zeros behind the last token."""
    B, H, L, d = x.shape
    x = torch.cat([x.float(), x.new_zeros(B, H, -L % CHUNK, d, dtype=torch.float32)], 2)
    return x.view(B, H, -1, CHUNK, d)


def _log_decay(s):
    """[B,H,L] log of each token's decay in 64 bits."""
    c = s["case"]
    B, H, L = c["B"], c["H"], c["L"]
    if c["decay"] == "none":
        return torch.zeros(B, H, L, dtype=torch.float64, device="cuda")
    a = s["decay"].double()
    if c["decay"] == "head":
        return a[None, :, None].expand(B, H, L)
    if c["decay"] == "logit":
        return -(torch.clamp(a, min=0) + torch.log1p(torch.exp(-a.abs())))
    return a


def _attn_plain(s):
    c = s["case"]
    B, H, L, dk, dv = (c[k] for k in ("B", "H", "L", "dk", "dv"))
    dt = s["q"].dtype
    q, q1 = _phi(_chunks(s["q"]), c["phi"])
    k, k1 = _phi(_chunks(s["k"]), c["phi"])
    v, dO = _chunks(s["v"]), _chunks(s["dO"])
    nc = v.shape[2]
    live = (torch.arange(nc * CHUNK, device="cuda") < L).view(nc, CHUNK, 1)
    q, k = q * live, k * live                                # phi(0) is not 0 for elu1
    a = torch.cat([_log_decay(s), torch.zeros(B, H, -L % CHUNK, dtype=torch.float64,
                                              device="cuda")], 2)
    # log decays: from a chunk's start to each token, over a chunk, from the first token on
    cum = a.view(B, H, nc, CHUNK).cumsum(-1)
    total = cum[..., -1]
    run = torch.cat([torch.zeros_like(total[..., :1]), total.cumsum(-1)], -1)
    hi = cum.float()
    lo = (cum - hi.double()).float()
    diff = (hi[..., :, None] - hi[..., None, :]) + (lo[..., :, None] - lo[..., None, :])
    within = torch.exp(torch.clamp(diff, max=0)).tril()      # [j,i]: the decay from i to j
    head = torch.exp(cum.float())[..., None]                 # from the chunk's start to j
    tail = torch.exp((total[..., None] - cum).float())[..., None]   # from i to the chunk's end
    over = (run[..., :, None] - run[..., None, :]).tril()
    over = torch.exp(over.float()).tril()                    # between the chunks' ends
    zero = torch.zeros(B, H, 1, dk, dv, device="cuda")
    # states at the chunks' ends, and their gradients from the tokens behind them
    adds = (k * tail).transpose(-1, -2) @ v
    S = torch.cat([zero if s["S0"] is None else s["S0"][:, :, None], adds], 2)
    S = (over @ S.flatten(-2)).view(B, H, nc + 1, dk, dv)
    grads = (q * head).transpose(-1, -2) @ dO
    G = torch.cat([grads, zero if s["dSf"] is None else s["dSf"][:, :, None]], 2)
    G = (over.transpose(-1, -2) @ G.flatten(-2)).view(B, H, nc + 1, dk, dv)
    before, behind = S[:, :, :-1], G[:, :, 1:]
    scores = (q @ k.transpose(-1, -2)) * within
    dscores = (dO @ v.transpose(-1, -2)) * within
    dq_in = (dO @ before.transpose(-1, -2)) * head
    dk_in = (v @ behind.transpose(-1, -2)) * tail
    dq = dscores @ k + dq_in
    dk_ = dscores.transpose(-1, -2) @ q + dk_in
    dv_ = scores.transpose(-1, -2) @ dO + (k @ behind) * tail
    out = {"dq": (dq * q1).view(B, H, -1, dk)[:, :, :L].to(dt),
           "dk": (dk_ * k1).view(B, H, -1, dk)[:, :, :L].to(dt),
           "dv": dv_.view(B, H, -1, dv)[:, :, :L].to(dt)}
    if c["decay"] != "none":
        # A token's decay lies between every pair (i < t <= j): pairs of one chunk, pairs with one
        # token in it, and pairs around it.
        pairs = dscores * (q @ k.transpose(-1, -2))
        ones = torch.ones(CHUNK, CHUNK, device="cuda")
        da = ((pairs @ ones.triu(1)) * ones.tril()).sum(-2)
        da = da + (dq_in * q).sum(-1).flip(-1).cumsum(-1).flip(-1)
        earlier = (dk_in * k).sum(-1)
        da = da + (earlier @ ones.triu(1))
        da = da + ((behind * before).sum((-1, -2)) * torch.exp(total.float()))[..., None]
        da = da.reshape(B, H, -1)[..., :L]
        if c["decay"] == "head":
            da = da.sum((0, 2))
        elif c["decay"] == "logit":
            da = -da / (1 + torch.exp(-s["decay"]))
        out["ddecay"] = da
    if c["states"]:
        out["dS0"] = G[:, :, 0]
    return out


def _norm_parts(x, norm):
    """The normalised rows and 1 / deviation."""
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_grad(g, n, r, norm):
    """The gradient of a row from that of its normalised form."""
    g = g - n * (g * n).mean(-1, keepdim=True) - (g.mean(-1, keepdim=True) if norm == "layer"
                                                  else 0.0)
    return g * r


def _gated_plain(s):
    c = s["case"]
    B, H, L, d = (c[k] for k in ("B", "H", "L", "d"))
    dt = s["x"].dtype
    x = s["x"].float().permute(0, 2, 1, 3)                           # [B,L,H,d]
    z = s["gate"].float().view(B, L, H, d)
    dy = s["dy"].float().view(B, L, H, d)
    w = s["weight"] if c["shared"] else s["weight"].view(H, d)
    sig = 1 / (1 + torch.exp(-z))
    act, slope = z * sig, sig * (1 + z * (1 - sig))
    if c["gate_first"]:
        n, r = _norm_parts(x * act, c["norm"])
        dw = dy * n
        u = _norm_grad(dy * w, n, r, c["norm"])
        dx, dz = u * act, u * x * slope
    else:
        n, r = _norm_parts(x, c["norm"])
        dw = dy * act * n
        dz = dy * n * w * slope
        dx = _norm_grad(dy * act * w, n, r, c["norm"])
    dw = dw.sum((0, 1, 2)) if c["shared"] else dw.sum((0, 1)).view(-1)
    return {"dx": dx.permute(0, 2, 1, 3).to(dt), "dgate": dz.reshape(B, L, H * d).to(dt),
            "dweight": dw}


def _resid_plain(s):
    c = s["case"]
    dy = s["dy"].float()
    n, r = _norm_parts(s["r"].float(), c["norm"])
    dr = _norm_grad(dy * s["weight"], n, r, c["norm"]) + s["dr"].float()
    out = {"dresidual": dr.to(s["r"].dtype), "dweight": (dy * n).sum(0)}
    if c["norm"] == "layer":
        out["dbias"] = dy.sum(0)
    du = 0.5 * dr
    x = s["x"].float()
    if c["post"]:
        n, r = _norm_parts(x, c["norm"])
        u = n * s["post_weight"]
    else:
        u = x
    if c["scale"]:
        out["dscale"] = (du * u).sum(0)
        du = du * s["scale"]
    if c["post"]:
        out["dpost_weight"] = (du * n).sum(0)
        du = _norm_grad(du * s["post_weight"], n, r, c["norm"])
    out["dx"] = du.to(s["x"].dtype)
    return out


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"rotary": _rotary_plain, "attn": _attn_plain, "gated": _gated_plain,
                "resid": _resid_plain}[op](s)
    from causal_linear_attention_chunkwise_gb300 import api
    if op == "rotary":
        if not c["backward"]:
            return api.la_rotary_fwd(s["q"], s["k"], s["inv_freq"], offsets=s["offsets"],
                                     interleaved=c["interleaved"], scale=s["scale"],
                                     q_out=s["q2"], k_out=s["k2"])
        api.la_rotary_bwd(s["q2"], s["k2"], s["inv_freq"], offsets=s["offsets"],
                          interleaved=c["interleaved"], scale=s["scale"], q_out=s["q"],
                          k_out=s["k"])
        return s["packed"]
    if op == "attn":
        api.la_set_feature_map(c["phi"])
        dq, dk, dv, ddecay, dS0 = api.la_chunk_bwd(
            s["q"], s["k"], s["v"], s["dO"], decay_kind=c["decay"], decay=s["decay"], S0=s["S0"],
            dS_final=s["dSf"])
        out = {"dq": dq, "dk": dk, "dv": dv}
        if c["decay"] != "none":
            out["ddecay"] = ddecay
        if c["states"]:
            out["dS0"] = dS0
        return out
    if op == "gated":
        dx, dgate, dweight, _ = api.la_gated_norm_bwd(
            s["dy"], s["x"], s["gate"], s["weight"], norm=c["norm"], activation="silu",
            gate_first=c["gate_first"], eps=EPS)
        return {"dx": dx, "dgate": dgate, "dweight": dweight}
    dx, dres, dweight, dbias, dpost, dscale = api.la_residual_norm_bwd(
        s["dy"], s["r"], s["weight"], dr=s["dr"], x=s["x"], post_weight=s["post_weight"],
        scale=s["scale"], alpha=0.5, norm=c["norm"], eps=EPS, want_dbias=c["norm"] == "layer")
    out = {"dresidual": dres, "dweight": dweight, "dx": dx}
    if c["norm"] == "layer":
        out["dbias"] = dbias
    if c["scale"]:
        out["dscale"] = dscale
    if c["post"]:
        out["dpost_weight"] = dpost
    return out


def work(case):
    e = {"bf16": 2, "f32": 4}
    a = e[case["dtype"]]
    if case["op"] == "rotary":
        B, L, d, r = (case[k] for k in ("B", "L", "d", "rot"))
        heads = case["Hq"] + case["Hk"]
        # a sine and a cosine for each token and pair, counted as 20 operations each
        return {"bytes": 2 * B * L * heads * d * a + 4 * (B + r // 2),
                "flops": B * L * (3 * heads * r + 20 * r)}
    if case["op"] == "attn":
        B, H, L, dk, dv = (case[k] for k in ("B", "H", "L", "dk", "dv"))
        T = B * H * L
        data = T * (4 * dk + 3 * dv) * a
        decay = {"none": 0, "head": 8 * H}.get(case["decay"], 8 * T)
        states = 3 * B * H * dk * dv * 4 if case["states"] else 0
        # a token: two updates of a state and three products with one; with a decay two scalings
        return {"bytes": data + decay + states,
                "flops": T * dk * dv * (10 if case["decay"] == "none" else 12)}
    if case["op"] == "gated":
        n = case["B"] * case["H"] * case["L"] * case["d"]
        w = case["d"] * (1 if case["shared"] else case["H"])
        return {"bytes": 5 * n * a + 8 * w, "flops": 22 * n}
    n, r = case["R"] * case["D"], e[case["res_dtype"]]
    # dy, r, dr and the two gradients; x where its norm or scale has a gradient
    acts = n * (2 * a + 3 * r) + (n * a if case["post"] or case["scale"] else 0)
    weights = 4 * case["D"] * (2 + (case["norm"] == "layer") + 2 * bool(case["post"])
                               + 2 * bool(case["scale"]))
    return {"bytes": acts + weights, "flops": (24 if case["post"] else 12) * n}


# ---------------------------------------------------------------- 64 bits
def _rotary64(s):
    c = s["case"]
    rot, sign = c["rot"], -1.0 if c["backward"] else 1.0
    pos = s["offsets"][:, None].double() + torch.arange(c["L"], device="cuda").double()
    turn = torch.polar(torch.full_like(pos[..., None], s["scale"]),
                       sign * pos[..., None] * s["inv_freq"].double())[:, None]

    def rotated(x):
        x = x.double()
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else \
            torch.complex(x[..., :rot // 2], x[..., rot // 2:rot])
        z = z * turn
        y = x.clone()
        if c["interleaved"]:
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    if not c["backward"]:
        return [rotated(s["q"]), rotated(s["k"])]
    flat = lambda x: x.transpose(1, 2).flatten(2)  # noqa: E731
    dq, dk = flat(rotated(s["q2"])), flat(rotated(s["k2"]))
    return torch.cat([dq, dk, torch.zeros_like(dk)], -1)


def _attn64(s):
    c = s["case"]
    B, H, L, dk, dv = (c[k] for k in ("B", "H", "L", "dk", "dv"))
    if L > 40000 or B * H * L * dk * dv > 10 << 30:
        return None
    rows = lambda t: t.double().reshape(B * H, L, -1).transpose(0, 1).contiguous()  # noqa: E731
    q, k, v, dO = rows(s["q"]), rows(s["k"]), rows(s["v"]), rows(s["dO"])
    q1, k1 = torch.ones_like(q), torch.ones_like(k)
    if c["phi"] == "elu1":
        q1, k1 = torch.exp(q.clamp(max=0)), torch.exp(k.clamp(max=0))
        q, k = torch.nn.functional.elu(q) + 1, torch.nn.functional.elu(k) + 1
    decay = None if s["decay"] is None else s["decay"].double()
    a = torch.ones(L, B * H, 1, 1, dtype=torch.double, device="cuda")
    if c["decay"] == "head":
        a = torch.exp(decay).repeat(B).view(1, B * H, 1, 1).expand(L, B * H, 1, 1)
    elif c["decay"] == "token":
        a = torch.exp(decay).view(B * H, L).t()[..., None, None].contiguous()
    elif c["decay"] == "logit":
        a = torch.sigmoid(-decay).view(B * H, L).t()[..., None, None].contiguous()
    zero = torch.zeros(B * H, dk, dv, dtype=torch.double, device="cuda")
    S = zero.clone() if s["S0"] is None else s["S0"].double().reshape(B * H, dk, dv).clone()
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(L):
        S = torch.baddbmm(a[t] * S, k[t][:, :, None], v[t][:, None, :])
        dq[t] = torch.bmm(S, dO[t][:, :, None])[..., 0]
    G = zero.clone() if s["dSf"] is None else s["dSf"].double().reshape(B * H, dk, dv).clone()
    last = (G * S).sum((-1, -2))
    for t in range(L - 1, -1, -1):  # G: the gradient of the state after token t
        G = torch.baddbmm(G, q[t][:, :, None], dO[t][:, None, :])
        dk_[t] = torch.bmm(G, v[t][:, :, None])[..., 0]
        dv_[t] = torch.bmm(k[t][:, None, :], G)[:, 0]
        G = a[t] * G
    back = lambda t: t.transpose(0, 1).reshape(B, H, L, -1)  # noqa: E731
    out = {"dq": back(dq * q1), "dk": back(dk_ * k1), "dv": back(dv_)}
    if c["decay"] != "none":
        # <G_t, S_t> falls by q_t dq_t and gains k_t dk_t from token to token
        da = ((q * dq).sum(-1) - (k * dk_).sum(-1)).flip(0).cumsum(0).flip(0) + last
        da = da.t().reshape(B, H, L)
        out["ddecay"] = da.sum((0, 2)) if c["decay"] == "head" else \
            da * -torch.sigmoid(decay) if c["decay"] == "logit" else da
    if c["states"]:
        out["dS0"] = G.view(B, H, dk, dv)
    return out


def _norm64(x, norm):
    if norm == "layer":
        x = x - x.sum(-1, keepdim=True) / x.shape[-1]
    return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _leaf(t):
    return t.detach().double().requires_grad_(True)


def _gated64(s):
    c = s["case"]
    B, H, L, d = (c[k] for k in ("B", "H", "L", "d"))
    x, z, w = _leaf(s["x"]), _leaf(s["gate"]), _leaf(s["weight"])
    gate = torch.nn.functional.silu(z).view(B, L, H, d)
    scale = w if c["shared"] else w.view(H, d)
    rows = x.transpose(1, 2)
    y = _norm64(rows * gate, c["norm"]) * scale if c["gate_first"] else \
        _norm64(rows, c["norm"]) * scale * gate
    dx, dz, dw = torch.autograd.grad(y, (x, z, w), s["dy"].double().view(B, L, H, d))
    return {"dx": dx, "dgate": dz, "dweight": dw}


def _resid64(s):
    c = s["case"]
    r, w = _leaf(s["r"]), _leaf(s["weight"])
    y = _norm64(r, c["norm"]) * w
    dr, dw = torch.autograd.grad(y, (r, w), s["dy"].double())
    del y
    dr = dr + s["dr"].double()
    out = {"dresidual": dr, "dweight": dw}
    if c["norm"] == "layer":
        out["dbias"] = s["dy"].double().sum(0)
    x = _leaf(s["x"])
    leaves, names, u = [x], ["dx"], x
    if c["post"]:
        leaves.append(_leaf(s["post_weight"]))
        names.append("dpost_weight")
        u = _norm64(u, c["norm"]) * leaves[-1]
    if c["scale"]:
        leaves.append(_leaf(s["scale"]))
        names.append("dscale")
        u = u * leaves[-1]
    out.update(zip(names, torch.autograd.grad(u, leaves, dr / 2)))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _rotary64, "attn": _attn64, "gated": _gated64,
            "resid": _resid64}[case["op"]](s)
