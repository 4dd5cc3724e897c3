"""Workloads of the block operators for causal token mixing: gated linear
attention (forward, backward, one-token steps), rotary positions, and the
gated residual with the norms before and after a block.

Every case is one call (one direction of one operator). Sizes follow this
library's layers: head width 32, 36 or 70 heads, hidden widths 1152 and 2240,
16384 tokens of a 4096 px image, 21 x 30 x 52 of a 480p clip.
"""
import math

import torch

own = False

D = 32


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 64 requests: a token each, its state read and written
        {"name": "step_b64", "op": "gated", "B": 64, "N": 1, "H": 70, "io": "bf16", "carry": True,
         "packed": False},
        # a prompt chunk of 8 requests on top of a carried state
        {"name": "gated_chunk", "op": "gated", "B": 8, "N": 509, "H": 36, "io": "bf16",
         "carry": True, "packed": False},
        # the tokens of a 480p clip, several sequences packed in the row
        {"name": "gated_480p", "op": "gated", "B": 1, "N": 32760, "H": 70, "io": "bf16",
         "carry": False, "packed": True},
        # float32 tensors, ragged length
        {"name": "gated_f32", "op": "gated", "B": 3, "N": 2003, "H": 36, "io": "f32",
         "carry": False, "packed": False},
        # training: the gradients of a 16384-token layer
        {"name": "gated_bwd_4k", "op": "gated_bwd", "B": 1, "N": 16384, "H": 70, "io": "bf16",
         "carry": False, "packed": False},
        # training in float32 with a carried state, ragged length
        {"name": "gated_bwd_f32", "op": "gated_bwd", "B": 2, "N": 1021, "H": 20, "io": "f32",
         "carry": True, "packed": True},
        # positions of queries and keys of a 16384-token layer, halves layout
        {"name": "rotary_4k", "op": "rotary", "B": 1, "N": 16384, "H": 70, "Hk": 70, "D": 32,
         "rot": 32, "io": "bf16", "layout": "half", "scaling": "none", "inverse": False,
         "far": 0},
        # gradients of a partly rotated wider head, positions far out, scaled by parts
        {"name": "rotary_far", "op": "rotary", "B": 4, "N": 1000, "H": 16, "Hk": 4, "D": 128,
         "rot": 96, "io": "f32", "layout": "interleaved", "scaling": "parts", "inverse": True,
         "far": 900000},
        # the end of one block and the start of the next, 16384 tokens, adaptive layer norm
        {"name": "norm_4k", "op": "norm", "B": 1, "N": 16384, "C": 2240, "io": "bf16",
         "norm": "layer", "post": False, "modulate": True},
        # norms before and after the block, few ragged rows
        {"name": "norm_rms_small", "op": "norm", "B": 2, "N": 77, "C": 1152, "io": "f32",
         "norm": "rms", "post": True, "modulate": False},
        # training: gradients of both norms, gate and modulation
        {"name": "norm_bwd_1024px", "op": "norm_bwd", "B": 4, "N": 1024, "C": 2240, "io": "bf16",
         "norm": "rms", "post": True, "modulate": True},
        {"name": "norm_bwd_4k", "op": "norm_bwd", "B": 1, "N": 16384, "C": 2240, "io": "bf16",
         "norm": "layer", "post": False, "modulate": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "gated", "gated", "gated_bwd", "gated_bwd", "rotary", "norm",
                     "norm_bwd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "step":
        return {"op": "gated", "B": _log(rng, 1, 400), "N": rng.choice([1, 1, 2, 3]),
                "H": rng.randint(1, 80), "io": io, "carry": True, "packed": False}
    if op in ("gated", "gated_bwd"):
        B, H = _log(rng, 1, 8), _log(rng, 2, 80)
        most = 16384 * 70 // (2 if io == "f32" else 1)
        N = _log(rng, 17, min(16384, max(17, most // (B * H))))
        return {"op": op, "B": B, "N": N, "H": H, "io": io, "carry": rng.random() < 0.5,
                "packed": rng.random() < 0.3}
    if op == "rotary":
        width = rng.choice([32, 32, 64, 128])
        H = _log(rng, 1, 64)
        B = _log(rng, 1, 16)
        N = _log(rng, 1, max(1, min(16384, 16384 * 70 * 32 // (B * H * width * 2))))
        return {"op": "rotary", "B": B, "N": N, "H": H, "Hk": rng.choice([0, 1, H]), "D": width,
                "rot": rng.choice([width, width, width // 2, width - 8, 2 * rng.randint(1, width // 2)]),
                "io": io, "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "base", "parts"]),
                "inverse": rng.random() < 0.4, "far": rng.choice([0, 5000, 900000])}
    C = 8 * _log(rng, 4, 640)
    B = _log(rng, 1, 8)
    N = _log(rng, 1, max(1, min(16384, 16384 * 1120 // (C * B))))
    return {"op": op, "B": B, "N": N, "C": C, "io": io, "norm": rng.choice(["layer", "rms"]),
            "post": rng.random() < 0.5, "modulate": rng.random() < 0.6}


def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] in ("gated", "gated_bwd"):
        rows = case["B"] * case["N"] * case["H"]
        states = case["B"] * case["H"] * D * D * 4
        if case["op"] == "gated":
            # Q, K, V read and O written, the log gates; per token: S = a S + k^T v (3 D^2), q S (2 D^2)
            moved = rows * (4 * D * e + 4) + states * (2 if case["carry"] else 1)
            return {"bytes": moved, "flops": rows * 5 * D * D}
        moved = rows * (7 * D * e + 8) + (states * 3 if case["carry"] else 0)
        # S again (3 D^2), dS (3 D^2), dq, dk, dv (2 D^2 each), the gate's D^2 products (2 D^2)
        return {"bytes": moved, "flops": rows * 14 * D * D}
    if case["op"] == "rotary":
        rows = case["B"] * case["N"]
        heads = case["H"] + case["Hk"]
        return {"bytes": rows * (heads * case["D"] * 2 * e + 4), "flops": rows * heads * case["rot"] * 3}
    n = case["B"] * case["N"] * case["C"]
    small = 4 * case["C"] * ((3 if case["modulate"] else 0) * case["B"] + 1 + (1 if case["post"] else 0))
    if case["op"] == "norm":
        return {"bytes": 4 * n * e + small, "flops": 12 * n}
    return {"bytes": 6 * n * e + 2 * small, "flops": 30 * n}


# -------------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    dt = _dtype(case)
    st = {"case": dict(case)}
    if case["op"] in ("gated", "gated_bwd"):
        B, N, H = case["B"], case["N"], case["H"]
        for name in ("Q", "K", "V"):
            st[name] = randn(B, N, H, D).to(dt)
        # log gates as a layer makes them: a rate per head between 0.002 and 0.5
        # a token, times a positive factor that depends on the token
        rate = torch.exp(math.log(0.002) + rand(H) * math.log(250.0))
        G = -rate * torch.nn.functional.softplus(randn(B, N, H) + 0.5)
        if case["packed"]:
            # sequence starts: the gate of a first token lets nothing through
            first = rand(B, N, 1) < 4.0 / max(N, 8)
            G = torch.where(first, torch.full_like(G, -math.inf), G)
        st["G"] = G.float()
        st["scale"] = D ** -0.5
        st["S"] = randn(B, H, D, D) * 2.0 if case["carry"] else None
        if case["op"] == "gated_bwd":
            st["dO"] = randn(B, N, H, D).to(dt)
            st["dS"] = randn(B, H, D, D) * 0.5 if case["carry"] else None
    elif case["op"] == "rotary":
        B, N, H, Hk, W = case["B"], case["N"], case["H"], case["Hk"], case["D"]
        st["Q"] = randn(B, N, H, W).to(dt)
        st["K"] = randn(B, N, Hk, W).to(dt) if Hk else None
        # each row of the batch stands at its own place of its own sequence
        start = (rand(B, 1) * (case["far"] + 1)).to(torch.int32)
        st["pos"] = start + torch.arange(N, device="cuda", dtype=torch.int32)[None]
        st["scaling"] = {"none": None, "linear": ("linear", 4.0), "base": ("base", 8.0),
                         "parts": ("parts", 16.0, 4096, 1.0, 32.0)}[case["scaling"]]
        st["mscale"] = 0.1 * math.log(16.0) + 1.0 if case["scaling"] == "parts" else 1.0
    else:
        B, N, C = case["B"], case["N"], case["C"]
        st["x"] = (randn(B, N, C) * 2.0).to(dt)
        st["f"] = (randn(B, N, C) + 0.1).to(dt)
        st["gate"] = randn(B, C) * 0.5 if case["modulate"] else None
        st["mod_scale"] = randn(B, C) * 0.3 if case["modulate"] else None
        st["mod_shift"] = randn(B, C) * 0.3 if case["modulate"] else None
        st["w_pre"] = 1.0 + 0.1 * randn(C)
        st["w_post"] = 1.0 + 0.1 * randn(C) if case["post"] else None
        st["alpha"] = 0.7
        if case["op"] == "norm_bwd":
            st["dh"] = randn(B, N, C).to(dt)
            st["dy"] = randn(B, N, C).to(dt)
    return st


# --------------------------------------------------------------- plain forms

def _gated_plain(Q, K, V, G, S0, scale, C=64):
    """Chunks of C tokens: inside a chunk the masked products weighted by the
    decay between two tokens, between chunks a lower triangle of decays applied
    to the chunks' own states. A gate of -inf lets nothing through: such gates
    are counted apart from the sum of the others."""
    B, N, H, _ = Q.shape
    T = max(1, -(-N // C))
    pad = T * C - N

    def split(x):  # [B, N, H, w] -> [B, H, T, C, w]
        x = torch.cat([x, x.new_zeros(B, pad, H, x.shape[-1])], 1)
        return x.reshape(B, T, C, H, -1).permute(0, 3, 1, 2, 4)

    q, k, v = split(Q), split(K), split(V)
    stop = torch.isinf(G)
    g = split(torch.where(stop, torch.zeros_like(G), G).double()[..., None])[..., 0]
    n = split(stop.double()[..., None])[..., 0]
    c, m = g.cumsum(-1), n.cumsum(-1)                                 # inside the chunk, [B, H, T, C]
    low = torch.ones(C, C, device=Q.device).tril() > 0
    open_ = low & (m[..., :, None] == m[..., None, :])
    L = torch.where(open_, torch.exp(torch.where(open_, c[..., :, None] - c[..., None, :], 0.0)),
                    0.0).float()
    head = torch.where(m == 0, torch.exp(c), 0.0).float()             # from before the chunk to token i
    tail = torch.where(m == m[..., -1:], torch.exp(c[..., -1:] - c), 0.0).float()  # from token j to its end
    own_state = (k * tail[..., None]).transpose(-1, -2) @ v           # [B, H, T, D, D]
    # decay from the end of chunk s to the start of chunk t
    ct, mt = c[..., -1].cumsum(-1), m[..., -1].cumsum(-1)
    ct0 = torch.cat([torch.zeros_like(ct[..., :1]), ct], -1)          # before chunk 0, after chunk 0, ...
    mt0 = torch.cat([torch.zeros_like(mt[..., :1]), mt], -1)
    low = torch.ones(T + 1, T + 1, device=Q.device).tril() > 0
    open_ = low & (mt0[..., :, None] == mt0[..., None, :])
    A = torch.where(open_, torch.exp(torch.where(open_, ct0[..., :, None] - ct0[..., None, :], 0.0)),
                    0.0).float()
    first = torch.zeros_like(own_state[:, :, 0]) if S0 is None else S0
    states = torch.cat([first[:, :, None], own_state], 2).reshape(B, H, T + 1, -1)
    before = (A @ states).reshape(B, H, T + 1, D, D)                  # state before chunk t; last: the end
    o = (L * (q @ k.transpose(-1, -2))) @ v + head[..., None] * (q @ before[:, :, :T])
    o = scale * o.permute(0, 2, 3, 1, 4).reshape(B, T * C, H, D)[:, :N]
    return o, before[:, :, T]


def _frequencies(case, st):
    """Turning rate of each pair, in 64 bits."""
    rot = case["rot"]
    k = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    base = 10000.0
    kind = st["scaling"]
    if kind and kind[0] == "base" and rot > 2:
        base = base * kind[1] ** (rot / (rot - 2))
    f = base ** (-2.0 * k / rot)
    if kind and kind[0] == "linear":
        f = f / kind[1]
    if kind and kind[0] == "parts":
        _, factor, length, slow, fast = kind
        turns = length * f / (2.0 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f


def _rotary_plain(x, cos, sin, rot, layout):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if layout == "interleaved" else (x[..., : rot // 2], x[..., rot // 2: rot])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([ra, rb], -1).flatten(-2) if layout == "interleaved" else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _norm_plain(x, f, gate, w_post, w_pre, mod_scale, mod_shift, alpha, kind, eps=1e-6):
    u = f if w_post is None else f * torch.rsqrt((f * f).mean(-1, keepdim=True) + eps) * w_post
    h = x + alpha * (u if gate is None else gate[:, None] * u)
    a = h - h.mean(-1, keepdim=True) if kind == "layer" else h
    y = a * torch.rsqrt((a * a).mean(-1, keepdim=True) + eps) * w_pre
    if mod_scale is not None:
        y = y * (1.0 + mod_scale[:, None]) + mod_shift[:, None]
    return h, y


def _leaf(x):
    return None if x is None else x.detach().float().requires_grad_()


def run(state):
    st, case = state, state["case"]
    if own:
        return _run_own(st, case)
    dt = _dtype(case)
    if case["op"] == "gated":
        with torch.no_grad():
            o, S = _gated_plain(st["Q"].float(), st["K"].float(), st["V"].float(), st["G"], st["S"],
                                st["scale"])
            return {"O": o.to(dt), "S": S}
    if case["op"] == "gated_bwd":
        q, k, v, g, s = (_leaf(st[n]) for n in ("Q", "K", "V", "G", "S"))
        o, S = _gated_plain(q, k, v, g, s, st["scale"])
        ins = [q, k, v, g] + ([] if s is None else [s])
        outs, grads = ([o], [st["dO"].float()]) if s is None else ([o, S], [st["dO"].float(), st["dS"]])
        d = torch.autograd.grad(outs, ins, grads)
        out = {"dQ": d[0].to(dt), "dK": d[1].to(dt), "dV": d[2].to(dt), "dG": d[3]}
        if s is not None:
            out["dS"] = d[4]
        return out
    if case["op"] == "rotary":
        angle = st["pos"].double()[..., None, None] * _frequencies(case, st)
        if case["inverse"]:
            angle = -angle
        cos = (torch.cos(angle) * st["mscale"]).float()
        sin = (torch.sin(angle) * st["mscale"]).float()
        out = {"Q": _rotary_plain(st["Q"], cos, sin, case["rot"], case["layout"]).to(dt)}
        if st["K"] is not None:
            out["K"] = _rotary_plain(st["K"], cos, sin, case["rot"], case["layout"]).to(dt)
        return out
    names = ("x", "f", "gate", "w_post", "w_pre", "mod_scale", "mod_shift")
    if case["op"] == "norm":
        with torch.no_grad():
            h, y = _norm_plain(*(None if st[n] is None else st[n].float() for n in names), st["alpha"],
                               case["norm"])
            return {"h": h.to(dt), "y": y.to(dt)}
    leaves = {n: _leaf(st[n]) for n in names if st[n] is not None}
    h, y = _norm_plain(*(leaves.get(n) for n in names), st["alpha"], case["norm"])
    d = torch.autograd.grad([h, y], list(leaves.values()), [st["dh"].float(), st["dy"].float()])
    out = dict(zip(leaves, d))
    return {"d" + n: (g.to(dt) if n in ("x", "f") else g) for n, g in out.items()}


# ------------------------------------------------------- the library's calls

def _run_own(st, case):
    import linear_attention_diffusion_b200 as la
    if case["op"] == "gated":
        O, S = la.gated_attention(st["Q"], st["K"], st["V"], st["G"], S_in=st["S"], scale=st["scale"],
                                  want_state=True)
        return {"O": O, "S": S}
    if case["op"] == "gated_bwd":
        dQ, dK, dV, dG, dS = la.gated_attention_backward(
            st["Q"], st["K"], st["V"], st["G"], st["dO"], S_in=st["S"], dS_out=st["dS"],
            scale=st["scale"])
        out = {"dQ": dQ, "dK": dK, "dV": dV, "dG": dG}
        if dS is not None:
            out["dS"] = dS
        return out
    if case["op"] == "rotary":
        Q, K = la.rotary(st["Q"], st["K"], positions=st["pos"], rot=case["rot"], layout=case["layout"],
                         scaling=st["scaling"], mscale=st["mscale"], inverse=case["inverse"])
        return {"Q": Q} if K is None else {"Q": Q, "K": K}
    params = {n: st[n] for n in ("gate", "w_post", "w_pre", "mod_scale", "mod_shift")}
    if case["op"] == "norm":
        h, y = la.gate_residual_norm(st["x"], st["f"], **params, norm=case["norm"], alpha=st["alpha"])
        return {"h": h, "y": y}
    d = la.gate_residual_norm_backward(st["x"], st["f"], st["dy"], st["dh"], **params, norm=case["norm"],
                                       alpha=st["alpha"])
    names = ("x", "f", "gate", "w_post", "w_pre", "mod_scale", "mod_shift")
    return {"d" + n: g for n, g in zip(names, d) if g is not None}


# --------------------------------------------- the definitions, in 64 bits

def _gated_exact(st, case):
    """Token by token: S_n = a_n S_{n-1} + k_n^T v_n, o_n = scale q_n S_n; then
    the adjoint recurrence backwards."""
    q, k, v = (st[n].double() for n in ("Q", "K", "V"))
    a = torch.exp(st["G"].double())
    B, N, H, _ = q.shape
    scale = st["scale"]
    S = torch.zeros(B, H, D, D, device=q.device, dtype=torch.float64) if st["S"] is None else st["S"].double()
    back = case["op"] == "gated_bwd"
    past = torch.empty((N,) + S.shape, device=q.device, dtype=torch.float64) if back else None
    O = torch.empty_like(q)
    for n in range(N):
        if back:
            past[n] = S
        S = a[:, n, :, None, None] * S + k[:, n, :, :, None] * v[:, n, :, None, :]
        if not back:
            O[:, n] = scale * (q[:, n, :, None, :] @ S)[:, :, 0]
    if not back:
        return {"O": O, "S": S}
    dO = st["dO"].double() * scale
    dS = torch.zeros_like(S) if st["dS"] is None else st["dS"].double()
    dQ, dK, dV, dG = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q), torch.empty_like(a)
    for n in range(N - 1, -1, -1):
        dQ[:, n] = (S @ dO[:, n, :, :, None])[..., 0]
        dS = dS + q[:, n, :, :, None] * dO[:, n, :, None, :]
        dK[:, n] = (dS @ v[:, n, :, :, None])[..., 0]
        dV[:, n] = (k[:, n, :, None, :] @ dS)[:, :, 0]
        S = past[n]
        dS = a[:, n, :, None, None] * dS
        dG[:, n] = (dS * S).sum((-1, -2))
    out = {"dQ": dQ, "dK": dK, "dV": dV, "dG": dG}
    if st["S"] is not None:
        out["dS"] = dS
    return out


def _rotary_exact(st, case):
    """Each pair as a complex number times exp(i angle)."""
    rot, half = case["rot"], case["rot"] // 2
    rates = []
    for j in range(half):
        base = 10000.0
        kind = st["scaling"]
        if kind and kind[0] == "base" and rot > 2:
            base = 10000.0 * kind[1] ** (rot / (rot - 2))
        r = base ** (-2.0 * j / rot)
        if kind and kind[0] == "linear":
            r /= kind[1]
        elif kind and kind[0] == "parts":
            _, factor, length, slow, fast = kind
            w = min(1.0, max(0.0, (length * r / (2.0 * math.pi) - slow) / (fast - slow)))
            r = (1.0 - w) * r / factor + w * r
        rates.append(r)
    angle = st["pos"].double()[:, :, None] * torch.tensor(rates, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, st["mscale"]), -angle if case["inverse"] else angle)
    first = [2 * j if case["layout"] == "interleaved" else j for j in range(half)]
    second = [2 * j + 1 if case["layout"] == "interleaved" else j + half for j in range(half)]
    out = {}
    for name in ("Q", "K"):
        if st[name] is not None:
            y = st[name].double().clone()
            z = torch.complex(y[..., first], y[..., second]) * turn[:, :, None]
            y[..., first], y[..., second] = z.real, z.imag
            out[name] = y
    return out


def _norm_exact(st, case, eps=1e-6):
    """h and y, and their gradients by the chain rule, row by row of the formulas."""
    x, f = st["x"].double(), st["f"].double()
    C = x.shape[-1]
    one = torch.ones(1, 1, C, dtype=torch.float64, device=x.device)
    gate = one if st["gate"] is None else st["gate"].double()[:, None]
    wo = st["w_pre"].double()
    mul = one if st["mod_scale"] is None else 1.0 + st["mod_scale"].double()[:, None]
    add = 0.0 * one if st["mod_shift"] is None else st["mod_shift"].double()[:, None]
    al = st["alpha"]
    if st["w_post"] is None:
        fn, u = None, f
    else:
        rf = 1.0 / torch.sqrt(f.pow(2).sum(-1, keepdim=True) / C + eps)
        fn = f * rf
        u = fn * st["w_post"].double()
    h = x + al * gate * u
    mean = h.sum(-1, keepdim=True) / C if case["norm"] == "layer" else 0.0
    rh = 1.0 / torch.sqrt((h - mean).pow(2).sum(-1, keepdim=True) / C + eps)
    hn = (h - mean) * rh
    if case["op"] == "norm":
        return {"h": h, "y": hn * wo * mul + add}
    dy, dh = st["dy"].double(), st["dh"].double()
    t = dy * wo * mul
    back = t - hn * (t * hn).sum(-1, keepdim=True) / C
    if case["norm"] == "layer":
        back = back - t.sum(-1, keepdim=True) / C
    dh = dh + rh * back
    du = al * gate * dh
    out = {"dx": dh, "df": du}
    if fn is not None:
        t = du * st["w_post"].double()
        out["df"] = rf * (t - fn * (t * fn).sum(-1, keepdim=True) / C)
    if st["gate"] is not None:
        out["dgate"] = al * (u * dh).sum(1)
    if fn is not None:
        out["dw_post"] = (du * fn).sum((0, 1))
    out["dw_pre"] = (dy * mul * hn).sum((0, 1))
    if st["mod_scale"] is not None:
        out["dmod_scale"] = (dy * hn * wo).sum(1)
        out["dmod_shift"] = dy.sum(1)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    with torch.no_grad():
        if case["op"] in ("gated", "gated_bwd"):
            return _gated_exact(st, case)
        if case["op"] == "rotary":
            return _rotary_exact(st, case)
        return _norm_exact(st, case)
