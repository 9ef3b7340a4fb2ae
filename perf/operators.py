"""Cases of the sequence-mixer operators: what is timed and compared, and their plain forms.

Three operators sit around the quaternion scan:

* ``norm_rotate``: the norm of queries and keys for each head, and their rotation by the
  conjugate of the cumulative quaternion, in one pass (forward and backward);
* ``delta``: the gated delta rule over whole sequences, chunked (forward; forward and backward);
* ``step``: the gated delta rule for single tokens, on states that stay in a pool.

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits, with
``own`` true through the framework's calls.
"""
import math

import torch

own = False

CHUNK = 64   # steps per chunk of the plain chunked form (and of the chunk carries)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def _rot(name, grad, B, S, H, Hq, Hk, D, J, dt, cum, norm, weights):
    return {"name": name, "op": "norm_rotate", "grad": grad, "B": B, "S": S, "H": H, "Hq": Hq, "Hk": Hk, "D": D,
            "J": J, "dt": dt, "cum": cum, "norm": norm, "weights": weights}


def _delta(name, grad, B, S, Hk, Hv, Dk, Dv, dt, gates, packed=0, init=False):
    return {"name": name, "op": "delta", "grad": grad, "B": B, "S": S, "Hk": Hk, "Hv": Hv, "Dk": Dk, "Dv": Dv,
            "dt": dt, "gates": gates, "packed": packed, "init": init}


def _step(name, N, T, Hk, Hv, Dk, Dv, dt, gates, pool, idle):
    return {"name": name, "op": "step", "N": N, "T": T, "Hk": Hk, "Hv": Hv, "Dk": Dk, "Dv": Dv, "dt": dt,
            "gates": gates, "pool": pool, "idle": idle}


def listed():
    return [
        # One token of eight sequences while serving: latency alone.
        _rot("rotate fwd token", False, 8, 1, 16, 16, 16, 128, 32, "bf16", "f32", "rms", True),
        # The mamba3 workload (8 x 4096 x 16 x 32 quaternions): a training step's forward.
        _rot("rotate fwd mamba3", False, 8, 4096, 16, 16, 16, 128, 32, "bf16", "f32", "l2", False),
        # The small workload in 32 bits: a step of a small model, forward and backward.
        _rot("rotate bwd small", True, 4, 1024, 8, 8, 8, 64, 16, "f32", "f32", "rms", True),
        # Shared key heads, a rotation of part of the head, an odd length: gradients of shared rotations.
        _rot("rotate bwd shared", True, 2, 4099, 8, 32, 8, 96, 16, "bf16", "bf16", "rms", True),
        # Seventeen prompts of unequal length packed into one batch: prefill while serving.
        _delta("delta fwd packed", False, 1, 4333, 8, 16, 128, 128, "bf16", "f32", 17, True),
        # The mamba3 workload's forward.
        _delta("delta fwd mamba3", False, 8, 4096, 16, 16, 128, 128, "bf16", "f32"),
        # The long workload: few heads, one long sequence; the state's chain is the length.
        _delta("delta fwd long", False, 1, 131072, 16, 16, 64, 64, "bf16", "f32"),
        # The small workload in 32 bits, with an initial state and an odd length: a training step.
        _delta("delta train small", True, 4, 1000, 4, 8, 64, 64, "f32", "f32", 0, True),
        # The mamba3 workload: a training step, forward and backward.
        _delta("delta train mamba3", True, 8, 4096, 16, 16, 128, 128, "bf16", "bf16"),
        # One token of one sequence: latency alone.
        _step("delta step one", 1, 1, 16, 16, 128, 128, "bf16", "f32", 4, 0),
        # One token of a full batch of sequences, some of its rows idle.
        _step("delta step batch", 256, 1, 16, 32, 128, 128, "bf16", "f32", 300, 9),
        # Four tokens at once (checked drafts) of a smaller batch, in 32 bits.
        _step("delta step four", 48, 4, 8, 8, 64, 64, "f32", "f32", 64, 0),
    ]


def _spread(rng, low, high):
    """A whole number between the two, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["rotate fwd", "rotate bwd", "delta fwd", "delta train", "delta packed", "step"])
    dt = rng.choice(["f32", "bf16", "bf16"])
    if kind.startswith("rotate"):
        J = rng.choice([8, 16, 24, 32])
        D = rng.choice([4 * J, 4 * J, 4 * J + 32])
        H = rng.choice([1, 2, 4, 8, 16])
        Hk = H * rng.choice([1, 1, 2])
        Hq = Hk * rng.choice([1, 1, 4])
        tokens = _spread(rng, 1, min(32768, 2 ** 25 // (D * (Hq + Hk))))
        B = min(tokens, _spread(rng, 1, 8))
        return _unnamed(_rot("", kind == "rotate bwd", B, max(1, tokens // B), H, Hq, Hk, D, J, dt, rng.choice(["f32", dt]),
                             rng.choice(["rms", "l2"]), rng.random() < 0.6))
    Dk = rng.choice([64, 96, 128, 128])
    Dv = rng.choice([64, 128, 128])
    Hk = rng.choice([2, 4, 8, 16])
    Hv = Hk * rng.choice([1, 1, 2])
    if kind == "step":
        N = _spread(rng, 1, max(1, 256 * 32 * 128 * 128 // (Hv * Dk * Dv)) // 2)
        N = min(N, 512)
        idle = rng.randrange(0, max(1, N // 8))
        return _unnamed(_step("", N, rng.choice([1, 1, 2, 3, 5]), Hk, Hv, Dk, Dv, dt, "f32" if rng.random() < 0.7 else dt,
                              N + rng.randrange(0, 40), idle))
    most = 2 ** 22 // Hv if kind == "delta train" else 2 ** 25 // Hv   # token rows of all heads, over 8 (training) or 1
    tokens = _spread(rng, 40, min(65536, most // 8))
    if kind == "delta packed":
        return _unnamed(_delta("", False, 1, tokens, Hk, Hv, Dk, Dv, dt, "f32", _spread(rng, 2, min(24, tokens)), True))
    B = _spread(rng, 1, min(8, tokens))
    gates = "f32" if kind == "delta fwd" or dt == "f32" else "bf16"
    return _unnamed(_delta("", kind == "delta train", B, max(1, tokens // B), Hk, Hv, Dk, Dv, dt, gates, 0, rng.random() < 0.5))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def work(c):
    e = {"f32": 4, "bf16": 2}[c["dt"]]
    if c["op"] == "norm_rotate":
        rows = c["B"] * c["S"]
        x = rows * (c["Hq"] + c["Hk"]) * c["D"]                       # values of q and k together
        turn = rows * c["H"] * c["J"] * 4 * {"f32": 4, "bf16": 2}[c["cum"]]
        w = 2 * c["D"] * 4 if c["weights"] else 0
        if c["grad"]:   # q, k, their cotangents and the turns in; d_q, d_k, d_cum and the weights' gradients out
            return {"bytes": 3 * x * e + 2 * turn + 2 * w, "flops": 25 * x}
        return {"bytes": 2 * x * e + turn + w, "flops": 11 * x}
    ge = {"f32": 4, "bf16": 2}[c["gates"]]
    if c["op"] == "step":
        live = c["N"] - c["idle"]
        state = live * c["Hv"] * c["Dk"] * c["Dv"]
        tok = c["N"] * c["T"]
        return {"bytes": 2 * 4 * state + tok * (2 * c["Hk"] * c["Dk"] + 2 * c["Hv"] * c["Dv"]) * e + 2 * tok * c["Hv"] * ge,
                "flops": 7 * state * c["T"]}
    tok = c["B"] * c["S"]
    seqs = c["packed"] or c["B"]
    state = seqs * c["Hv"] * c["Dk"] * c["Dv"] * 4
    io = tok * (2 * c["Hk"] * c["Dk"] + 2 * c["Hv"] * c["Dv"]) * e + 2 * tok * c["Hv"] * ge
    one = tok * c["Hv"] * c["Dk"] * c["Dv"]
    if not c["grad"]:   # q, k, v, gates (and states) in; o and the final states out
        return {"bytes": io + state * (2 if c["init"] else 1), "flops": 7 * one}
    # the forward, then the cotangent in and five gradients out
    back = tok * (2 * c["Hk"] * c["Dk"] + 2 * c["Hv"] * c["Dv"]) * e + 2 * tok * c["Hv"] * ge
    return {"bytes": io + back + state * (4 if c["init"] else 2), "flops": 23 * one}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, dt = case, DT[case["dt"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if c["op"] == "norm_rotate":
        s = {"q": randn(c["B"], c["S"], c["Hq"], c["D"]).to(dt), "k": (1.5 * randn(c["B"], c["S"], c["Hk"], c["D"])).to(dt)}
        turn = randn(c["B"], c["S"], c["H"], c["J"], 4)
        s["cum"] = (turn / turn.norm(dim=-1, keepdim=True)).to(DT[c["cum"]])
        for w in ("w_q", "w_k"):
            s[w] = 1 + 0.2 * randn(c["D"]) if c["weights"] else None
        if c["grad"]:
            s["d_qo"], s["d_ko"] = randn(*s["q"].shape).to(dt), randn(*s["k"].shape).to(dt)
        return {"case": c, **s}

    B, T = (c["N"], c["T"]) if c["op"] == "step" else (c["B"], c["S"])

    def unit(*shape):   # as the norm before it leaves queries and keys
        x = randn(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s = {"q": unit(B, T, c["Hk"], c["Dk"]), "k": unit(B, T, c["Hk"], c["Dk"]), "v": randn(B, T, c["Hv"], c["Dv"]).to(dt)}
    rate = torch.exp(torch.linspace(math.log(0.005), math.log(2.0), c["Hv"], device="cuda"))   # slow and quick heads
    s["g"] = (-rate * torch.nn.functional.softplus(randn(B, T, c["Hv"]))).to(DT[c["gates"]])
    s["beta"] = torch.sigmoid(randn(B, T, c["Hv"])).to(DT[c["gates"]])
    if c["op"] == "step":
        order = torch.randperm(c["pool"], generator=gen, device="cuda")[: c["N"]]
        still = torch.randperm(c["N"], generator=gen, device="cuda")[: c["idle"]]
        order[still] = -1
        s["slots"] = order.to(torch.int32)
        s["state"] = 0.3 * randn(c["pool"], c["Hv"], c["Dk"], c["Dv"])
        return {"case": c, **s}
    seqs = c["packed"] or c["B"]
    s["init"] = 0.3 * randn(seqs, c["Hv"], c["Dk"], c["Dv"]) if c["init"] else None
    s["offsets"] = None
    if c["packed"]:
        cut = torch.sort(torch.randint(0, c["S"] + 1, (seqs - 1,), generator=gen, device="cuda"))[0]
        ends = torch.tensor([0, c["S"]], device="cuda")
        s["offsets"] = torch.cat([ends[:1], cut, ends[1:]]).to(torch.int32)
        s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    if c["grad"]:
        s["d_o"] = randn(B, T, c["Hv"], c["Dv"]).to(dt)
        s["d_final"] = 0.1 * randn(seqs, c["Hv"], c["Dk"], c["Dv"])
    return {"case": c, **s}


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------
def _plain_rotate(x, turn, w, norm):
    """The norm over the head, then conj(turn) times each of the first 4J values taken as quaternions."""
    D, H, J = x.shape[-1], turn.shape[2], turn.shape[3]
    total = (x * x).sum(-1, keepdim=True)
    n = x * torch.rsqrt((total / D if norm == "rms" else total) + 1e-6)
    if w is not None:
        n = n * w
    part = n[..., : 4 * J].reshape(*x.shape[:2], H, x.shape[2] // H, J, 4)
    a, b, c, d = part.unbind(-1)
    r, i, j, k = turn[:, :, :, None].unbind(-1)
    out = torch.stack([r * a + i * b + j * c + k * d, r * b - i * a - j * d + k * c,
                       r * c + i * d - j * a - k * b, r * d - i * c + j * b - k * a], -1)
    return torch.cat([out.reshape(*x.shape[:3], 4 * J), n[..., 4 * J:]], -1)


def _plain_norm_rotate(s):
    c = s["case"]
    names = ["q", "k", "cum"] + (["w_q", "w_k"] if c["weights"] else [])
    f = {n: s[n].float() for n in names}
    if c["grad"]:
        f = {n: t.detach().requires_grad_() for n, t in f.items()}
    with torch.set_grad_enabled(c["grad"]):
        qo = _plain_rotate(f["q"], f["cum"], f.get("w_q"), c["norm"])
        ko = _plain_rotate(f["k"], f["cum"], f.get("w_k"), c["norm"])
        if not c["grad"]:
            return {"q": qo.to(s["q"].dtype), "k": ko.to(s["k"].dtype)}
        grads = torch.autograd.grad([qo, ko], [f[n] for n in names], [s["d_qo"].float(), s["d_ko"].float()])
    return {"d_" + n: d.to(s[n].dtype) for n, d in zip(names, grads)}


def _inverse(a):
    """(1 + a)^-1 for strictly lower triangular a [.., 64, 64], from the inverses of its diagonal blocks."""
    t = torch.eye(CHUNK, device=a.device).expand_as(a).contiguous()
    n = 1
    while n < CHUNK:
        blocks = a.unflatten(-2, (CHUNK // (2 * n), 2 * n)).unflatten(-1, (CHUNK // (2 * n), 2 * n))
        here = torch.diagonal(blocks, dim1=-4, dim2=-2)[..., n:, :n, :].movedim(-1, -3)        # below the diagonal
        inv = torch.diagonal(t.unflatten(-2, (CHUNK // (2 * n), 2 * n)).unflatten(-1, (CHUNK // (2 * n), 2 * n)),
                             dim1=-4, dim2=-2).movedim(-1, -3)
        low = -(inv[..., n:, n:] @ here @ inv[..., :n, :n])
        top = torch.cat([inv[..., :n, :n], torch.zeros_like(low)], -1)
        block = torch.cat([top, torch.cat([low, inv[..., n:, n:]], -1)], -2)                     # [.., m, 2n, 2n]
        t = torch.diag_embed(block.movedim(-3, -1), dim1=-4, dim2=-2).flatten(-4, -3).flatten(-2, -1)
        n *= 2
    return t


def _plain_delta_rule(q, k, v, g, beta, init):
    """o and the final state for q (scaled), k [B,S,Hk,Dk], v [B,S,Hv,Dv], g, beta [B,S,Hv], chunked."""
    B, S, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    more = -S % CHUNK
    chunks = (S + more) // CHUNK

    def lay(x):   # [B,Hv,chunks,64,..], padded with zeros
        x = x.repeat_interleave(Hv // x.shape[2], 2) if x.shape[2] != Hv else x
        x = torch.cat([x, x.new_zeros(B, more, *x.shape[2:])], 1) if more else x
        return x.unflatten(1, (chunks, CHUNK)).movedim(3, 1)

    q, k, v, g, beta = (lay(x) for x in (q, k, v, g, beta))
    total = g.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = (total[..., :, None] - total[..., None, :]).masked_fill(~low, -math.inf).exp()
    grown = total.exp()[..., None]
    a = (k @ k.mT) * decay * beta[..., None]
    t = _inverse(a.masked_fill(torch.eye(CHUNK, dtype=torch.bool, device=q.device), 0.0))
    rhs = t @ (beta[..., None] * torch.cat([v, grown * k], -1))
    u0, w = rhs[..., :Dv], rhs[..., Dv:]
    kept = k * (total[..., -1:] - total).exp()[..., None]
    last = total[..., -1].exp()[..., None, None]
    state = torch.zeros(B, Hv, Dk, Dv, device=q.device) if init is None else init
    states, us = [], []
    for i in range(chunks):   # the state's chain: one chunk needs the last one's
        states.append(state)
        us.append(u0[:, :, i] - w[:, :, i] @ state)
        state = last[:, :, i] * state + kept[:, :, i].mT @ us[i]
    us, states = torch.stack(us, 2), torch.stack(states, 2)
    o = grown * (q @ states) + ((q @ k.mT) * decay) @ us
    return o.movedim(1, 3).flatten(1, 2)[:, :S], state


def _plain_delta(s):
    c = s["case"]
    names = ["q", "k", "v", "g", "beta"]
    f = {n: s[n].float() for n in names}
    if c["init"]:
        names.append("init")
        f["init"] = s["init"]
    if c["grad"]:
        f = {n: t.detach().requires_grad_() for n, t in f.items()}
    scale = c["Dk"] ** -0.5
    if c["packed"]:   # one row per sequence, short ones filled up with steps that change nothing
        off = s["offsets"].long()
        at = off[:-1, None] + torch.arange(s["longest"], device=off.device)
        inside = at < off[1:, None]
        at = at.clamp(max=c["S"] - 1)
        rows = {n: f[n][0][at] * inside.reshape(*at.shape, *[1] * (f[n].dim() - 2)) for n in names[:5]}
        o, final = _plain_delta_rule(rows["q"] * scale, rows["k"], rows["v"], rows["g"], rows["beta"], f.get("init"))
        out = torch.empty(1, c["S"], c["Hv"], c["Dv"], device=o.device)
        out[0, at[inside]] = o[inside]
        return {"o": out.to(s["v"].dtype), "final": final}
    with torch.set_grad_enabled(c["grad"]):
        o, final = _plain_delta_rule(f["q"] * scale, f["k"], f["v"], f["g"], f["beta"], f.get("init"))
        if not c["grad"]:
            return {"o": o.to(s["v"].dtype), "final": final}
        grads = torch.autograd.grad([o, final], [f[n] for n in names], [s["d_o"].float(), s["d_final"]])
    return {"o": o.detach().to(s["v"].dtype), "final": final.detach(), **{"d_" + n: d.to(s[n].dtype) for n, d in zip(names, grads)}}


def _plain_step(s):
    c = s["case"]
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    slots = s["slots"][live].long()
    shared = c["Hv"] // c["Hk"]
    q, k, v = (s[n][live].float() for n in ("q", "k", "v"))
    q, k = q.repeat_interleave(shared, 2) * c["Dk"] ** -0.5, k.repeat_interleave(shared, 2)
    alpha, beta = s["g"][live].float().exp(), s["beta"][live].float()
    state = s["state"][slots]
    o = torch.zeros(c["N"], c["T"], c["Hv"], c["Dv"], device=v.device)
    for t in range(c["T"]):   # each token's state needs the last one's
        state = state * alpha[:, t, :, None, None]
        err = v[:, t] - (state * k[:, t, ..., None]).sum(-2)
        state = state + k[:, t, ..., None] * (beta[:, t, :, None] * err)[..., None, :]
        o[live, t] = (state * q[:, t, ..., None]).sum(-2)
    s["state"][slots] = state
    return {"o": o.to(s["v"].dtype), "state": s["state"]}


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm_rotate": _plain_norm_rotate, "delta": _plain_delta, "step": _plain_step}[c["op"]](s)
    import quaternion_cumulative_product_gb300 as qs

    if c["op"] == "norm_rotate":
        if not c["grad"]:
            q, k = qs.quat_norm_rotate_fwd(s["q"], s["k"], s["cum"], s["w_q"], s["w_k"], norm=c["norm"], eps=1e-6)
            return {"q": q, "k": k}
        d = qs.quat_norm_rotate_bwd(s["q"], s["k"], s["cum"], s["d_qo"], s["d_ko"], s["w_q"], s["w_k"], norm=c["norm"], eps=1e-6)
        return {"d_" + n: x for n, x in zip(["q", "k", "cum", "w_q", "w_k"], d) if x is not None}
    if c["op"] == "step":
        o = qs.quat_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
        return {"o": o, "state": s["state"]}
    five = [s[n] for n in ("q", "k", "v", "g", "beta")]
    if not c["grad"]:
        o, final = qs.quat_delta_fwd(*five, s["init"], offsets=s["offsets"])
        return {"o": o, "final": final}
    o, final, carries, errors = qs.quat_delta_fwd_carries(*five, s["init"])
    d = qs.quat_delta_bwd(*five, carries, errors, s["d_o"], s["d_final"])
    names = ["q", "k", "v", "g", "beta"] + (["init"] if c["init"] else [])
    return {"o": o, "final": final, **{"d_" + n: x for n, x in zip(names, d)}}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits, token by token
# ---------------------------------------------------------------------------------------------
#: Conjugate-left multiplication: row m, column n of the matrix of conj(r) is SIGN[m][n] * r[WHICH[m][n]].
WHICH = [[0, 1, 2, 3], [1, 0, 3, 2], [2, 3, 0, 1], [3, 2, 1, 0]]
SIGN = [[1, 1, 1, 1], [-1, 1, 1, -1], [-1, -1, 1, 1], [-1, 1, -1, 1]]


def _exact_rotate(c, s):
    out = {}
    H, J, D = c["H"], c["J"], c["D"]
    which, sign = torch.tensor(WHICH, device="cuda"), torch.tensor(SIGN, device="cuda", dtype=torch.float64)
    turn = s["cum"].double()
    m = turn[..., which] * sign                                                     # [B,S,H,J,4,4]
    d_m = 0
    for n in ("q", "k"):
        x = s[n].double()
        w = s["w_" + n].double() if c["weights"] else torch.ones(D, device="cuda", dtype=torch.float64)
        div = D if c["norm"] == "rms" else 1
        r = ((x * x).sum(-1, keepdim=True) / div + 1e-6) ** -0.5
        y = x * r * w
        heads = (*x.shape[:2], H, x.shape[2] // H)
        part = y[..., : 4 * J].reshape(*heads, J, 4)
        if not c["grad"]:
            z = torch.einsum("bshjmn,bshgjn->bshgjm", m, part).reshape(*x.shape[:3], 4 * J)
            out[n] = torch.cat([z, y[..., 4 * J:]], -1)
            continue
        dz = s["d_%so" % n].double()
        dpart = dz[..., : 4 * J].reshape(*heads, J, 4)
        dy = torch.cat([torch.einsum("bshjmn,bshgjm->bshgjn", m, dpart).reshape(*x.shape[:3], 4 * J), dz[..., 4 * J:]], -1)
        d_m = d_m + torch.einsum("bshgjm,bshgjn->bshjmn", dpart, part)
        if c["weights"]:
            out["d_w_" + n] = (dy * x * r).sum((0, 1, 2))
        dn = dy * w
        out["d_" + n] = dn * r - x * r ** 3 * (dn * x).sum(-1, keepdim=True) / div
    if c["grad"]:
        d_turn = torch.zeros_like(turn)
        for a in range(4):
            for b in range(4):
                d_turn[..., WHICH[a][b]] += SIGN[a][b] * d_m[..., a, b]
        out["d_cum"] = d_turn
    return out


def _exact_delta(c, s):
    seqs, Hv, Dk, Dv = c["packed"] or c["B"], c["Hv"], c["Dk"], c["Dv"]
    shared = Hv // c["Hk"]
    q, k, v, g, beta = (s[n].double() for n in ("q", "k", "v", "g", "beta"))
    q, k = (x.repeat_interleave(shared, 2) for x in (q * Dk ** -0.5, k))
    state = torch.zeros(seqs, Hv, Dk, Dv, device="cuda", dtype=torch.float64)
    if c["init"]:
        state += s["init"]
    if c["packed"]:   # one sequence after the other, token by token; sequences in step with one another
        off = s["offsets"].tolist()
        length = [b - a for a, b in zip(off, off[1:])]
        o = torch.zeros(1, c["S"], Hv, Dv, device="cuda", dtype=torch.float64)
        offs = torch.tensor(off, device="cuda")
        for t in range(max(length)):
            on = torch.tensor([i for i in range(seqs) if length[i] > t], device="cuda")
            at = offs[on] + t
            st = state[on] * g[0, at].exp()[..., None, None]
            err = v[0, at] - torch.einsum("nhk,nhkv->nhv", k[0, at], st)
            st = st + k[0, at][..., None] * (beta[0, at][..., None] * err)[..., None, :]
            o[0, at] = torch.einsum("nhk,nhkv->nhv", q[0, at], st)
            state[on] = st
        return {"o": o, "final": state}
    o = torch.empty(*v.shape, device="cuda", dtype=torch.float64)
    S, every = c["S"], 64
    alpha = g.exp()[..., None, None]
    marks = []

    def forward(state, t):
        kept = state * alpha[:, t]
        err = v[:, t] - (k[:, t, :, None] @ kept)[:, :, 0]
        return kept, err, torch.baddbmm(kept.flatten(0, 1), k[:, t].flatten(0, 1)[..., None],
                                        (beta[:, t, :, None] * err).flatten(0, 1)[:, None]).view_as(kept)

    for t in range(S):
        if c["grad"] and t % every == 0:
            marks.append(state)
        state = forward(state, t)[2]
        o[:, t] = (q[:, t, :, None] @ state)[:, :, 0]
    out = {"o": o, "final": state}
    if not c["grad"]:
        return out
    d_o = s["d_o"].double()
    d = {n: torch.empty_like(x) for n, x in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta))}
    ds = s["d_final"].double()
    for m in reversed(range(len(marks))):
        steps, kept_of = range(m * every, min(S, (m + 1) * every)), []
        st = marks[m]
        for t in steps:
            kept, err, st = forward(st, t)
            kept_of.append((kept, err, st))
        for t in reversed(steps):
            kept, err, st = kept_of.pop()
            do, kt, b = d_o[:, t, :, None], k[:, t, :, None], beta[:, t, :, None]
            ds = ds + q[:, t, ..., None] * do
            d["q"][:, t] = (st @ do.mT)[..., 0]
            du = (kt @ ds)[:, :, 0]
            de = b * du
            d["beta"][:, t] = (err * du).sum(-1)
            d["v"][:, t] = de
            d["k"][:, t] = (ds @ (b * err)[..., None])[..., 0] - (kept @ de[..., None])[..., 0]
            ds = ds - k[:, t, ..., None] * de[:, :, None]
            d["g"][:, t] = (ds * kept).sum((-1, -2))
            ds = ds * alpha[:, t]
    d["q"] *= Dk ** -0.5
    for n in ("q", "k"):
        d[n] = d[n].unflatten(2, (c["Hk"], shared)).sum(3)
    if c["init"]:
        d["init"] = ds
    return {**out, **{"d_" + n: x for n, x in d.items()}}


def _exact_step(c, s):
    shared = c["Hv"] // c["Hk"]
    state = s["state"].double()
    o = torch.zeros(c["N"], c["T"], c["Hv"], c["Dv"], device="cuda", dtype=torch.float64)
    on = torch.tensor([i for i, x in enumerate(s["slots"].tolist()) if x >= 0], device="cuda")
    at = s["slots"].long()[on]
    head = torch.arange(c["Hv"], device="cuda") // shared
    st = state[at]
    for t in range(c["T"]):
        kt, qt = (s[n][on, t].double()[:, head] for n in ("k", "q"))
        st = st * s["g"][on, t].double().exp()[..., None, None]
        err = s["v"][on, t].double() - torch.einsum("nhk,nhkv->nhv", kt, st)
        st = st + torch.einsum("nhk,nhv->nhkv", kt, s["beta"][on, t].double()[..., None] * err)
        o[on, t] = torch.einsum("nhk,nhkv->nhv", qt * c["Dk"] ** -0.5, st)
    state[at] = st
    return {"o": o, "state": state}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "delta" and case["S"] * max(case["grad"] * 6, 1) > 140000:
        return None   # too many steps one after the other
    return {"norm_rotate": _exact_rotate, "delta": _exact_delta, "step": _exact_step}[case["op"]](case, s)
