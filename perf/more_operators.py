"""Cases of the operators of a residual block around the scan, and their plain forms.

* ``norm``: layer norm over the model's width, forward and backward (the block's input);
* ``decay``: linear attention with a decay for each head over whole sequences, equal or packed
  (forward; forward and backward): the state ``M_t = exp(g_t) M_{t-1} + k_t v_t^T`` read by
  ``o_t = scale M_t^T q_t``;
* ``step``: the same recurrence for single tokens, on states that stay in a pool;
* ``dropout``: dropout from a counter-based generator (Philox4x32-10), added on the residual,
  and its gradient, which makes the mask again.

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits, with
``own`` true through the framework's calls.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64   # steps per chunk of the plain chunked form
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def _norm(name, grad, B, S, D, dt, weights, beside=0):
    """``beside``: columns of a joint projection next to the normed ones (its rows are then apart)."""
    return {"name": name, "op": "norm", "grad": grad, "B": B, "S": S, "D": D, "dt": dt, "weights": weights, "beside": beside}


def _dropout(name, grad, B, S, D, dt, p, residual):
    return {"name": name, "op": "dropout", "grad": grad, "B": B, "S": S, "D": D, "dt": dt, "p": p, "residual": residual}


def _decay(name, grad, B, S, Hk, Hv, Dk, Dv, dt, gates, packed=0, init=False):
    return {"name": name, "op": "decay", "grad": grad, "B": B, "S": S, "Hk": Hk, "Hv": Hv, "Dk": Dk, "Dv": Dv,
            "dt": dt, "gates": gates, "packed": packed, "init": init}


def _step(name, N, T, Hk, Hv, Dk, Dv, dt, gates, pool, idle):
    return {"name": name, "op": "step", "N": N, "T": T, "Hk": Hk, "Hv": Hv, "Dk": Dk, "Dv": Dv, "dt": dt,
            "gates": gates, "pool": pool, "idle": idle}


def listed():
    return [
        # One token of eight sequences while serving: latency alone.
        _norm("norm fwd token", False, 8, 1, 2048, "bf16", True),
        # The mamba3 workload (8 x 4096 tokens, 16 heads of 128 = a width of 2048): a training step's forward.
        _norm("norm fwd mamba3", False, 8, 4096, 2048, "bf16", True),
        # ... and its backward.
        _norm("norm bwd mamba3", True, 8, 4096, 2048, "bf16", True),
        # An odd width out of a joint projection, an odd length, 32 bits.
        _norm("norm bwd odd", True, 2, 4099, 1001, "f32", True, 24),
        # A small model's step in 32 bits: an odd number of values, without a residual.
        _dropout("dropout train small", True, 3, 1001, 511, "f32", 0.25, False),
        # The mamba3 workload: the mixer's output onto the residual, and its gradient.
        _dropout("dropout train mamba3", True, 8, 4096, 2048, "bf16", 0.1, True),
        # Seventeen prompts of unequal length packed into one batch: prefill while serving.
        _decay("decay fwd packed", False, 1, 4333, 8, 16, 128, 128, "bf16", "f32", 17, True),
        # The long workload: few heads, one long sequence.
        _decay("decay fwd long", False, 1, 131072, 16, 16, 64, 64, "bf16", "f32"),
        # The small workload in 32 bits, with an initial state and an odd length: a training step.
        _decay("decay train small", True, 4, 1000, 4, 8, 64, 64, "f32", "f32", 0, True),
        # The mamba3 workload: a training step, forward and backward.
        _decay("decay train mamba3", True, 8, 4096, 16, 16, 128, 128, "bf16", "f32"),
        # One token of one sequence: latency alone.
        _step("decay step one", 1, 1, 16, 16, 128, 128, "bf16", "f32", 4, 0),
        # One token of a full batch of sequences, some of its rows idle.
        _step("decay step batch", 256, 1, 16, 32, 128, 128, "bf16", "f32", 300, 9),
    ]


def _spread(rng, low, high):
    """A whole number between the two, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["norm fwd", "norm bwd", "dropout", "decay fwd", "decay train", "decay packed", "step"])
    dt = rng.choice(["f32", "bf16", "bf16"])
    if kind.startswith("norm") or kind == "dropout":
        D = _spread(rng, 32, 8192)
        if rng.random() < 0.6:
            D = -(-D // 64) * 64
        tokens = _spread(rng, 1, max(1, min(32768, 2 ** 25 // D)))
        B = min(tokens, _spread(rng, 1, 8))
        S = max(1, tokens // B)
        if kind == "dropout":
            return _unnamed(_dropout("", rng.random() < 0.7, B, S, D, dt, rng.choice([0.05, 0.1, 0.25, 0.5]), rng.random() < 0.6))
        return _unnamed(_norm("", kind == "norm bwd", B, S, D, dt, rng.random() < 0.8, rng.choice([0, 0, 0, 64, 17])))
    Dk = rng.choice([32, 64, 96, 128, 128])
    Dv = rng.choice([64, 80, 128, 128])
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hv = Hk * rng.choice([1, 1, 2])
    if kind == "step":
        N = min(_spread(rng, 1, max(1, 256 * 32 * 128 * 128 // (Hv * Dk * Dv)) // 2), 512)
        idle = rng.randrange(0, max(1, N // 8))
        return _unnamed(_step("", N, rng.choice([1, 1, 2, 3, 5]), Hk, Hv, Dk, Dv, dt, "f32" if rng.random() < 0.7 else dt,
                              N + rng.randrange(0, 40), idle))
    most = 2 ** 22 // Hv if kind == "decay train" else 2 ** 25 // Hv   # token rows of all heads, over 8 (training) or 1
    tokens = _spread(rng, 40, min(65536, most // 8))
    if kind == "decay packed":
        return _unnamed(_decay("", False, 1, tokens, Hk, Hv, Dk, Dv, dt, "f32", _spread(rng, 2, min(24, tokens)), True))
    B = _spread(rng, 1, min(8, tokens))
    gates = "f32" if dt == "f32" or rng.random() < 0.6 else "bf16"
    return _unnamed(_decay("", kind == "decay train", B, max(1, tokens // B), Hk, Hv, Dk, Dv, dt, gates, 0, rng.random() < 0.5))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def work(c):
    e = BYTES[c["dt"]]
    if c["op"] == "norm":
        x = c["B"] * c["S"] * c["D"]
        w = 2 * c["D"] * 4 if c["weights"] else 0
        if c["grad"]:   # x and the cotangent in, d_x and the weights' gradients out
            return {"bytes": 3 * x * e + (w // 2 + w if c["weights"] else 0), "flops": 16 * x}
        return {"bytes": 2 * x * e + w, "flops": 8 * x}
    if c["op"] == "dropout":
        x = c["B"] * c["S"] * c["D"]
        one = (3 if c["residual"] else 2) * x * e
        return {"bytes": one + (2 * x * e if c["grad"] else 0) + 16, "flops": (4 if c["grad"] else 2) * x}
    ge = BYTES[c["gates"]]
    if c["op"] == "step":
        live = c["N"] - c["idle"]
        state = live * c["Hv"] * c["Dk"] * c["Dv"]
        tok = c["N"] * c["T"]
        return {"bytes": 2 * 4 * state + tok * (2 * c["Hk"] * c["Dk"] + 2 * c["Hv"] * c["Dv"]) * e + tok * c["Hv"] * ge,
                "flops": 5 * state * c["T"]}
    tok = c["B"] * c["S"]
    state = (c["packed"] or c["B"]) * c["Hv"] * c["Dk"] * c["Dv"] * 4
    io = tok * (2 * c["Hk"] * c["Dk"] + 2 * c["Hv"] * c["Dv"]) * e + tok * c["Hv"] * ge
    one = tok * c["Hv"] * c["Dk"] * c["Dv"]
    if not c["grad"]:   # q, k, v, gates (and states) in; o and the final states out
        return {"bytes": io + state * (2 if c["init"] else 1), "flops": 5 * one}
    # the forward, then its cotangents in and the gradients out
    return {"bytes": 2 * io + state * (4 if c["init"] else 2), "flops": 17 * one}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, dt = case, DT[case["dt"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if c["op"] == "norm":   # a residual stream: features of unequal size, some far from zero
        size, middle = torch.exp(0.5 * randn(c["D"] + c["beside"])), 0.5 * randn(c["D"] + c["beside"])
        x = (randn(c["B"], c["S"], c["D"] + c["beside"]) * size + middle).to(dt)[..., : c["D"]]
        w, b = (1 + 0.2 * randn(c["D"]), 0.2 * randn(c["D"])) if c["weights"] else (None, None)
        s = {"x": x, "w": w, "b": b}
        if c["grad"]:
            s["d_y"] = randn(c["B"], c["S"], c["D"]).to(dt)
        return {"case": c, **s}
    if c["op"] == "dropout":
        s = {"x": randn(c["B"], c["S"], c["D"]).to(dt)}
        s["residual"] = (2 * randn(c["B"], c["S"], c["D"])).to(dt) if c["residual"] else None
        s["d_y"] = randn(c["B"], c["S"], c["D"]).to(dt) if c["grad"] else None
        # (seed, offset): any 64-bit numbers; a training program counts the offset up call by call
        s["key"] = torch.randint(-2 ** 62, 2 ** 62, (2,), generator=gen, device="cuda", dtype=torch.int64)
        return {"case": c, **s}

    B, T = (c["N"], c["T"]) if c["op"] == "step" else (c["B"], c["S"])

    def unit(*shape):   # as the norm before it leaves queries and keys
        x = randn(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s = {"q": unit(B, T, c["Hk"], c["Dk"]), "k": unit(B, T, c["Hk"], c["Dk"]), "v": randn(B, T, c["Hv"], c["Dv"]).to(dt)}
    rate = torch.exp(torch.linspace(math.log(0.005), math.log(2.0), c["Hv"], device="cuda"))   # slow and quick heads
    s["g"] = (-rate * torch.nn.functional.softplus(randn(B, T, c["Hv"]))).to(DT[c["gates"]])
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
EPS = 1e-5


def _plain_norm(s):
    x = s["x"].float()
    x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    if not s["case"]["grad"]:
        y = n if s["w"] is None else n * s["w"] + s["b"]
        return {"y": y.to(s["x"].dtype)}
    d_y = s["d_y"].float()
    d_n = d_y if s["w"] is None else d_y * s["w"]
    d_x = r * (d_n - d_n.mean(-1, keepdim=True) - n * (d_n * n).mean(-1, keepdim=True))
    out = {"d_x": d_x.to(s["x"].dtype)}
    if s["w"] is not None:
        out |= {"d_w": (d_y * n).flatten(0, 1).sum(0), "d_b": d_y.flatten(0, 1).sum(0)}
    return out


def _plain_words(key, count):
    """32-bit words 0 .. count-1 of Philox4x32-10: word i is word i % 4 of the counter (i // 4, offset) under the seed."""
    low = 0xFFFFFFFF
    block = torch.arange((count + 3) // 4, device=key.device)
    zero = torch.zeros_like(block)
    c = [block & low, block >> 32, zero + (key[1] & low), zero + ((key[1] >> 32) & low)]
    k0, k1 = key[0] & low, (key[0] >> 32) & low

    def product(a, m):   # (high, low) halves of a 32 x 32 bit product
        return (a * (m >> 16) + ((a * (m & 0xFFFF)) >> 16)) >> 16, (a * m) & low

    for _ in range(10):
        h0, l0 = product(c[0], 0xD2511F53)
        h1, l1 = product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack(c, -1).flatten()[:count]


def _plain_dropout(s):
    p = s["case"]["p"]
    keep = (_plain_words(s["key"], s["x"].numel()) >= int(p * 2 ** 32)).view(s["x"].shape)
    y = torch.where(keep, s["x"].float() * (1 / (1 - p)), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(s["x"].dtype)}
    if s["d_y"] is not None:
        out["d_x"] = torch.where(keep, s["d_y"].float() * (1 / (1 - p)), 0.0).to(s["x"].dtype)
    return out


def _plain_decay_rule(q, k, v, g, init):
    """o and the final state for q (scaled), k [B,S,Hk,Dk], v [B,S,Hv,Dv], g [B,S,Hv], chunked."""
    B, S, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    more = -S % CHUNK
    chunks = (S + more) // CHUNK

    def lay(x):   # [B,Hv,chunks,64,..], padded with zeros
        x = x.repeat_interleave(Hv // x.shape[2], 2) if x.shape[2] != Hv else x
        x = torch.cat([x, x.new_zeros(B, more, *x.shape[2:])], 1) if more else x
        return x.unflatten(1, (chunks, CHUNK)).movedim(3, 1)

    q, k, v = (lay(x) for x in (q, k, v))
    total = lay(g.double()).cumsum(-1)   # sums of logarithms, and their differences, in 64 bits
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = (total[..., :, None] - total[..., None, :]).float().masked_fill(~low, -math.inf).exp()
    o = ((q @ k.mT) * decay) @ v
    kept = k * (total[..., -1:] - total).float().exp()[..., None]
    added = (kept.mT @ v).flatten(-2)                                     # each chunk's part of the state at its end
    ends = total[..., -1].cumsum(-1)                                      # [B,Hv,chunks]
    begins = torch.cat([torch.zeros_like(ends[..., :1]), ends], -1)       # ... to the beginning of a chunk, and to the end of all
    before = torch.ones(chunks + 1, chunks, dtype=torch.bool, device=q.device).tril(-1)
    reach = (begins[..., :, None] - ends[..., None, :]).float().masked_fill(~before, -math.inf).exp()
    states = (reach @ added).unflatten(-1, (Dk, Dv))
    if init is not None:
        states = states + begins.float().exp()[..., None, None] * init[:, :, None]
    o = o + total.float().exp()[..., None] * (q @ states[:, :, :-1])
    return o.movedim(1, 3).flatten(1, 2)[:, :S], states[:, :, -1]


def _plain_decay(s):
    c = s["case"]
    names = ["q", "k", "v", "g"]
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
        rows = {n: f[n][0][at] * inside.reshape(*at.shape, *[1] * (f[n].dim() - 2)) for n in names[:4]}
        o, final = _plain_decay_rule(rows["q"] * scale, rows["k"], rows["v"], rows["g"], f.get("init"))
        out = torch.empty(1, c["S"], c["Hv"], c["Dv"], device=o.device)
        out[0, at[inside]] = o[inside]
        return {"o": out.to(s["v"].dtype), "final": final}
    with torch.set_grad_enabled(c["grad"]):
        o, final = _plain_decay_rule(f["q"] * scale, f["k"], f["v"], f["g"], f.get("init"))
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
    alpha = s["g"][live].float().exp()
    state = s["state"][slots]
    o = torch.zeros(c["N"], c["T"], c["Hv"], c["Dv"], device=v.device)
    for t in range(c["T"]):   # each token's state needs the last one's
        state = state * alpha[:, t, :, None, None] + k[:, t, ..., None] * v[:, t, :, None, :]
        o[live, t] = (state * q[:, t, ..., None]).sum(-2)
    s["state"][slots] = state
    return {"o": o.to(s["v"].dtype), "state": s["state"]}


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "dropout": _plain_dropout, "decay": _plain_decay, "step": _plain_step}[c["op"]](s)
    import quaternion_cumulative_product_gb300 as qs
    if c["op"] == "norm":
        if not c["grad"]:
            return {"y": qs.quat_layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)}
        d_x, d_w, d_b = qs.quat_layer_norm_bwd(s["x"], s["d_y"], s["w"], s["b"], eps=EPS)
        return {"d_x": d_x, "d_w": d_w, "d_b": d_b} if s["w"] is not None else {"d_x": d_x}
    if c["op"] == "dropout":
        out = {"y": qs.quat_dropout_fwd(s["x"], s["key"], c["p"], s["residual"])}
        if c["grad"]:
            out["d_x"] = qs.quat_dropout_bwd(s["d_y"], s["key"], c["p"])
        return out
    if c["op"] == "step":
        return {"o": qs.quat_decay_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"]), "state": s["state"]}
    if not c["grad"]:
        o, final = qs.quat_decay_fwd(s["q"], s["k"], s["v"], s["g"], s["init"], offsets=s["offsets"])
        return {"o": o, "final": final}
    o, final = qs.quat_decay_fwd(s["q"], s["k"], s["v"], s["g"], s["init"])
    d_q, d_k, d_v, d_g, d_init = qs.quat_decay_bwd(s["q"], s["k"], s["v"], s["g"], s["d_o"], s["d_final"], s["init"])
    out = {"o": o, "final": final, "d_q": d_q, "d_k": d_k, "d_v": d_v, "d_g": d_g}
    return out | {"d_init": d_init} if c["init"] else out


# ---------------------------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_norm(c, s):
    out = {}
    x = s["x"].double()
    with torch.enable_grad():
        x.requires_grad_(c["grad"])
        w, b = (None, None) if s["w"] is None else (s["w"].double().requires_grad_(c["grad"]), s["b"].double().requires_grad_(c["grad"]))
        y = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + EPS).sqrt()
        if w is not None:
            y = y * w + b
        if not c["grad"]:
            return {"y": y}
        leaves = {"d_x": x} | ({} if w is None else {"d_w": w, "d_b": b})
        out = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), s["d_y"].double())))
    return out


def _exact_dropout(c, s):
    """The generator on the host, with 64-bit products."""
    seed, offset = (int(x) % 2 ** 64 for x in s["key"].tolist())
    count = s["x"].numel()
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    keep = np.empty((count + 3) // 4 * 4, dtype=bool)
    for at in range(0, len(keep) // 4, 1 << 20):   # pieces that stay in the host's caches
        block = np.arange(at, min(at + (1 << 20), len(keep) // 4), dtype=np.uint64)
        x0, x1 = block & low, block >> half
        x2, x3 = np.full_like(block, offset % 2 ** 32), np.full_like(block, offset >> 32)
        for i in range(10):
            ka = np.uint64((seed % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32)
            kb = np.uint64(((seed >> 32) + i * 0xBB67AE85) % 2 ** 32)
            a, b = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
            x0, x1, x2, x3 = (b >> half) ^ x1 ^ ka, b & low, (a >> half) ^ x3 ^ kb, a & low
        drop = np.uint64(int(c["p"] * 2 ** 32))
        for i, x in enumerate((x0, x1, x2, x3)):
            keep[4 * at + i: 4 * (at + len(block)): 4] = x >= drop
    keep = torch.from_numpy(keep[:count]).cuda().view(s["x"].shape)
    y = s["x"].double() * keep / (1 - c["p"])
    out = {"y": y if s["residual"] is None else y + s["residual"].double()}
    if c["grad"]:
        out["d_x"] = s["d_y"].double() * keep / (1 - c["p"])
    return out


def _exact_sequence(c, q, k, v, g, state):
    """One head of one sequence: every pair of steps of a long block at once, the state between blocks."""
    outs = []
    for at in range(0, q.shape[0], 2048):
        qb, kb, vb, gb = (x[at: at + 2048] for x in (q, k, v, g))
        n = gb.cumsum(0)
        far = n[:, None] - n[None]
        far = torch.where(torch.ones_like(far, dtype=torch.bool).tril(), far, -math.inf).exp()
        outs.append(((qb @ kb.T) * far) @ vb + (n.exp()[:, None] * qb) @ state)
        state = n[-1].exp() * state + (kb * (n[-1] - n).exp()[:, None]).T @ vb
    return torch.cat(outs) if outs else v, state


def _exact_decay(c, s):
    shared, scale = c["Hv"] // c["Hk"], c["Dk"] ** -0.5
    seqs = c["packed"] or c["B"]
    off = s["offsets"].tolist() if c["packed"] else None
    names = ["q", "k", "v", "g"] + (["init"] if c["init"] else [])
    out = {"o": torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda"),
           "final": torch.zeros(seqs, c["Hv"], c["Dk"], c["Dv"], dtype=torch.float64, device="cuda")}
    if c["grad"]:
        out |= {"d_" + n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in names}
    for n in range(seqs):
        b, rows = (0, slice(off[n], off[n + 1])) if c["packed"] else (n, slice(0, c["S"]))
        for h in range(c["Hv"]):
            f = {"q": s["q"][b, rows, h // shared], "k": s["k"][b, rows, h // shared], "v": s["v"][b, rows, h], "g": s["g"][b, rows, h]}
            f = {m: x.double() for m, x in f.items()}
            f["init"] = s["init"][n, h].double() if c["init"] else torch.zeros(c["Dk"], c["Dv"], dtype=torch.float64, device="cuda")
            with torch.set_grad_enabled(c["grad"]):
                if c["grad"]:
                    f = {m: x.requires_grad_() for m, x in f.items()}
                o, final = _exact_sequence(c, f["q"] * scale, f["k"], f["v"], f["g"], f["init"])
                if c["grad"]:
                    grads = dict(zip(f, torch.autograd.grad([o, final], list(f.values()), [s["d_o"][b, rows, h].double(), s["d_final"][n, h].double()])))
                    for m in ("q", "k"):
                        out["d_" + m][b, rows, h // shared] += grads[m]
                    out["d_v"][b, rows, h], out["d_g"][b, rows, h] = grads["v"], grads["g"]
                    if c["init"]:
                        out["d_init"][n, h] = grads["init"]
            out["o"][b, rows, h], out["final"][n, h] = o.detach(), final.detach()
    return out


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
        st = st * s["g"][on, t].double().exp()[..., None, None] + torch.einsum("nhk,nhv->nhkv", kt, s["v"][on, t].double())
        o[on, t] = torch.einsum("nhk,nhkv->nhv", qt * c["Dk"] ** -0.5, st)
    state[at] = st
    return {"o": o, "state": state}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decay":   # products of 2048 x 2048 x D, some of them several times over for the gradients
        pairs = case["B"] * case["S"] * case["Hv"] * min(case["S"], 2048) * (case["Dk"] + case["Dv"]) * (4 if case["grad"] else 1)
        if pairs > 8e12 or (case["packed"] or case["B"]) * case["Hv"] * (1 + case["S"] // 2048) > 4000:
            return None
    return {"norm": _exact_norm, "dropout": _exact_dropout, "decay": _exact_decay, "step": _exact_step}[case["op"]](case, s)
