"""Workloads of linear attention with a fixed decay for each head, and of the queries and keys that it reads.

A layer without an erase gate keeps, for each head, the state S <- a S + k v^T with one decay a for the head and
reads o = S^T q.  Its queries and keys are normalised for each head and rotated by their position.  The operators

  attn_fwd, attn_bwd   whole prompts, batched or packed, and their gradients
  attn_step            one token for each sequence, the states updated in place
  rope_fwd, rope_bwd   the norms of q and k for each head with the position rotation, and their gradients

``run`` makes the library's calls where ``own`` is true and computes the same
in elementary torch operations where it is not.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
CHUNK = 64  # of the plain form
F32, F64 = torch.float32, torch.float64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # Training, 8 sequences of 4096 tokens, 16 heads of 128: no state comes in and none is kept.
        {"name": "attn_fwd_train", "op": "attn_fwd", "B": 8, "T": 4096, "H": 16, "dk": 128, "dv": 128, "seqs": 0,
         "state": "none", "dtype": "bf16"},
        # One prompt before decoding: few heads' chains, and the state they leave.
        {"name": "attn_fwd_prompt", "op": "attn_fwd", "B": 1, "T": 4096, "H": 16, "dk": 128, "dv": 128, "seqs": 0,
         "state": "out", "dtype": "bf16"},
        # Continued prompts of 24 users packed into one row, lengths that divide nothing, some of them empty.
        {"name": "attn_fwd_packed", "op": "attn_fwd", "B": 1, "T": 5003, "H": 6, "dk": 64, "dv": 128, "seqs": 24,
         "state": "both", "dtype": "bf16"},
        # FP32 inputs at odd sizes, a narrow value head.
        {"name": "attn_fwd_odd_f32", "op": "attn_fwd", "B": 3, "T": 1371, "H": 5, "dk": 64, "dv": 32, "seqs": 0,
         "state": "both", "dtype": "f32"},
        # The training shape's backward.
        {"name": "attn_bwd_train", "op": "attn_bwd", "B": 8, "T": 4096, "H": 16, "dk": 128, "dv": 128, "seqs": 0,
         "state": "none", "dtype": "bf16"},
        # FP32 backward over packed sequences with the gradients of both states (truncated back-propagation).
        {"name": "attn_bwd_packed_f32", "op": "attn_bwd", "B": 1, "T": 3001, "H": 4, "dk": 128, "dv": 64, "seqs": 7,
         "state": "both", "dtype": "f32"},
        # One decode step of 256 sequences: the states are read and written once.
        {"name": "attn_step_256", "op": "attn_step", "N": 256, "H": 16, "dk": 128, "dv": 128, "dtype": "bf16"},
        # A single sequence's token: nothing but latency.
        {"name": "attn_step_1", "op": "attn_step", "N": 1, "H": 16, "dk": 128, "dv": 128, "dtype": "bf16"},
        # The queries and keys of the training shape, every channel rotated.
        {"name": "rope_fwd_train", "op": "rope_fwd", "B": 8, "T": 4096, "Hq": 16, "Hk": 16, "d": 128, "rot": 128,
         "pairs": "halves", "weights": True, "far": False, "dtype": "bf16"},
        # Decode: one token each of 256 sequences at far positions, grouped key heads.
        {"name": "rope_fwd_decode", "op": "rope_fwd", "B": 256, "T": 1, "Hq": 16, "Hk": 4, "d": 128, "rot": 64,
         "pairs": "halves", "weights": True, "far": True, "dtype": "bf16"},
        # The training shape's backward, with the weights' gradients.
        {"name": "rope_bwd_train", "op": "rope_bwd", "B": 8, "T": 4096, "Hq": 16, "Hk": 16, "d": 128, "rot": 128,
         "pairs": "halves", "weights": True, "far": False, "dtype": "bf16"},
        # FP32 backward at odd sizes, neighbouring pairs, positions that restart within a packed row.
        {"name": "rope_bwd_odd_f32", "op": "rope_bwd", "B": 1, "T": 5003, "Hq": 11, "Hk": 3, "d": 64, "rot": 48,
         "pairs": "neighbours", "weights": True, "far": True, "dtype": "f32"},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))

    op, dtype = rng.choice(["attn_fwd", "attn_bwd", "attn_step", "rope_fwd", "rope_bwd"]), rng.choice(["bf16", "bf16", "f32"])
    if op in ("rope_fwd", "rope_bwd"):
        Hk, d = rng.randint(1, 16), rng.choice([32, 64, 128])
        Hq = min(32, Hk * rng.choice([1, 1, 2, 4]))
        most = 32768 * 32 * 128 // ((Hq + Hk) * d) // (1 if dtype == "bf16" else 2)
        tokens = log(1, min(65536, most))
        B = 1 if rng.random() < 0.5 else rng.randint(1, min(256, tokens))
        return {"op": op, "B": B, "T": tokens // B, "Hq": Hq, "Hk": Hk, "d": d, "rot": rng.choice([d, d, d // 2, 8 * rng.randint(0, d // 8)]),
                "pairs": rng.choice(["halves", "halves", "neighbours"]), "weights": rng.random() < 0.8, "far": rng.random() < 0.5,
                "dtype": dtype}
    H, dk, dv = rng.randint(1, 16), rng.choice([32, 64, 128, 128]), rng.choice([32, 64, 128, 128])
    if op == "attn_step":
        return {"op": op, "N": log(1, 256 * 16 // H), "H": H, "dk": dk, "dv": dv, "dtype": dtype}
    most = 32768 * 16 * 128 // (H * max(dk, dv)) // (1 if dtype == "bf16" else 4)
    tokens = log(1, min(32768, most))
    B = 1 if rng.random() < 0.5 else rng.randint(1, min(16, tokens))
    return {"op": op, "B": B, "T": tokens // B, "H": H, "dk": dk, "dv": dv,
            "seqs": rng.randint(1, 40) if B == 1 and rng.random() < 0.6 else 0,
            "state": rng.choice(["none", "out", "both"]), "dtype": dtype}


def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] in ("rope_fwd", "rope_bwd"):
        tokens, heads, d = c["B"] * c["T"], c["Hq"] + c["Hk"], c["d"]
        small = 4 * tokens + 2 * c["rot"] + 8 * d * c["weights"]
        if c["op"] == "rope_fwd":
            return {"bytes": 2 * e * tokens * heads * d + small, "flops": 7 * tokens * heads * d}
        return {"bytes": 3 * e * tokens * heads * d + small + 8 * d * c["weights"], "flops": 14 * tokens * heads * d}
    square = c["dk"] * c["dv"]
    if c["op"] == "attn_step":
        chains = c["N"] * c["H"]
        return {"bytes": chains * (8 * square + e * (2 * c["dk"] + 2 * c["dv"])) + 4 * c["H"], "flops": 5 * chains * square}
    rows, state = c["B"] * c["T"] * c["H"], 4 * (c["seqs"] or c["B"]) * c["H"] * square
    if c["op"] == "attn_fwd":
        # a token's state update and the read of its output
        return {"bytes": e * rows * (2 * c["dk"] + 2 * c["dv"]) + 4 * c["H"] + state * {"none": 0, "out": 1, "both": 2}[c["state"]],
                "flops": 4 * rows * square}
    # q, k, v, do in, dq, dk, dv out; two states to update and three gradients to read from them
    return {"bytes": e * rows * (4 * c["dk"] + 3 * c["dv"]) + 4 * c["H"] + state * {"none": 0, "out": 1, "both": 3}[c["state"]],
            "flops": 10 * rows * square}


def _cuts(seed, T, seqs):
    at = np.sort(np.random.RandomState(seed % (1 << 31)).randint(0, T + 1, seqs - 1))
    return torch.from_numpy(np.concatenate([[0], at, [T]]).astype(np.int32)).to(DEVICE)


def prepare(case, seed):
    """Queries and keys of normed size, values as a projection leaves them, decays in a geometric row over the heads,
    states that a prompt has left, gradients of mixed size; the table of rotation frequencies."""
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    c, dt = case, DTYPES[case["dtype"]]

    def rnd(shape, dtype=dt, scale=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=DEVICE, dtype=F32).mul_(scale).add_(mean).to(dtype)

    s = {"case": dict(case)}
    if c["op"] in ("rope_fwd", "rope_bwd"):
        B, T, d, R = c["B"], c["T"], c["d"], c["rot"]
        loud = torch.ones(d, device=DEVICE)
        loud[:: 29] = 6.0
        for name, heads in (("q", c["Hq"]), ("k", c["Hk"])):
            s[name] = (rnd((B, T, heads, d), F32) * loud).to(dt)
            s["weight_" + name] = rnd((d,), F32, 0.2, 1.0) if c["weights"] else None
            if c["op"] == "rope_bwd":
                s["d_" + name] = rnd((B, T, heads, d), dt, 0.5)
        s["inv_freq"] = (1e4 ** (-torch.arange(0, R, 2, dtype=F64, device=DEVICE) / R)).to(F32) if R else None
        s["positions"] = None  # the token's index in its row
        if c["far"] and T == 1:
            s["positions"] = torch.randint(0, 1 << 20, (B, 1), generator=g, device=DEVICE, dtype=torch.int32)
        elif c["far"]:  # sequences packed into each row, each from a position of its own on
            first = torch.randint(0, 1 << 17, (B, 4), generator=g, device=DEVICE, dtype=torch.int32)
            part = torch.arange(T, device=DEVICE) * 4 // T
            s["positions"] = (first[:, part] + torch.arange(T, device=DEVICE, dtype=torch.int32)).contiguous()
        s["q_scale"] = d ** -0.5
        return s
    H, dk, dv = c["H"], c["dk"], c["dv"]
    slopes = 2.0 ** (-8.0 * (torch.arange(H, dtype=F64, device=DEVICE) + 1) / H)
    s["alpha"] = torch.exp(-slopes).to(F32)
    lead = (c["N"], H) if c["op"] == "attn_step" else (c["B"], c["T"], H)
    N = c["N"] if c["op"] == "attn_step" else c["seqs"] or c["B"]
    s["q"], s["k"], s["v"] = rnd((*lead, dk), dt, dk ** -0.5), rnd((*lead, dk)), rnd((*lead, dv), dt, 0.7)
    if c["op"] == "attn_step":
        s["state"] = rnd((N, H, dk, dv), F32, 2.0)
        return s
    s["cu_seqlens"] = _cuts(seed, c["T"], c["seqs"]) if c["seqs"] else None
    s["initial_state"] = rnd((N, H, dk, dv), F32, 2.0) if c["state"] == "both" else None
    if c["op"] == "attn_bwd":
        s["d_o"] = rnd((*lead, dv), dt, 0.5)
        s["d_final_state"] = rnd((N, H, dk, dv), F32, 0.5) if c["state"] != "none" else None
    return s


# ---- the plain form: elementary operations in 32 bits -----------------------


def _bounds(s):
    """Offsets of the sequences in the flattened token axis."""
    c = s["case"]
    if s["cu_seqlens"] is not None:
        return s["cu_seqlens"].to(torch.int64)
    return torch.arange(c["B"] + 1, device=DEVICE) * c["T"]


def _power(alpha, n):
    """alpha^n [H, ...] for whole n: through 64 bits, as n reaches the longest sequence."""
    log = torch.log(alpha.to(F64).clamp(2.0 ** -15, 1.0)).reshape(-1, *[1] * n.dim())
    return torch.exp(log * n.to(F64)).to(F32)


def _walk(a, b, c, bounds, alpha, carry, late):
    """out_i = sum_{j <= i} alpha^(i-j) (a_i . b_j) c_j + alpha^(i+1-late) carry^T a_i within each sequence, and the carry
    behind it, alpha^len carry + sum_j alpha^(len-1+late-j) b_j c_j^T.  a, b: [L, H, x], c: [L, H, y]; carry [N, H, x, y].
    Every sequence is cut into chunks: token t of sequence n sits in chunk first[n] + (t - start) / CHUNK."""
    L, H, x = a.shape
    y, N = c.shape[-1], bounds.numel() - 1
    t = torch.arange(L, device=DEVICE)
    start, length = bounds[:-1], bounds[1:] - bounds[:-1]
    first = start // CHUNK + torch.arange(N, device=DEVICE)
    chunks = L // CHUNK + N
    n = (torch.searchsorted(bounds[1:].contiguous(), t, right=True)).clamp(max=N - 1)
    at = first[n] * CHUNK + (t - start[n])                       # a token's place in [chunks * CHUNK]
    ids = torch.arange(chunks, device=DEVICE)
    of = (torch.searchsorted(first, ids, right=True) - 1).clamp(min=0)
    m = ids - first[of]                                          # a chunk's place in its sequence
    held = (length[of] - m * CHUNK).clamp(0, CHUNK)              # its tokens

    def lay(z):
        out = torch.zeros((chunks * CHUNK, *z.shape[1:]), dtype=F32, device=DEVICE)
        out[at] = z
        return out.reshape(chunks, CHUNK, H, -1).permute(2, 0, 1, 3)  # [H, chunks, CHUNK, .]

    A, B, C = lay(a), lay(b), lay(c)
    i = torch.arange(CHUNK, device=DEVICE)
    inside = _power(alpha, (i[:, None] - i).clamp(min=0)) * (i[:, None] >= i)        # [H, CHUNK, CHUNK]
    out = ((A @ B.transpose(-1, -2)) * inside[:, None]) @ C
    to_end = _power(alpha, (held[:, None] - 1 + late - i).clamp(min=0)) * (i < held[:, None])
    left = ((B * to_end[..., None]).transpose(-1, -2) @ C).reshape(H, chunks, x * y)  # what a chunk adds to the carry
    gap = m[:, None] - m - 1
    follows = (of[:, None] == of) & (gap >= 0)
    carried = (_power(alpha, gap.clamp(min=0) * CHUNK) * follows) @ left
    behind = (length[:, None] - m * CHUNK - held)                                    # tokens of n behind a chunk
    mine = of == torch.arange(N, device=DEVICE)[:, None]
    last = (_power(alpha, behind.clamp(min=0)) * mine) @ left                        # [H, N, x y]
    if carry is not None:
        was = carry.reshape(N, H, x * y).transpose(0, 1)
        carried = carried + _power(alpha, m.clamp(min=0) * CHUNK)[..., None] * was[:, of]
        last = last + _power(alpha, length)[..., None] * was
    out = out + _power(alpha, i + 1 - late)[:, None, :, None] * (A @ carried.reshape(H, chunks, x, y))
    out = out.permute(1, 2, 0, 3).reshape(chunks * CHUNK, H, y)[at]
    return out, last.transpose(0, 1).reshape(N, H, x, y)


def _attn_fwd(s):
    c, dt = s["case"], s["q"].dtype
    L, H = c["B"] * c["T"], c["H"]
    q, k, v = (s[n].reshape(L, H, -1).to(F32) for n in ("q", "k", "v"))
    o, last = _walk(q, k, v, _bounds(s), s["alpha"], s["initial_state"], 0)
    out = {"o": o.reshape(s["v"].shape).to(dt)}
    if c["state"] != "none":
        out["final_state"] = last
    return out


def _attn_bwd(s):
    """dq reads the forward state, dk and dv the state's gradient: walks over the tokens, and over the tokens in reverse."""
    c, dt = s["case"], s["q"].dtype
    L, H, bounds = c["B"] * c["T"], c["H"], _bounds(s)
    q, k, v, do = (s[n].reshape(L, H, -1).to(F32) for n in ("q", "k", "v", "d_o"))
    into, back = s["initial_state"], s["d_final_state"]
    dq, _ = _walk(do, v, k, bounds, s["alpha"], None if into is None else into.transpose(-1, -2), 0)
    turned = L - bounds.flip(0)
    qr, kr, vr, dr = (z.flip(0) for z in (q, k, v, do))
    gone = None if back is None else back.flip(0)
    dk, _ = _walk(vr, dr, qr, turned, s["alpha"], None if gone is None else gone.transpose(-1, -2), 1)
    dv, first = _walk(kr, qr, dr, turned, s["alpha"], gone, 1)
    out = {"dq": dq.reshape(s["q"].shape).to(dt), "dk": dk.flip(0).reshape(s["k"].shape).to(dt),
           "dv": dv.flip(0).reshape(s["v"].shape).to(dt)}
    if c["state"] == "both":
        out["d_initial_state"] = first.flip(0)
    return out


def _attn_step(s):
    q, k, v = (s[n].to(F32) for n in ("q", "k", "v"))
    a = s["alpha"].clamp(2.0 ** -15, 1.0)[:, None, None]
    s["state"].copy_(a * s["state"] + k[..., :, None] * v[..., None, :])
    return {"o": (s["state"] * q[..., :, None]).sum(-2).to(s["q"].dtype), "state": s["state"]}


def _angles(s):
    """cos and sin [B or 1, T, 1, rot / 2] of position times frequency: the product and its period need 64 bits."""
    at = s["positions"]
    if at is None:
        at = torch.arange(s["case"]["T"], device=DEVICE)[None]
    turn = at.to(F64)[..., None, None] * s["inv_freq"].to(F64)
    return torch.cos(turn).to(F32), torch.sin(turn).to(F32)


def _rotate(n, s, sign):
    c, R = s["case"], s["case"]["rot"]
    if not R:
        return n
    cos, sin = _angles(s)
    sin = sin * sign
    if c["pairs"] == "halves":
        one, two = n[..., : R // 2], n[..., R // 2: R]
        return torch.cat([one * cos - two * sin, two * cos + one * sin, n[..., R:]], -1)
    one, two = n[..., 0:R:2], n[..., 1:R:2]
    return torch.cat([torch.stack([one * cos - two * sin, two * cos + one * sin], -1).flatten(-2), n[..., R:]], -1)


def _rope_fwd(s):
    out = {}
    for name, scale in (("q", s["q_scale"]), ("k", 1.0)):
        x, w = s[name].to(F32), s["weight_" + name]
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        out[name] = (_rotate(n if w is None else n * w, s, 1.0) * scale).to(s[name].dtype)
    return out


def _rope_bwd(s):
    out = {}
    for name, scale in (("q", s["q_scale"]), ("k", 1.0)):
        x, w, dt = s[name].to(F32), s["weight_" + name], s[name].dtype
        dn = _rotate(s["d_" + name].to(F32) * scale, s, -1.0)
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        if w is not None:
            out["d_weight_" + name] = (dn * x * r).sum((0, 1, 2))
            dn = dn * w
        out["d_" + name] = (r * (dn - x * r.square() * (dn * x).mean(-1, keepdim=True))).to(dt)
    return out


# ---- one pass ---------------------------------------------------------------


def _own(s):
    import delta_rule_linear_gdn2_amd as gdn2

    c = s["case"]
    if c["op"] == "attn_fwd":
        o, last = gdn2.gdn2_linear_attn_fwd(s["q"], s["k"], s["v"], s["alpha"], s["initial_state"],
                                            output_final_state=c["state"] != "none", cu_seqlens=s["cu_seqlens"])
        return {"o": o, "final_state": last}
    if c["op"] == "attn_bwd":
        return gdn2.gdn2_linear_attn_bwd(s["q"], s["k"], s["v"], s["alpha"], s["d_o"], initial_state=s["initial_state"],
                                         d_final_state=s["d_final_state"], output_d_initial_state=c["state"] == "both",
                                         cu_seqlens=s["cu_seqlens"])
    if c["op"] == "attn_step":
        return {"o": gdn2.gdn2_linear_attn_step(s["q"], s["k"], s["v"], s["alpha"], s["state"]), "state": s["state"]}
    how = dict(positions=s["positions"], weight_q=s["weight_q"], weight_k=s["weight_k"], q_scale=s["q_scale"], eps=EPS,
               interleaved=c["pairs"] == "neighbours")
    if c["op"] == "rope_fwd":
        return dict(zip("qk", gdn2.gdn2_qk_norm_rope(s["q"], s["k"], s["inv_freq"], **how)))
    return gdn2.gdn2_qk_norm_rope_bwd(s["q"], s["k"], s["d_q"], s["d_k"], s["inv_freq"], **how)


def run(state):
    if own:
        return {k: v for k, v in _own(state).items() if v is not None}
    return {"attn_fwd": _attn_fwd, "attn_bwd": _attn_bwd, "attn_step": _attn_step, "rope_fwd": _rope_fwd,
            "rope_bwd": _rope_bwd}[state["case"]["op"]](state)


def exact(case, seed):
    """The definitions in 64 bits: the recurrence token by token, and the norm and rotation as complex numbers with
    the gradients by reverse mode."""
    s, c = prepare(case, seed), case

    def wide(v):
        return None if v is None else v.to(F64)

    if c["op"] in ("rope_fwd", "rope_bwd"):
        at = s["positions"] if s["positions"] is not None else torch.arange(c["T"], device=DEVICE)[None]
        R, out = c["rot"], {}
        for name, scale in (("q", s["q_scale"]), ("k", 1.0)):
            x, w = wide(s[name]).requires_grad_(True), wide(s["weight_" + name])
            w = w.requires_grad_(True) if w is not None else None
            n = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS)
            n = scale * (n * w if w is not None else n)
            if R:
                pairs = n[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2) if c["pairs"] == "halves" else n[..., :R].unflatten(-1, (R // 2, 2))
                turn = at.to(F64)[..., None, None] * wide(s["inv_freq"])
                z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(turn), turn)
                back = torch.view_as_real(z)
                back = back.transpose(-1, -2) if c["pairs"] == "halves" else back
                n = torch.cat([back.flatten(-2), n[..., R:]], -1)
            if c["op"] == "rope_fwd":
                out[name] = n.detach()
                continue
            got = torch.autograd.grad(n, [x] if w is None else [x, w], wide(s["d_" + name]))
            out.update(zip(("d_" + name, "d_weight_" + name), got))
        return out

    a = wide(s["alpha"]).clamp(2.0 ** -15, 1.0)[:, None, None]
    q, k, v = wide(s["q"]), wide(s["k"]), wide(s["v"])
    if c["op"] == "attn_step":
        S = a * wide(s["state"]) + k.unsqueeze(-1) * v.unsqueeze(-2)
        return {"o": (q.unsqueeze(-2) @ S).squeeze(-2), "state": S}
    if s["cu_seqlens"] is None:
        spans = [(slice(None), slice(None), 0, c["T"])]
    else:
        cu = s["cu_seqlens"].tolist()
        spans = [(slice(n, n + 1), slice(0, 1), lo, hi) for n, (lo, hi) in enumerate(zip(cu[:-1], cu[1:]))]
    N = c["seqs"] or c["B"]
    start = wide(s["initial_state"])
    start = torch.zeros((N, c["H"], c["dk"], c["dv"]), dtype=F64, device=DEVICE) if start is None else start
    last = torch.zeros_like(start)
    o, dq, dk, dv = torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    do = wide(s["d_o"]) if c["op"] == "attn_bwd" else None
    for n, row, lo, hi in spans:
        S = start[n].clone()
        for t in range(lo, hi):
            S = torch.addcmul(a * S, k[row, t].unsqueeze(-1), v[row, t].unsqueeze(-2))
            if do is None:
                o[row, t] = (S * q[row, t].unsqueeze(-1)).sum(-2)
            else:
                dq[row, t] = (S * do[row, t].unsqueeze(-2)).sum(-1)
        last[n] = S
        if do is None:
            continue
        S = torch.zeros_like(start[n]) if s["d_final_state"] is None else wide(s["d_final_state"])[n].clone()
        for t in range(hi - 1, lo - 1, -1):
            S = torch.addcmul(S, q[row, t].unsqueeze(-1), do[row, t].unsqueeze(-2))
            dk[row, t] = (S * v[row, t].unsqueeze(-2)).sum(-1)
            dv[row, t] = (S * k[row, t].unsqueeze(-1)).sum(-2)
            S = a * S
        last[n] = S
    if do is None:
        return {"o": o, "final_state": last if c["state"] != "none" else None}
    return {"dq": dq, "dk": dk, "dv": dv, "d_initial_state": last if c["state"] == "both" else None}
