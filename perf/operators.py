"""Workloads of the operators that train a layer around the recurrence.

A layer is: norm, mixer prologue, recurrence, mixer epilogue, output
projection, and back onto the residual stream through a norm, a gate, a
residual scale and dropout.  The operators here are

  block_fwd, block_bwd   the step from one block to the next: norm of the block's
                         output, gate, dropout, residual scale, the sum with the
                         residual stream, and the norm in front of the next
                         block; and its gradients
  dropout                counter-based dropout alone (its own adjoint)
  epilogue_bwd           gradients of the mixer epilogue (RMS norm, output gate)
  prologue_bwd           gradients of the mixer prologue (causal convolution,
                         SiLU, L2 norm, gate sigmoids)

``run`` makes the library's calls where ``own`` is true and computes the same
in elementary torch operations where it is not.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
EPS = 1e-5      # RMS norms
EPS_L2 = 1e-6   # L2 norm of q and k
F32, F64 = torch.float32, torch.float64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # Training, 8 sequences of 4096 tokens, 16 heads of 128: FP32 residual stream, an output gate per
        # channel and token, norms on both sides and dropout.
        {"name": "block_fwd_train", "op": "block_fwd", "rows": 32768, "D": 2048, "dtype": "bf16", "res": "f32",
         "gate": "full", "act": "sigmoid", "post": True, "pre": True, "p": 0.1, "scale": 0.5},
        # One decode step of 256 sequences: a learned scale per channel, no dropout.
        {"name": "block_fwd_decode_256", "op": "block_fwd", "rows": 256, "D": 2048, "dtype": "bf16", "res": "bf16",
         "gate": "channel", "act": "identity", "post": True, "pre": True, "p": 0.0, "scale": 1.0},
        # One sequence's single token, the plain pre-norm block: nothing but latency.
        {"name": "block_fwd_decode_1", "op": "block_fwd", "rows": 1, "D": 2048, "dtype": "bf16", "res": "bf16",
         "gate": "none", "act": "identity", "post": False, "pre": True, "p": 0.0, "scale": 1.0},
        # FP32 at sizes that divide nothing, one gate value per token.
        {"name": "block_fwd_odd_f32", "op": "block_fwd", "rows": 5003, "D": 1371, "dtype": "f32", "res": "f32",
         "gate": "token", "act": "silu", "post": True, "pre": True, "p": 0.25, "scale": 0.7},
        # The training shape's backward, with the residual stream in bf16.
        {"name": "block_bwd_train", "op": "block_bwd", "rows": 32768, "D": 2048, "dtype": "bf16", "res": "bf16",
         "gate": "full", "act": "sigmoid", "post": True, "pre": True, "p": 0.1, "scale": 0.5},
        # FP32 backward at odd sizes; the channel gate's gradient is a third sum over the rows.
        {"name": "block_bwd_odd_f32", "op": "block_bwd", "rows": 4099, "D": 1001, "dtype": "f32", "res": "f32",
         "gate": "channel", "act": "identity", "post": True, "pre": True, "p": 0.0, "scale": 1.0},
        # Dropout on a training activation; and FP32 rows of odd length.
        {"name": "dropout_train", "op": "dropout", "rows": 32768, "D": 2048, "dtype": "bf16", "p": 0.1},
        {"name": "dropout_odd_f32", "op": "dropout", "rows": 777, "D": 5461, "dtype": "f32", "p": 0.5},
        # The epilogue's backward at the training shape (a row is a token's head), and a small FP32 one.
        {"name": "epilogue_bwd_train", "op": "epilogue_bwd", "rows": 524288, "dv": 128, "dtype": "bf16",
         "act": "sigmoid"},
        {"name": "epilogue_bwd_f32_64", "op": "epilogue_bwd", "rows": 16001, "dv": 64, "dtype": "f32", "act": "silu"},
        # The prologue's backward at the training shape, and over 24 packed sequences that carry a
        # convolution state (some of them empty).
        {"name": "prologue_bwd_train", "op": "prologue_bwd", "B": 8, "T": 4096, "H": 16, "dk": 128, "dv": 128, "K": 4,
         "seqs": 0, "state": False, "dtype": "bf16"},
        {"name": "prologue_bwd_packed", "op": "prologue_bwd", "B": 1, "T": 5003, "H": 6, "dk": 64, "dv": 128, "K": 4,
         "seqs": 24, "state": True, "dtype": "bf16"},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))

    op = rng.choice(["block_fwd", "block_bwd", "dropout", "epilogue_bwd", "prologue_bwd"])
    if op == "epilogue_bwd":
        dv = rng.choice([32, 64, 128])
        return {"op": op, "rows": log(1, 524288), "dv": dv, "dtype": rng.choice(["bf16", "f32"]),
                "act": rng.choice(["sigmoid", "silu"])}
    if op == "prologue_bwd":
        H, dk, dv = rng.randint(1, 16), rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
        K = rng.choice([4, 4, 4, rng.randint(1, 16)])
        dtype = rng.choice(["bf16", "f32"])
        most = min(32768 * 16 * 128 * 4 // (H * max(dk, dv) * K), 32768 * 16 * 640 // (H * (3 * dk + 2 * dv)))
        tokens = log(1, min(32768, most) // (1 if dtype == "bf16" else 2))
        B = 1 if rng.random() < 0.5 else rng.randint(1, min(8, tokens))
        return {"op": op, "B": B, "T": tokens // B, "H": H, "dk": dk, "dv": dv, "K": K,
                "seqs": rng.randint(1, 40) if B == 1 and rng.random() < 0.7 else 0, "state": rng.random() < 0.6,
                "dtype": dtype}
    D, dtype = log(16, 8192), rng.choice(["bf16", "bf16", "f32"])
    res = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
    rows = log(1, 32768 * 2048 // D // (1 if res == "bf16" else 2))
    p = rng.choice([0.0, 0.1, round(rng.uniform(0.01, 0.9), 3)])
    if op == "dropout":
        return {"op": op, "rows": rows, "D": D, "dtype": dtype, "p": p}
    gate = rng.choice(["none", "channel", "token", "full"])
    return {"op": op, "rows": rows, "D": D, "dtype": dtype, "res": res,
            "gate": gate, "act": "identity" if gate == "none" else rng.choice(["sigmoid", "silu", "identity"]),
            "post": rng.random() < 0.7, "pre": rng.random() < 0.8, "p": p, "scale": round(rng.uniform(0.2, 1.5), 3)}


def _gate_size(c):
    return {"none": 0, "channel": c["D"], "token": c["rows"], "full": c["rows"] * c["D"]}[c["gate"]]


def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    op = c["op"]
    if op in ("block_fwd", "block_bwd"):
        n, r, D = c["rows"] * c["D"], 2 if c["res"] == "bf16" else 4, c["D"]
        gate = _gate_size(c) * (4 if c["gate"] == "channel" else e)
        weights = 4 * D * (int(c["post"]) + int(c["pre"]))
        if op == "block_fwd":
            return {"bytes": n * (e + 2 * r) + (n * e if c["pre"] else 0) + gate + weights,
                    "flops": n * (4 + 4 * c["post"] + 4 * c["pre"])}
        # dx' in; du, dx out; u in where a norm or a gate acts on it; x', dh in with the norm in front of the next block
        reads_u = c["post"] or c["gate"] != "none"
        return {"bytes": n * ((2 if reads_u else 1) * e + 2 * r) + (n * (e + r) if c["pre"] else 0) + 2 * gate + 2 * weights,
                "flops": n * (6 + 10 * c["post"] + 10 * c["pre"])}
    if op == "dropout":
        return {"bytes": 2 * e * c["rows"] * c["D"], "flops": c["rows"] * c["D"]}
    if op == "epilogue_bwd":
        return {"bytes": 5 * e * c["rows"] * c["dv"] + 8 * c["dv"], "flops": 20 * c["rows"] * c["dv"]}
    tokens, K, H = c["B"] * c["T"], c["K"], c["H"]
    ch = H * (2 * c["dk"] + c["dv"])                        # convolution channels
    wide = H * (3 * c["dk"] + 2 * c["dv"])                  # and the two gates'
    state = 4 * (c["seqs"] or c["B"]) * ch * (K - 1) * (3 if c["state"] else 0)
    return {"bytes": 3 * e * tokens * wide + 2 * 4 * ch * K + state, "flops": tokens * (ch * (6 * K + 15) + 6 * (wide - ch))}


def prepare(case, seed):
    """Activations of the size that a norm leaves, a residual stream with a few large channels, gradients
    of mixed size, weights around one, filters of a trained convolution's size."""
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    c, dt = case, DTYPES[case["dtype"]]

    def rnd(shape, dtype, scale=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=DEVICE, dtype=F32).mul_(scale).add_(mean).to(dtype)

    s = {"case": dict(case), "seed": (seed * 0x9E3779B97F4A7C15 + 12345) & 0xFFFFFFFFFFFFFFFF, "offset": 3 + seed % 1000}
    op = c["op"]
    if op in ("block_fwd", "block_bwd"):
        rows, D, rd = c["rows"], c["D"], DTYPES[c["res"]]
        loud = torch.ones(D, device=DEVICE)
        loud[:: 97] = 8.0
        s["u"] = rnd((rows, D), dt, 0.7)
        s["x"] = (rnd((rows, D), F32, 2.0) * loud).to(rd)
        s["weight_post"] = rnd((D,), F32, 0.2, 1.0) if c["post"] else None
        s["weight_pre"] = rnd((D,), F32, 0.2, 1.0) if c["pre"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: rnd((D,), F32, 0.5, 0.3),
                     "token": lambda: rnd((rows,), dt), "full": lambda: rnd((rows, D), dt)}[c["gate"]]()
        if op == "block_fwd":  # a layer's output buffers
            s["x_out"] = torch.empty_like(s["x"])
            s["h"] = torch.empty_like(s["u"]) if c["pre"] else None
        else:
            s["d_x_out"] = rnd((rows, D), rd, 0.5)
            s["d_h"] = rnd((rows, D), dt, 0.5) if c["pre"] else None
    elif op == "dropout":
        s["x"] = rnd((c["rows"], c["D"]), dt)
    elif op == "epilogue_bwd":
        s["o"], s["gate"] = rnd((c["rows"], c["dv"]), dt, 0.3), rnd((c["rows"], c["dv"]), dt)
        s["weight"], s["d_y"] = rnd((c["dv"],), F32, 0.2, 1.0), rnd((c["rows"], c["dv"]), dt, 0.5)
    else:
        B, T, H, dk, dv, K = (c[n] for n in ("B", "T", "H", "dk", "dv", "K"))
        N = c["seqs"] or B
        widths = {"q": dk, "k": dk, "v": dv}
        s["x"] = {n: rnd((B, T, H, d), dt) for n, d in widths.items()}
        s["conv"] = {n: rnd((H * d, K), F32, 0.5) for n, d in widths.items()}
        s["b_logit"], s["w_logit"] = rnd((B, T, H, dk), dt), rnd((B, T, H, dv), dt)
        s["d"] = {n: rnd((B, T, H, d), dt, 0.5) for n, d in {**widths, "b": dk, "w": dv}.items()}
        shape = (N, H * (2 * dk + dv), K - 1)
        s["conv_state"] = rnd(shape, dt).to(F32) if c["state"] else None
        s["d_conv_state_out"] = rnd(shape, F32, 0.5) if c["state"] else None
        s["cu_seqlens"] = None
        if c["seqs"]:
            cuts = np.sort(np.random.RandomState(seed % (1 << 31)).randint(0, T + 1, N - 1))
            s["cu_seqlens"] = torch.from_numpy(np.concatenate([[0], cuts, [T]]).astype(np.int32)).to(DEVICE)
        s["q_scale"] = dk ** -0.5
    return s


# ---- the plain form: elementary operations in 32 bits -----------------------


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(g, act):
    """The gate's value and derivative."""
    if act == "identity":
        return g, torch.ones_like(g)
    sg = _sigmoid(g)
    return (sg, sg * (1 - sg)) if act == "sigmoid" else (g * sg, sg * (1 + g * (1 - sg)))


def _rnorm(z):
    return torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS)


def _keep(rows, D, p, seed, offset):
    """The dropout factor of every element: 0 or 1 / (1 - p), p a multiple of 2^-16.  Philox4x32 with ten
    rounds; a block of 128 bits serves eight elements of a row."""
    threshold, groups = int(math.floor(p * 65536 + 0.5)), -(-D // 8)
    word = 0xFFFFFFFF
    block = torch.arange(rows * groups, dtype=torch.int64, device=DEVICE)
    a, b = block & word, block >> 32
    c, d = torch.full_like(a, offset & word), torch.full_like(a, offset >> 32)
    k0, k1 = seed & word, seed >> 32
    for _ in range(10):  # the generator's rounds
        p0, p1 = a * 0xD2511F53, c * 0xCD9E8D57  # 64-bit products: the shifts below take their bits
        a, b, c, d = ((p1 >> 32) & word) ^ b ^ k0, p1 & word, ((p0 >> 32) & word) ^ d ^ k1, p0 & word
        k0, k1 = (k0 + 0x9E3779B9) & word, (k1 + 0xBB67AE85) & word
    bits = torch.stack([a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16, c & 0xFFFF, c >> 16, d & 0xFFFF, d >> 16], -1)
    kept = bits.reshape(rows, groups * 8)[:, :D] >= threshold
    return kept.to(F32) * (65536.0 / (65536 - threshold))


def _block_fwd(s):
    c = s["case"]
    u, x = s["u"].to(F32), s["x"].to(F32)
    n = u * _rnorm(u) * s["weight_post"] if c["post"] else u
    if c["gate"] != "none":
        g = s["gate"].to(F32)
        n = n * _act(g[:, None] if c["gate"] == "token" else g, c["act"])[0]
    if c["p"]:
        n = n * _keep(c["rows"], c["D"], c["p"], s["seed"], s["offset"])
    x_out = (x + c["scale"] * n).to(s["x"].dtype)
    if not c["pre"]:
        return {"x_out": x_out}
    z = x_out.to(F32)  # the norm is that of the stored stream, as the backward pass sees it
    return {"x_out": x_out, "h": (z * _rnorm(z) * s["weight_pre"]).to(s["u"].dtype)}


def _block_bwd(s):
    c, dt, rd = s["case"], s["u"].dtype, s["x"].dtype
    u, t = s["u"].to(F32), s["d_x_out"].to(F32)
    out = {}
    if c["pre"]:
        z, dh = s["x"].to(F32), s["d_h"].to(F32)
        r = _rnorm(z)
        wd = s["weight_pre"] * dh
        out["d_weight_pre"] = (dh * z * r).sum(0)
        t = t + r * wd - z * r.pow(3) * (wd * z).mean(-1, keepdim=True)
    out["d_x"] = t.to(rd)
    b = t * c["scale"]
    if c["p"]:
        b = b * _keep(c["rows"], c["D"], c["p"], s["seed"], s["offset"])
    r = _rnorm(u) if c["post"] else 1.0
    n = u * r * s["weight_post"] if c["post"] else u
    if c["gate"] != "none":
        g = s["gate"].to(F32)
        a, da = _act(g[:, None] if c["gate"] == "token" else g, c["act"])
        dg = b * n * da
        out["d_gate"] = {"full": lambda: dg.to(dt), "token": lambda: dg.sum(1).to(dt), "channel": lambda: dg.sum(0)}[c["gate"]]()
        b = b * a
    if c["post"]:
        out["d_weight_post"] = (b * u * r).sum(0)
        wb = s["weight_post"] * b
        b = r * wb - u * r.pow(3) * (wb * u).mean(-1, keepdim=True)
    out["d_u"] = b.to(dt)
    return out


def _epilogue_bwd(s):
    o, dy, w, dt = s["o"].to(F32), s["d_y"].to(F32), s["weight"], s["o"].dtype
    a, da = _act(s["gate"].to(F32), s["case"]["act"])
    r = _rnorm(o)
    dn = dy * a
    wd = w * dn
    return {"d_o": (r * wd - o * r.pow(3) * (wd * o).mean(-1, keepdim=True)).to(dt),
            "d_gate": (dy * o * r * w * da).to(dt), "d_weight": (dn * o * r).sum(0)}


def _conv_bwd(s, name, chan0):
    """One convolution path: every sequence's tokens behind its K - 1 earlier inputs, in one long axis."""
    c = s["case"]
    B, T, H, K, dt = c["B"], c["T"], c["H"], c["K"], s["x"][name].dtype
    d, N, cu = s["x"][name].shape[-1], c["seqs"] or c["B"], s["cu_seqlens"]
    C, L = H * d, B * T
    t = torch.arange(L, device=DEVICE)
    if cu is None:
        cu = torch.arange(N + 1, device=DEVICE) * T
    cu = cu.to(torch.int64)
    at = t + (torch.searchsorted(cu[1:].contiguous(), t, right=True) + 1) * (K - 1)  # a token's place on the long axis
    first = cu[:-1] + torch.arange(N, device=DEVICE) * (K - 1)                       # a sequence's earlier inputs
    before = (first[:, None] + torch.arange(K - 1, device=DEVICE)).reshape(-1)
    last = (cu[1:] + (torch.arange(N, device=DEVICE)) * (K - 1))[:, None] + torch.arange(K - 1, device=DEVICE)
    taps = torch.arange(K, device=DEVICE)
    M = L + N * (K - 1)
    w = s["conv"][name]
    long = torch.zeros((M, C), dtype=F32, device=DEVICE)
    long[at] = s["x"][name].reshape(L, C).to(F32)
    if s["conv_state"] is not None:
        long[before] = s["conv_state"][:, chan0:chan0 + C].transpose(1, 2).reshape(-1, C)
    window = long[at[:, None] - (K - 1) + taps]  # [L, K, C]
    y = (window * w.T).sum(1)
    a, da = _act(y, "silu")
    dv = s["d"][name].reshape(L, C).to(F32)
    if name != "v":
        scale = s["q_scale"] if name == "q" else 1.0
        v, e = a.reshape(L, H, d), dv.reshape(L, H, d)
        r = torch.rsqrt(v.square().sum(-1, keepdim=True) + EPS_L2)
        dv = (scale * (r * e - v * r.pow(3) * (v * e).sum(-1, keepdim=True))).reshape(L, C)
    dy = dv * da
    spread = torch.zeros((M + K - 1, C), dtype=F32, device=DEVICE)
    spread[at] = dy
    d_long = (spread[torch.arange(M, device=DEVICE)[:, None] + (K - 1) - taps] * w.T).sum(1)
    if s["d_conv_state_out"] is not None:
        d_long.index_add_(0, last.reshape(-1), s["d_conv_state_out"][:, chan0:chan0 + C].transpose(1, 2).reshape(-1, C))
    d_conv = (dy[:, None, :] * window).sum(0).T.contiguous()
    return d_long[at].reshape(B, T, H, d).to(dt), d_conv, d_long[before].reshape(N, K - 1, C).transpose(1, 2)


def _prologue_bwd(s):
    c, dt = s["case"], s["b_logit"].dtype
    hk = c["H"] * c["dk"]
    q, k, v = _conv_bwd(s, "q", 0), _conv_bwd(s, "k", hk), _conv_bwd(s, "v", 2 * hk)
    b, w = _sigmoid(s["b_logit"].to(F32)), _sigmoid(s["w_logit"].to(F32))
    out = {"d_xq": q[0], "d_xk": k[0], "d_xv": v[0], "d_conv_q": q[1], "d_conv_k": k[1], "d_conv_v": v[1],
           "d_b_logit": (s["d"]["b"].to(F32) * b * (1 - b)).to(dt), "d_w_logit": (s["d"]["w"].to(F32) * w * (1 - w)).to(dt)}
    if c["state"]:
        out["d_conv_state"] = torch.cat([q[2], k[2], v[2]], 1)
    return out


# ---- one pass ---------------------------------------------------------------


def _own(s):
    import delta_rule_linear_gdn2_amd as gdn2

    c = s["case"]
    op = c["op"]
    if op in ("block_fwd", "block_bwd"):
        how = dict(gate=s["gate"], gate_layout=c["gate"], gate_act=c["act"], weight_post=s["weight_post"],
                   weight_pre=s["weight_pre"], eps=EPS, residual_scale=c["scale"], dropout_p=c["p"], seed=s["seed"],
                   offset=s["offset"])
        if op == "block_bwd":
            return gdn2.gdn2_block_norm_bwd(s["x"], s["u"], s["d_x_out"], s["d_h"], **how)
        return gdn2.gdn2_block_norm_fwd(s["x"], s["u"], x_out=s["x_out"], h=s["h"], **how)
    if op == "dropout":
        return gdn2.gdn2_dropout(s["x"], c["p"], s["seed"], s["offset"])
    if op == "epilogue_bwd":
        return gdn2.gdn2_mixer_epilogue_bwd(s["o"], s["gate"], s["weight"], s["d_y"], eps=EPS, act=c["act"])
    x, w, d = s["x"], s["conv"], s["d"]
    return gdn2.gdn2_mixer_prologue_bwd(
        x["q"], x["k"], x["v"], w["q"], w["k"], w["v"], s["b_logit"], s["w_logit"], d["q"], d["k"], d["v"], d["b"], d["w"],
        conv_state=s["conv_state"], d_conv_state_out=s["d_conv_state_out"], output_d_conv_state=c["state"],
        cu_seqlens=s["cu_seqlens"], q_scale=s["q_scale"], eps_l2=EPS_L2)


def run(state):
    c = state["case"]
    if own:
        got = _own(state)
        if c["op"] == "block_fwd":
            got = dict(zip(("x_out", "h"), got))
        if c["op"] == "dropout":
            got = {"y": got}
        return {k: v for k, v in got.items() if v is not None}
    if c["op"] == "dropout":
        return {"y": (state["x"].to(F32) * _keep(c["rows"], c["D"], c["p"], state["seed"], state["offset"])).to(state["x"].dtype)}
    return {"block_fwd": _block_fwd, "block_bwd": _block_bwd, "epilogue_bwd": _epilogue_bwd,
            "prologue_bwd": _prologue_bwd}[c["op"]](state)


def exact(case, seed):
    """The definitions in 64 bits, with the gradients by reverse mode from the forward formulas."""
    s = prepare(case, seed)
    c = case

    def wide(v):
        return None if v is None else v.to(F64)

    def leaf(v):
        return None if v is None else v.to(F64).requires_grad_(True)

    def gated(g):
        return {"sigmoid": torch.sigmoid, "silu": lambda z: z * torch.sigmoid(z), "identity": lambda z: z}[c["act"]](g)

    def rms(z, weight):
        return z / torch.sqrt((z * z).sum(-1, keepdim=True) / z.shape[-1] + EPS) * weight

    def factor():
        rows, D, cut = c["rows"], c["D"], int(math.floor(c["p"] * 65536 + 0.5))
        M = np.uint64(0xFFFFFFFF)
        n = np.arange(rows * ((D + 7) // 8), dtype=np.uint64)
        x = [n & M, n >> np.uint64(32), np.full_like(n, s["offset"] & 0xFFFFFFFF), np.full_like(n, s["offset"] >> 32)]
        key = [s["seed"] & 0xFFFFFFFF, s["seed"] >> 32]
        for _ in range(10):
            lo, hi = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
            x = [(hi >> np.uint64(32)) ^ x[1] ^ np.uint64(key[0]), hi & M, (lo >> np.uint64(32)) ^ x[3] ^ np.uint64(key[1]), lo & M]
            key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
        halves = np.stack([w.astype(np.uint32) for w in x], 1).view(np.uint16)  # little endian: the low half first
        keep = torch.from_numpy((halves.reshape(rows, -1)[:, :D] >= cut)).to(DEVICE)
        return keep.to(F64) / (1 - cut / 65536)

    op = c["op"]
    if op == "dropout":
        return {"y": s["x"].to(F64) * factor()}
    if op in ("block_fwd", "block_bwd"):
        u, gate, post, pre = leaf(s["u"]), leaf(s["gate"]), leaf(s["weight_post"]), leaf(s["weight_pre"])
        branch = rms(u, post) if c["post"] else u * 1.0
        if gate is not None:
            branch = branch * (gated(gate)[:, None] if c["gate"] == "token" else gated(gate))
        branch = c["scale"] * branch * (factor() if c["p"] else 1.0)
        if op == "block_fwd":
            x_out = (wide(s["x"]) + branch).detach()
            out = {"x_out": x_out}
            if c["pre"]:
                out["h"] = rms(x_out.to(s["x"].dtype).to(F64), wide(s["weight_pre"]))
            return out
        out = {}
        t = wide(s["d_x_out"])
        if c["pre"]:
            x = leaf(s["x"])
            dx, out["d_weight_pre"] = torch.autograd.grad(rms(x, pre), [x, pre], wide(s["d_h"]))
            t = t + dx
        names = {"d_u": u, "d_gate": gate, "d_weight_post": post}
        names = {k: v for k, v in names.items() if v is not None}
        out.update(zip(names, torch.autograd.grad(branch, list(names.values()), t)))
        return {**out, "d_x": t}
    if op == "epilogue_bwd":
        o, gate, w = leaf(s["o"]), leaf(s["gate"]), leaf(s["weight"])
        got = torch.autograd.grad(rms(o, w) * gated(gate), [o, gate, w], wide(s["d_y"]))
        return dict(zip(("d_o", "d_gate", "d_weight"), got))

    B, T, H, K, N = c["B"], c["T"], c["H"], c["K"], c["seqs"] or c["B"]
    bounds = [(n, 0, T) for n in range(B)] if s["cu_seqlens"] is None else [
        (0, a, b) for a, b in zip(s["cu_seqlens"].tolist()[:-1], s["cu_seqlens"].tolist()[1:])]
    out, states, chan0 = {}, [], 0
    for name in ("q", "k", "v"):
        x, w = wide(s["x"][name]), leaf(s["conv"][name])
        C = w.shape[0]
        dx, dw, ds = torch.zeros_like(x), torch.zeros_like(w), []
        for n, (row, lo, hi) in enumerate(bounds):
            part = x[row, lo:hi].reshape(hi - lo, C).clone().requires_grad_(True)
            head = torch.zeros((K - 1, C), dtype=F64, device=DEVICE) if s["conv_state"] is None else wide(s["conv_state"][n, chan0:chan0 + C].T)
            head = head.clone().requires_grad_(True)
            line = torch.cat([head, part])
            y = sum(w[:, i] * line[i:i + hi - lo] for i in range(K))
            v = (y * torch.sigmoid(y)).reshape(hi - lo, H, C // H)
            if name != "v":
                v = v / torch.sqrt((v * v).sum(-1, keepdim=True) + EPS_L2) * (s["q_scale"] if name == "q" else 1.0)
            total = (v * wide(s["d"][name][row, lo:hi])).sum()
            if s["d_conv_state_out"] is not None:
                total = total + (line[hi - lo:] * wide(s["d_conv_state_out"][n, chan0:chan0 + C].T)).sum()
            gx, gw, gs = torch.autograd.grad(total, [part, w, head], allow_unused=True)
            dx[row, lo:hi] = gx.reshape(hi - lo, H, C // H) if gx is not None else 0.0
            dw = dw + (gw if gw is not None else 0.0)
            ds.append(gs.T if gs is not None else torch.zeros((C, K - 1), dtype=F64, device=DEVICE))
        out["d_x" + name], out["d_conv_" + name] = dx, dw.detach()
        states.append(torch.stack(ds))
        chan0 += C
    for name in ("b", "w"):
        z = leaf(s[name + "_logit"])
        out["d_%s_logit" % name], = torch.autograd.grad(torch.sigmoid(z), [z], wide(s["d"][name]))
    if c["state"]:
        out["d_conv_state"] = torch.cat(states, 1)
    return out
