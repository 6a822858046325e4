"""Measured cases of the block-boundary norm and of the 8-bit activation checkpoints.

Two operators of a transformer's residual stream in training and serving:

* the block boundary: the norm after a block, its gate and scales, the
  residual sum and the norm before the next block
      z = x * rstd1 * (w_post + offset);  h = a * r + b * gate * z;
      y = h * rstd2 * (w_pre + offset)
  forward, and forward + backward with every gradient;
* norms that keep their input for the backward as 8-bit codes with one
  power-of-two scale per 32 columns (e4m3 or int8): RMSNorm, LayerNorm (about
  the row's mean), fused add + RMSNorm and the block boundary, forward +
  backward; and the encoding and decoding by themselves.

`run` computes them with elementary torch operations in 32 bits, or, with
`own` true, with this package's calls.  Gradients of the stream are taken at
the saved h, which is h rounded to the activations' type (or its checkpoint),
as in this package's fused add + RMSNorm.
"""
import math

import torch

own = False

EPS = 1e-6
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def _case(name, **kw):
    c = {"name": name, "op": "block", "step": False, "api": "calls", "dtype": "bf16", "w_dtype": "bf16", "post": True,
         "pre": True, "gate": "none", "rows_per_gate": 0, "ckpt": "none", "offset": 0.0, "a": 1.0, "b": 1.0,
         "frozen": False}
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of a small batch between two layers, norms before and after (latency)
        _case("block fwd decode 16x4096", M=16, N=4096, offset=1.0),
        # a long prompt through the same boundary, the widest rows of the package's own grid
        _case("block fwd 8192x8192", M=8192, N=8192, offset=1.0),
        # a ragged prompt with odd rows and a learned scale per channel
        _case("block fwd channel 1001x4097 fp16", M=1001, N=4097, dtype="fp16", w_dtype="fp16", gate="channel"),
        # a training step, both norms trainable
        _case("block step 8192x4096", M=8192, N=4096, step=True),
        # conditioning: one gate row per sequence of 1024 tokens, residual scaled
        _case("block step sequence 8192x2048", M=8192, N=2048, step=True, gate="sequence", rows_per_gate=1024, a=0.7),
        # a gate per token, single precision, only the norm before the next block
        _case("block step token 2048x4096 fp32", M=2048, N=4096, step=True, dtype="fp32", w_dtype="fp32", post=False,
              gate="token", rows_per_gate=1, b=0.5),
        # the norm after the block alone with a learned scale per channel, through autograd, fp32 master weights
        _case("block step post autograd 8192x5120", M=8192, N=5120, step=True, api="autograd", w_dtype="fp32", pre=False,
              gate="channel"),
        # the widest boundary with both of its saved rows in 8 bits
        _case("block step ckpt 8192x8192", M=8192, N=8192, step=True, ckpt="e4m3", offset=1.0),
        # RMSNorm keeping its input in 8 bits, frozen weight (adapters)
        _case("rms step ckpt frozen 2048x8192", op="rms", M=2048, N=8192, step=True, ckpt="int8", offset=1.0, frozen=True),
        # LayerNorm the same way with its weight and bias trained
        _case("ln step ckpt 4096x4096", op="ln", M=4096, N=4096, step=True, ckpt="int8"),
        # the residual stream of a pre-norm model kept in 8 bits
        _case("fadd step ckpt 8192x8192", op="fadd", M=8192, N=8192, step=True, ckpt="e4m3"),
        # an activation put aside and brought back, ragged rows
        _case("ckpt round trip 4000x4100", op="trip", M=4000, N=4100, ckpt="int8"),
    ]


def draw(rng):
    """Any operator, type, gate and format over row lengths from 64 to 16384
    and one to 32768 rows (up to 64 M elements), odd lengths in one draw of
    four."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    N = log(64, 16384)
    if rng.random() < 0.75:
        N = max(64, N // 32 * 32)
    M = log(1, max(1, min(32768, (1 << 26) // N)))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    op = rng.choice(["block", "block", "block", "rms", "ln", "fadd", "trip"])
    if op == "ln" and dtype == "fp32":
        dtype = "bf16"
    if dtype == "fp32":
        M = max(1, M // 2)
    w_dtype = dtype
    kw = dict(op=op, M=M, N=N, dtype=dtype, offset=rng.choice([0.0, 1.0]), frozen=rng.random() < 0.25)
    if op == "block":
        kw["step"] = rng.random() < 0.7
        post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        gate = rng.choice(["none", "channel", "sequence", "token"])
        kw.update(post=post, pre=pre, gate=gate, a=rng.choice([1.0, 0.8]), b=rng.choice([1.0, 0.25]))
        kw["rows_per_gate"] = 1 if gate == "token" else min(M, log(2, 4096)) if gate == "sequence" else 0
        if dtype != "fp32" and kw["step"] and rng.random() < 0.4:
            kw["ckpt"] = rng.choice(["e4m3", "int8"])
    else:
        kw["step"] = op != "trip"
        kw["ckpt"] = rng.choice(["e4m3", "int8"])
        if dtype == "bf16" and op == "rms" and rng.random() < 0.4:
            w_dtype = "fp32"
    c = _case("", w_dtype=w_dtype, **kw)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gate_rows(case):
    if case["gate"] == "none":
        return 0
    return 1 if case["gate"] == "channel" else -(-case["M"] // case["rows_per_gate"])


def _inputs(case, seed):
    M, N, T, TW = case["M"], case["N"], DT[case["dtype"]], DT[case["w_dtype"]]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # a residual stream has channels of very different size; a block's output is about one
    loud = torch.exp(0.5 * normal(N))
    t = {"x": normal(M, N).to(T)}
    if case["op"] in ("block", "fadd"):
        t["r"] = (normal(M, N) * loud).to(T)
    elif case["op"] != "block":
        t["x"] = (t["x"].float() * loud + (0.5 if case["op"] == "ln" else 0.0)).to(T)
    near = 1.0 - case["offset"]
    if case["op"] == "block":
        t["w_post"] = (near + 0.1 * normal(N)).to(TW) if case["post"] else None
        t["w_pre"] = (near + 0.1 * normal(N)).to(TW) if case["pre"] else None
        n = _gate_rows(case)
        t["gate"] = (0.5 + 0.3 * normal(n, N)).to(TW if n == 1 and case["gate"] == "channel" else T) if n else None
    elif case["op"] != "trip":
        t["w"] = (near + 0.1 * normal(N)).to(TW)
        if case["op"] == "ln":
            t["bias"] = (0.1 * normal(N)).to(TW)
    if case["step"]:
        if case["op"] != "block" or case["pre"]:
            t["dy"] = normal(M, N).to(T)
        if case["op"] in ("block", "fadd"):
            t["dh"] = normal(M, N).to(T)
    return t


def prepare(case, seed):
    s = dict(case)
    s["t"] = _inputs(case, seed)
    if case["api"] == "autograd":  # a module's parameters and the activations of its graph
        for k in ("x", "r", "w_post", "w_pre", "gate"):
            if s["t"].get(k) is not None:
                s["t"][k].requires_grad_(not (case["frozen"] and k.startswith("w")))
    return s


# ---------------------------------------------------------------------------
# The plain form
# ---------------------------------------------------------------------------
def _saved(v, s):
    """What a backward finds of the 32-bit rows v: v rounded to the
    activations' type, or decoded from its 8-bit codes."""
    if s["ckpt"] == "none":
        return v.to(DT[s["dtype"]]).float()
    M, N = v.shape
    G = -(-N // 32)
    p = torch.nn.functional.pad(v, (0, G * 32 - N)).view(M, G, 32)
    m, e = torch.frexp(p.abs().amax(2, keepdim=True))
    if s["ckpt"] == "e4m3":   # 448 = 0.875 * 2^9 is the largest code
        k = (e - 9 + (m > 0.875).int()).clamp(min=-126)
        q = torch.ldexp(p, -k).to(torch.float8_e4m3fn).float()
    else:                     # 127 = 0.9921875 * 2^7
        k = (e - 7 + (m > 0.9921875).int()).clamp(min=-126)
        q = torch.ldexp(p, -k).round()
    return torch.ldexp(q, k).view(M, G * 32)[:, :N]


def _rows_of_gate(s, g):
    """The gate of every row, [M, N] or [1, N]."""
    if s["gate"] in ("channel", "token"):
        return g
    return g.repeat_interleave(s["rows_per_gate"], 0)[: s["M"]]


def _block_plain(s):
    t, T, TW = s["t"], DT[s["dtype"]], DT[s["w_dtype"]]
    f = {k: v.detach().float() for k, v in t.items() if v is not None}
    a, b, off = s["a"], s["b"], s["offset"]
    x, r, out = f["x"], f["r"], {}
    rs1 = None
    z = x
    if s["post"]:
        rs1 = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        z = x * rs1 * (f["w_post"] + off)
    g = _rows_of_gate(s, f["gate"]) if "gate" in f else None
    h = a * r + b * (z if g is None else g * z)
    out["h"] = h.to(T)
    if s["pre"]:
        rs2 = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        out["y"] = (h * rs2 * (f["w_pre"] + off)).to(T)
    if not s["step"]:
        return out
    dh = f["dh"]
    if s["pre"]:
        xh = _saved(h, s) * rs2
        gy = f["dy"] * (f["w_pre"] + off)
        dh = rs2 * (gy - xh * (gy * xh).mean(1, keepdim=True)) + dh
        if not s["frozen"]:
            out["dw_pre"] = (f["dy"] * xh).sum(0).to(TW)
    out["dr"] = (a * dh).to(T)
    if s["ckpt"] != "none" and (s["post"] or g is not None):
        x = _saved(x, s)
    xh = x * rs1 if s["post"] else x
    z = xh * (f["w_post"] + off) if s["post"] else x
    if g is not None:
        dg = b * dh * z
        if s["gate"] == "channel":
            dg = dg.sum(0, keepdim=True)
        elif s["gate"] == "sequence":
            R, n = s["rows_per_gate"], f["gate"].shape[0]
            dg = torch.nn.functional.pad(dg, (0, 0, 0, n * R - s["M"])).view(n, R, -1).sum(1)
        out["dgate"] = dg.to(t["gate"].dtype)
    dz = b * dh if g is None else b * g * dh
    if s["post"]:
        if not s["frozen"]:
            out["dw_post"] = (dz * xh).sum(0).to(TW)
        gz = dz * (f["w_post"] + off)
        dz = rs1 * (gz - xh * (gz * xh).mean(1, keepdim=True))
    out["dx"] = dz.to(T)
    return out


def _norm_plain(s):
    t, T, TW = s["t"], DT[s["dtype"]], DT[s["w_dtype"]]
    f = {k: v.float() for k, v in t.items()}
    w, out = f["w"] + s["offset"], {}
    h = f["x"]
    if s["op"] == "fadd":
        h = h + f["r"]
        out["h"] = h.to(T)
    mu = h.mean(1, keepdim=True) if s["op"] == "ln" else 0.0
    c = h - mu
    rs = torch.rsqrt(c.square().mean(1, keepdim=True) + EPS)
    y = c * rs * w
    out["y"] = (y + f["bias"] if s["op"] == "ln" else y).to(T)
    xh = _saved(c, s) * rs   # LayerNorm keeps its row about the mean
    gy = f["dy"] * w
    dx = gy - xh * (gy * xh).mean(1, keepdim=True)
    if s["op"] == "ln":
        dx = dx - gy.mean(1, keepdim=True)
    dx = rs * dx
    out["dx"] = (dx + f["dh"] if s["op"] == "fadd" else dx).to(T)
    if not s["frozen"]:
        out["dw"] = (f["dy"] * xh).sum(0).to(TW)
        if s["op"] == "ln":
            out["db"] = f["dy"].sum(0).to(TW)
    return out


# ---------------------------------------------------------------------------
# This package's calls
# ---------------------------------------------------------------------------
def _own_state(s):
    """Buffers a program keeps from step to step: outputs, statistics,
    checkpoints and the workspace."""
    if "o" in s:
        return s["o"]
    import row_normalization_rmsnorm_gb300 as g
    t, M, N = s["t"], s["M"], s["N"]
    x, o = t["x"], {"g": g}
    s["o"] = o

    def like():
        return torch.empty_like(x)

    def vec(n=M):
        return torch.empty(n, dtype=torch.float32, device=x.device)

    def ckpt():
        return torch.empty(M, g.norm_ckpt_row_bytes(N), dtype=torch.uint8, device=x.device)

    o["fmt"] = {"none": g.NORM_SAVED_FULL, "e4m3": g.NORM_SAVED_E4M3, "int8": g.NORM_SAVED_INT8}[s["ckpt"]]
    kept = s["ckpt"] != "none"
    if s["op"] == "trip":
        o.update(ckpt=ckpt(), out=like())
        return o
    if s["op"] == "block":
        gate = t["gate"]
        o["h"] = like()
        o["y"] = like() if s["pre"] else None
        if s["step"]:
            tw = not s["frozen"]
            o["rs1"] = vec() if s["post"] else None
            o["rs2"] = vec() if s["pre"] else None
            o["xc"] = ckpt() if kept and (s["post"] or gate is not None) else None
            o["hc"] = ckpt() if kept and s["pre"] else None
            o["dx"], o["dr"] = like(), like()
            o["dgate"] = torch.empty_like(gate) if gate is not None else None
            o["dw_post"] = torch.empty_like(t["w_post"]) if s["post"] and tw else None
            o["dw_pre"] = torch.empty_like(t["w_pre"]) if s["pre"] and tw else None
            nb = g.norm_block_bwd_workspace_bytes(M, N, _gate_rows(s), o["dw_post"] is not None,
                                                  o["dw_pre"] is not None, o["dgate"] is not None)
            o["ws"] = torch.empty(nb, dtype=torch.uint8, device=x.device) if nb else None
        return o
    o.update(y=like(), dx=like(), rs=vec(), ckpt=ckpt())
    if s["op"] == "ln":
        o["mu"] = vec()
    if s["op"] == "fadd":
        o["h"] = like()
    o["dw"] = None if s["frozen"] else torch.empty_like(t["w"])
    o["db"] = None if s["frozen"] or s["op"] != "ln" else torch.empty_like(t["w"])
    nb = g.norm_bwd_workspace_bytes(M, N, o["dw"] is not None, o["db"] is not None)
    o["ws"] = torch.empty(nb, dtype=torch.uint8, device=x.device) if nb else None
    return o


def _block_own(s):
    t, o = s["t"], _own_state(s)
    g, R = o["g"], s["rows_per_gate"] or None
    if not s["step"]:
        g.norm_block_rms_fwd(t["x"], t["r"], t["w_post"], t["w_pre"], o["y"], o["h"], gate=t["gate"], rows_per_gate=R,
                             residual_scale=s["a"], block_scale=s["b"], offset=s["offset"], eps=EPS)
        return {k: o[k] for k in ("h", "y") if o[k] is not None}
    g.norm_block_rms_fwd(t["x"], t["r"], t["w_post"], t["w_pre"], o["y"], o["h"], o["rs1"], o["rs2"], gate=t["gate"],
                         rows_per_gate=R, x_ckpt=o["xc"], h_ckpt=o["hc"], ckpt_format=o["fmt"], residual_scale=s["a"],
                         block_scale=s["b"], offset=s["offset"], eps=EPS)
    saved_x = o["xc"] if s["ckpt"] != "none" else t["x"]
    saved_h = o["hc"] if s["ckpt"] != "none" else o["h"]
    g.norm_block_rms_bwd(t.get("dy"), t["dh"], saved_x if s["post"] or t["gate"] is not None else None,
                         saved_h if s["pre"] else None, t["w_post"], t["w_pre"], o["rs1"], o["rs2"], o["dx"], o["dr"],
                         o["dw_post"], o["dw_pre"], gate=t["gate"], dgate=o["dgate"], rows_per_gate=R,
                         saved_format=o["fmt"], workspace=o["ws"], residual_scale=s["a"], block_scale=s["b"],
                         offset=s["offset"])
    return {k: o[k] for k in ("h", "y", "dx", "dr", "dgate", "dw_post", "dw_pre") if o.get(k) is not None}


def _block_autograd(s):
    from row_normalization_rmsnorm_gb300 import autograd as A
    t = s["t"]
    gate = t["gate"][0] if s["gate"] == "channel" else t["gate"]
    y, h = A.block_rms_norm(t["x"], t["r"], t["w_post"], t["w_pre"], gate=gate, rows_per_gate=s["rows_per_gate"] or None,
                            residual_scale=s["a"], block_scale=s["b"], eps=EPS, offset=s["offset"],
                            checkpoint=None if s["ckpt"] == "none" else s["ckpt"])
    leaves = {"dx": t["x"], "dr": t["r"], "dgate": t["gate"], "dw_post": t["w_post"], "dw_pre": t["w_pre"]}
    leaves = {k: v for k, v in leaves.items() if v is not None and v.requires_grad}
    outs = [(y, t.get("dy")), (h, t["dh"])] if s["pre"] else [(h, t["dh"])]
    got = torch.autograd.grad([v for v, _ in outs], list(leaves.values()), [d for _, d in outs])
    out = dict(zip(leaves, got))
    out["h"] = h.detach()
    if s["pre"]:
        out["y"] = y.detach()
    return out


def _norm_own(s):
    t, o = s["t"], _own_state(s)
    g, off = o["g"], s["offset"]
    if s["op"] == "rms":
        g.norm_rms_fwd_ckpt(t["x"], t["w"], o["y"], o["rs"], o["ckpt"], o["fmt"], off, EPS)
        g.norm_rms_bwd_ckpt(t["dy"], o["ckpt"], o["fmt"], t["w"], o["rs"], o["dx"], o["dw"], o["ws"], off)
    elif s["op"] == "ln":
        g.norm_ln_fwd_ckpt(t["x"], t["w"], t["bias"], o["y"], o["mu"], o["rs"], o["ckpt"], o["fmt"], off, EPS)
        g.norm_ln_bwd_ckpt(t["dy"], o["ckpt"], o["fmt"], t["w"], o["rs"], o["dx"], o["dw"], o["db"], o["ws"], off)
    else:
        g.norm_fused_add_rms_fwd_ckpt(t["x"], t["r"], t["w"], o["y"], o["h"], o["rs"], o["ckpt"], o["fmt"], off, EPS)
        g.norm_fused_add_rms_bwd_ckpt(t["dy"], t["dh"], o["ckpt"], o["fmt"], t["w"], o["rs"], o["dx"], o["dw"], o["ws"],
                                      off)
    return {k: o[k] for k in ("h", "y", "dx", "dw", "db") if o.get(k) is not None}


def run(state):
    s = state
    if s["op"] == "trip":
        if not own:
            return {"back": _saved(s["t"]["x"].float(), s).to(DT[s["dtype"]])}
        o = _own_state(s)
        o["g"].norm_ckpt_encode(s["t"]["x"], o["ckpt"], o["fmt"])
        o["g"].norm_ckpt_decode(o["ckpt"], o["fmt"], o["out"])
        return {"back": o["out"]}
    if s["op"] == "block":
        if not own:
            return _block_plain(s)
        return _block_autograd(s) if s["api"] == "autograd" else _block_own(s)
    return _norm_own(s) if own else _norm_plain(s)


# ---------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------
def work(case):
    """Bytes and operations of a pass: a forward reads its inputs and writes
    its outputs (and checkpoints) once; a backward reads the gradients and what
    was saved once and writes the gradients of its inputs once."""
    M, N = case["M"], case["N"]
    s, sw = DT[case["dtype"]].itemsize, DT[case["w_dtype"]].itemsize
    MN = M * N
    q = M * (N + -(-N // 32)) if case["ckpt"] != "none" else 0   # one checkpoint
    kept = q if case["ckpt"] != "none" else MN * s               # one saved matrix, read again
    if case["op"] == "trip":
        return {"bytes": 2 * MN * s + 2 * q, "flops": 4 * MN}
    if case["op"] != "block":
        n = 4 if case["op"] == "fadd" else 2
        m = 3 if case["op"] == "fadd" else 2
        p = 1 if case["frozen"] else 2
        cols = (2 if case["op"] == "ln" else 1) * N * sw
        return {"bytes": (n + m) * MN * s + 2 * q + 8 * M + (1 + p) * cols, "flops": 26 * MN}
    gate = 0 if case["gate"] == "none" else _gate_rows(case) * N * (sw if case["gate"] == "channel" else s)
    norms = case["post"] + case["pre"]
    total = (3 + case["pre"]) * MN * s + norms * N * sw + gate
    if not case["step"]:
        return {"bytes": total, "flops": 12 * MN}
    saved = (1 if case["post"] or case["gate"] != "none" else 0) + (1 if case["pre"] else 0)
    total += saved * q if case["ckpt"] != "none" else 0
    total += (3 + case["pre"]) * MN * s + saved * kept + (1 if case["frozen"] else 2) * norms * N * sw + 2 * gate
    return {"bytes": total + 8 * M * norms, "flops": 42 * MN}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _codes64(v, fmt):
    """v through the 8-bit codes: for every 32 columns the smallest power of
    two that brings the largest value within the codes' range, then the
    nearest code, ties to even."""
    M, N = v.shape
    top = 448.0 if fmt == "e4m3" else 127.0
    out = torch.empty_like(v)
    whole = N // 32 * 32
    for lo, hi in ((0, whole), (whole, N)):
        if lo == hi:
            continue
        p = v[:, lo:hi].reshape(M, -1, min(32, hi - lo))
        big = p.abs().max(2, keepdim=True).values
        step = torch.exp2(torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / top)))
        step = torch.where(big > step * top, step * 2, step)
        step = torch.where(big <= step / 2 * top, step / 2, step)
        u = p / step
        if fmt == "e4m3":   # three bits after the leading one, 2^-9 the smallest spacing
            e = torch.floor(torch.log2(torch.where(u == 0, torch.ones_like(u), u.abs()))).clamp(min=-6)
            unit = torch.exp2(e - 3)
            u = torch.round(u / unit) * unit
        else:
            u = torch.round(u)
        out[:, lo:hi] = (u * step).reshape(M, hi - lo)
    return out


def exact(case, seed):
    d = {k: v.double() for k, v in _inputs(case, seed).items() if v is not None}
    T, off, fmt, N = DT[case["dtype"]], case["offset"], case["ckpt"], case["N"]

    def kept(v):
        return v.to(T).double() if fmt == "none" else _codes64(v, fmt)

    def norm_back(gv, xh, rs):
        return (gv - xh * ((gv * xh).sum(1, keepdim=True) / N)) * rs

    if case["op"] == "trip":
        return {"back": _codes64(d["x"], fmt)}
    if case["op"] != "block":
        o = {}
        h = d["x"]
        if case["op"] == "fadd":
            h = o["h"] = d["x"] + d["r"]
        W = d["w"] + off
        mu = h.sum(1, keepdim=True) / N if case["op"] == "ln" else torch.zeros_like(h[:, :1])
        rs = 1.0 / torch.sqrt(((h - mu) ** 2).sum(1, keepdim=True) / N + EPS)
        o["y"] = (h - mu) * rs * W + (d["bias"] if case["op"] == "ln" else 0.0)
        xh = kept((h.float().double() - mu) if case["op"] == "ln" else h.float().double()) * rs
        gv = d["dy"] * W
        o["dx"] = norm_back(gv, xh, rs) - (rs * gv.sum(1, keepdim=True) / N if case["op"] == "ln" else 0.0)
        if case["op"] == "fadd":
            o["dx"] = o["dx"] + d["dh"]
        if not case["frozen"]:
            o["dw"] = (d["dy"] * xh).sum(0)
            if case["op"] == "ln":
                o["db"] = d["dy"].sum(0)
        return o
    a, b, o = case["a"], case["b"], {}
    x, W1 = d["x"], d["w_post"] + off if case["post"] else 1.0
    rs1 = 1.0 / torch.sqrt((x * x).sum(1, keepdim=True) / N + EPS) if case["post"] else torch.ones_like(x[:, :1])
    gr = torch.ones_like(x[:1])
    if case["gate"] != "none":
        R = {"channel": case["M"], "token": 1}.get(case["gate"], case["rows_per_gate"])
        which = torch.arange(case["M"], device=x.device) // R
        gr = d["gate"][which]
    h = o["h"] = a * d["r"] + b * gr * (x * rs1 * W1)
    if case["pre"]:
        W2 = d["w_pre"] + off
        rs2 = 1.0 / torch.sqrt((h * h).sum(1, keepdim=True) / N + EPS)
        o["y"] = h * rs2 * W2
    if not case["step"]:
        return o
    dh = d["dh"]
    if case["pre"]:
        xh2 = kept(h) * rs2
        dh = dh + norm_back(d["dy"] * W2, xh2, rs2)
        if not case["frozen"]:
            o["dw_pre"] = (d["dy"] * xh2).sum(0)
    o["dr"] = a * dh
    if case["post"] or case["gate"] != "none":
        x = kept(x)
    xh1 = x * rs1
    if case["gate"] != "none":
        o["dgate"] = torch.zeros_like(d["gate"]).index_add_(0, which, b * dh * xh1 * W1)
    dz = b * gr * dh
    if case["post"]:
        if not case["frozen"]:
            o["dw_post"] = (dz * xh1).sum(0)
        o["dx"] = norm_back(dz * W1, xh1, rs1)
    else:
        o["dx"] = dz
    return o
