"""Uses of the block boundary and the checkpointed norms beside those of the
other files: outputs over inputs with several rows a row group, a norm before
the next block alone through autograd, and fp16 rows that overflow."""
import pytest
import torch

import block_util as U
from gpu_util import bits_equal
from test_block_autograd_gpu import rnd
from test_block_gpu import d, make, run

pytestmark = pytest.mark.gpu
F32, F16, BF = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def g():
    from conftest import built_package
    return built_package()


@pytest.fixture(scope="module")
def A(g):
    from row_normalization_rmsnorm_gb300 import autograd
    return autograd


# ---- outputs over inputs, many rows a group --------------------------------
@pytest.mark.parametrize("N", [128, 1001, 2048, 9000])
@pytest.mark.parametrize("gate", ["none", "sequence", "token"])
@pytest.mark.parametrize("fmt", [0, 2], ids=["full", "int8"])
def test_backward_over_its_gradients(g, N, gate, fmt):
    M = 1500 if N > 4096 else 9000 if N < 1000 else 4000
    c = make(M, N, BF, gate=gate, R=700)
    o = run(g, c, BF, 0.9, 1.0, 0.0, fmt)
    gv = None if c["g"] is None else c["g"].view
    rows = 0 if gv is None else gv.shape[0]
    for dx_over, dr_over in (("dy", "dh"), ("dh", "dy"), ("dh", None), (None, "dy")):
        t = {"dy": c["dy"].view.clone(), "dh": c["dh"].view.clone(), None: None}
        w1, w2 = torch.empty_like(c["w1"]), torch.empty_like(c["w2"])
        dg = None if gv is None else torch.empty_like(gv)
        nb = g.norm_block_bwd_workspace_bytes(M, N, rows, True, True, dg is not None)
        g.norm_block_rms_bwd(t["dy"], t["dh"], o["xq"] if fmt else c["x"].view, o["hq"] if fmt else o["h"].view, c["w1"],
                             c["w2"], o["rs1"], o["rs2"], t[dx_over], t[dr_over], w1, w2, gate=gv, dgate=dg,
                             rows_per_gate=c["R"], saved_format=fmt,
                             workspace=torch.empty(nb, dtype=torch.uint8, device="cuda"), residual_scale=0.9)
        for over, k in ((dx_over, "dx"), (dr_over, "dr")):
            assert over is None or bits_equal(t[over], o[k].view), (k, over)
        assert bits_equal(w1, o["dw_post"]) and bits_equal(w2, o["dw_pre"])
        assert dg is None or bits_equal(dg, o["dgate"].view)


@pytest.mark.parametrize("N", [128, 1001, 2048, 9000])
@pytest.mark.parametrize("fmt", [1, 2], ids=["e4m3", "int8"])
@pytest.mark.parametrize("op", ["rms", "ln", "fadd"])
def test_checkpointed_norms_over_their_inputs(g, op, N, fmt):
    M = 1500 if N > 4096 else 9000 if N < 1000 else 4000
    gen = torch.Generator(device="cuda").manual_seed(N)
    x, r, dy, dh = (torch.randn(M, N, generator=gen, device="cuda").to(BF) for _ in range(4))
    w, b = (torch.randn(N, generator=gen, device="cuda").to(BF) for _ in range(2))
    rb = g.norm_ckpt_row_bytes(N)
    ws = torch.empty(g.norm_bwd_workspace_bytes(M, N, True, op == "ln"), dtype=torch.uint8, device="cuda")

    def forward(x, r, y, h):
        q, rs = torch.zeros(M, rb, dtype=torch.uint8, device="cuda"), torch.empty(M, device="cuda")
        if op == "rms":
            g.norm_rms_fwd_ckpt(x, w, y, rs, q, fmt)
        elif op == "ln":
            g.norm_ln_fwd_ckpt(x, w, b, y, None, rs, q, fmt)
        else:
            g.norm_fused_add_rms_fwd_ckpt(x, r, w, y, h, rs, q, fmt)
        return q, rs

    def backward(dy, dh, q, rs, dx):
        dw, db = torch.empty_like(w), torch.empty_like(w)
        if op == "rms":
            g.norm_rms_bwd_ckpt(dy, q, fmt, w, rs, dx, dw, ws)
        elif op == "ln":
            g.norm_ln_bwd_ckpt(dy, q, fmt, w, rs, dx, dw, db, ws)
        else:
            g.norm_fused_add_rms_bwd_ckpt(dy, dh, q, fmt, w, rs, dx, dw, ws)
        return [dw] + ([db] if op == "ln" else [])

    y, h, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    q, rs = forward(x, r, y, h)
    dws = backward(dy, dh, q, rs, dx)
    for swap in (False, True)[:2 if op == "fadd" else 1]:
        x2, r2 = x.clone(), r.clone()
        y2, h2 = (r2, x2) if swap else (x2, r2)
        q2, rs2 = forward(x2, r2, y2, h2)
        assert bits_equal(y2, y) and torch.equal(q2, q) and torch.equal(rs2, rs)
        assert op != "fadd" or bits_equal(h2, h)
        dy2, dh2 = dy.clone(), dh.clone()
        dx2 = dh2 if swap else dy2
        assert all(bits_equal(p, t) for p, t in zip(backward(dy2, dh2, q, rs, dx2), dws))
        assert bits_equal(dx2, dx)


# ---- autograd without a norm after the block --------------------------------
@pytest.mark.parametrize("ckpt", [None, "e4m3", "int8"])
@pytest.mark.parametrize("shape", ["none", "channel", "sequence", "token", "rows"])
def test_autograd_without_a_norm_after_the_block(A, g, ckpt, shape):
    B, T, N = 3, 20, 1024
    x, r, w2 = rnd(B, T, N, seed=1, grad=True), rnd(B, T, N, seed=2, grad=True), rnd(N, seed=4, grad=True)
    sizes = {"none": None, "channel": (N,), "sequence": (B, 1, N), "token": (B, T, N), "rows": (6, N)}[shape]
    gate = None if sizes is None else rnd(*sizes, seed=5, grad=True)
    R = {"none": None, "channel": None, "sequence": T, "token": 1, "rows": 10}[shape]
    dy, dh = rnd(B, T, N, seed=6), rnd(B, T, N, seed=7)
    fmt = A.CHECKPOINT_FORMATS[ckpt]
    g2 = None if gate is None else gate.detach() if shape in ("channel", "rows") else gate.detach().reshape(-1, N)
    flat = [t.detach().view(-1, N) for t in (x, r, dy, dh)]
    want = without_post(g, flat[0], flat[1], w2.detach(), g2, R, flat[2], flat[3], fmt, 0.9, 0.5, 1.0)
    for train_gate in (True, False)[:1 if gate is None else 2]:
        gt = None if gate is None else gate if train_gate else gate.detach()
        y, h = A.block_rms_norm(x, r, None, w2, gate=gt, rows_per_gate=10 if shape == "rows" else None,
                                residual_scale=0.9, block_scale=0.5, eps=EPS, offset=1.0, checkpoint=ckpt)
        leaves = [t for t in (x, r, w2, gt) if t is not None and t.requires_grad]
        got = torch.autograd.grad([y, h], leaves, [dy, dh])
        assert bits_equal(y.detach().view(-1, N), want["y"]) and bits_equal(h.detach().view(-1, N), want["h"])
        for v, k, leaf in zip(got, ("dx", "dr", "dw_pre", "dgate"), leaves):
            assert v.shape == leaf.shape and bits_equal(v.reshape(want[k].shape), want[k]), k


def without_post(g, x, r, w2, gate, R, dy, dh, fmt, a, b, off):
    M, N = x.shape
    e = lambda: torch.empty_like(x)  # noqa: E731
    q = lambda want: torch.empty(M, g.norm_ckpt_row_bytes(N), dtype=torch.uint8, device="cuda") if want else None  # noqa: E731
    o = {"y": e(), "h": e(), "dx": e(), "dr": e(), "dw_pre": torch.empty_like(w2),
         "dgate": None if gate is None else torch.empty_like(gate)}
    s2, xq, hq = torch.empty(M, device="cuda"), q(fmt and gate is not None), q(fmt)
    g.norm_block_rms_fwd(x, r, None, w2, o["y"], o["h"], None, s2, gate=gate, rows_per_gate=R, x_ckpt=xq, h_ckpt=hq,
                         ckpt_format=fmt, residual_scale=a, block_scale=b, offset=off, eps=EPS)
    rows = 0 if gate is None else 1 if gate.dim() == 1 else gate.shape[0]
    nb = g.norm_block_bwd_workspace_bytes(M, N, rows, False, True, gate is not None)
    g.norm_block_rms_bwd(dy, dh, (xq if fmt else x) if gate is not None else None, hq if fmt else o["h"], None, w2, None, s2,
                         o["dx"], o["dr"], None, o["dw_pre"], gate=gate, dgate=o["dgate"], rows_per_gate=R,
                         saved_format=fmt, workspace=torch.empty(nb, dtype=torch.uint8, device="cuda"), residual_scale=a,
                         block_scale=b, offset=off)
    return o


def test_a_frozen_gate_keeps_no_x(A):
    """Without a norm after the block and with a frozen gate, the backward needs
    of x nothing: no checkpoint of it, and x itself may be written over."""
    M, N = 64, 2048
    x, r, w, gate = rnd(M, N, seed=1), rnd(M, N, seed=2, grad=True), rnd(N, seed=3, grad=True), rnd(N, seed=4)
    dy, dh = rnd(M, N, seed=5), rnd(M, N, seed=6)
    for ckpt in (None, "e4m3"):
        held = {}
        for frozen in (True, False):
            kept = []
            xg = x.clone().requires_grad_()
            with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
                y, h = A.block_rms_norm(xg, r, None, w, gate=gate.clone().requires_grad_(not frozen), checkpoint=ckpt)
            held[frozen] = [t for t in kept if t.dim() == 2]
            assert not frozen or all(t.data_ptr() != xg.data_ptr() for t in held[True])
            grads = torch.autograd.grad([y, h], (xg, r), [dy, dh])
            if frozen:
                first = grads
            assert all(bits_equal(p, t) for p, t in zip(grads, first))
        assert len(held[True]) == 1 and len(held[False]) == 2      # h (or its checkpoint); x too


# ---- overflow ----------------------------------------------------------------
def overflows(got, ref, tol):
    """fp16 values: the reference's rounding, infinite above the type's largest
    value and half a step (16) more."""
    top = U.TOP[F16] + 16
    over, under = ref.abs() - tol > top, ref.abs() + tol < top
    assert bool(over.any()) and bool(under.any())
    g = got.double()
    assert bool((g[over] == torch.copysign(torch.full_like(g[over], float("inf")), ref[over])).all())
    assert bool(((g - ref).abs() <= U.HALF[F16] * ref.abs() + U.TINY[F16] + tol)[under].all())


@pytest.mark.parametrize("N", [1024, 1001])
def test_fp16_overflow(g, N):
    """h beyond fp16 is infinite in h_out alone: y and the statistics come from
    the FP32 h, and so do the gradients where its checkpoint is kept.  A decoded
    or computed value beyond fp16 is infinite, one within it is not."""
    M = 40
    c = make(M, N, F16)
    c["r"].view.copy_((torch.randn(M, N, generator=torch.Generator().manual_seed(9)) * 3e4).clamp(-6.5e4, 6.5e4).half())
    c["r"].view[1] = 0.5
    o = run(g, c, F16, 1.5, 1.0, 0.0, 1)
    f = U.block_fwd(d(c["x"].view), d(c["r"].view), d(c["w1"]), d(c["w2"]), None, 1, 1.5, 1.0, 0.0, EPS)
    overflows(o["h"].view, f["h"], (1 + U.HALF[F16]) * U.K * f["h_scale"])
    U.close(o["y"].view, f["y"], f["y_scale"], what="y")
    U.close(o["rs2"], f["rs2"][:, 0], f["rs2_scale"][:, 0], what="rstd_pre")
    hq = U.decode(o["hq"], 1, N)
    assert U.near_codes(hq, f["h"], f["h_scale"], 1)
    ref = U.block_bwd(d(c["dy"].view), d(c["dh"].view), U.decode(o["xq"], 1, N), hq, d(c["w1"]), d(c["w2"]),
                      d(o["rs1"])[:, None], d(o["rs2"])[:, None], None, 1, 1.5, 1.0, 0.0)
    for k in ("dx", "dr"):
        U.close(o[k].view, ref[k], ref[k + "_scale"], what=k)
    back = torch.empty(M, N, dtype=F16, device="cuda")
    g.norm_ckpt_decode(o["hq"], 1, back)
    assert torch.equal(back, hq.to(F16)) and bool(back.isinf().any())
    # gradients that overflow
    c["dh"].view.copy_((torch.randn(M, N, generator=torch.Generator().manual_seed(8)) * 3e4).clamp(-6.5e4, 6.5e4).half())
    o = run(g, c, F16, 1.5, 1.0, 0.0, 1)
    ref = U.block_bwd(d(c["dy"].view), d(c["dh"].view), U.decode(o["xq"], 1, N), U.decode(o["hq"], 1, N), d(c["w1"]),
                      d(c["w2"]), d(o["rs1"])[:, None], d(o["rs2"])[:, None], None, 1, 1.5, 1.0, 0.0)
    overflows(o["dr"].view, ref["dr"], (1 + U.HALF[F16]) * U.K * ref["dr_scale"])
