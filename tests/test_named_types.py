"""An argument that is no tensor is a TypeError that names it, in the quick
acceptance of a call's arguments as in the checks behind it."""
import pytest
import torch

M, N = 4, 64
BF = torch.bfloat16


@pytest.fixture(scope="module")
def g():
    from conftest import built_package
    return built_package()


def block_bwd(device, **kw):
    mat, vec = torch.zeros(M, N, dtype=BF, device=device), torch.ones(N, dtype=BF, device=device)
    s = torch.ones(M, device=device)
    a = dict(dy=mat, dh_out=mat, x=mat, h=mat, w_post=vec, w_pre=vec, rstd_post=s, rstd_pre=s, dx=mat.clone(),
             dresidual=mat.clone(), gate=vec, dgate=vec.clone())
    return {**a, **kw}


@pytest.mark.parametrize("bad", [1.0, [0.0] * N, "dgate"], ids=["number", "list", "text"])
def test_dgate(g, bad):
    with pytest.raises(TypeError, match="dgate must be a torch.Tensor"):
        g.norm_block_rms_bwd(**block_bwd("cpu", dgate=bad))
    with pytest.raises(ValueError, match="dgate is given without a gate"):
        g.norm_block_rms_bwd(**block_bwd("cpu", gate=None))


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [1.0, [0.0] * N, b"0" * 4096], ids=["number", "list", "bytes"])
def test_on_a_gpu(g, bad):
    for arg in ("dgate", "workspace", "dx", "h", "dw_pre", "rstd_pre", "gate"):
        with pytest.raises(TypeError, match=f"{arg} must be a torch.Tensor"):
            g.norm_block_rms_bwd(**block_bwd("cuda", **{arg: bad}))
    for dtype in (BF, torch.float32):
        mat, vec = torch.zeros(M, N, dtype=dtype, device="cuda"), torch.ones(N, dtype=dtype, device="cuda")
        s, q = torch.ones(M, device="cuda"), torch.zeros(M, g.norm_ckpt_row_bytes(N), dtype=torch.uint8, device="cuda")
        for call in (lambda: g.norm_rms_bwd_ckpt(mat, q, 1, vec, s, mat.clone(), vec.clone(), bad),
                     lambda: g.norm_ln_bwd_ckpt(mat, q, 1, vec, s, mat.clone(), vec.clone(), None, bad),
                     lambda: g.norm_fused_add_rms_bwd_ckpt(mat, None, q, 1, vec, s, mat.clone(), vec.clone(), bad),
                     lambda: g.norm_rms_bwd(mat, mat, vec, s, mat.clone(), vec.clone(), bad),
                     lambda: g.norm_ln_bwd(mat, mat, vec, s, s, mat.clone(), vec.clone(), None, bad),
                     lambda: g.norm_fused_add_rms_bwd(mat, None, mat, vec, s, mat.clone(), vec.clone(), bad)):
            with pytest.raises(TypeError, match="workspace must be a torch.Tensor"):
                call()
