"""Forward-mode tangents: the functions have no forward-mode derivative, so an
input that carries a tangent is refused, never answered without one.  On the
CPU the kernels' calls are stood in for by ones that write zeros."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

M, N = 4, 32
OUTPUTS = {"norm_rms_fwd": (2,), "norm_rms_fwd_ckpt": (2,), "norm_ln_fwd": (3,), "norm_ln_fwd_ckpt": (3,),
           "norm_fused_add_rms_fwd": (3, 4), "norm_fused_add_rms_fwd_ckpt": (3, 4), "norm_block_rms_fwd": (4, 5)}


@pytest.fixture
def ag(monkeypatch):
    from conftest import built_package
    built_package()
    from row_normalization_rmsnorm_gb300 import autograd as AG
    for name, outs in OUTPUTS.items():
        def stand_in(*a, outs=outs, **kw):
            for i in outs:
                if a[i] is not None:
                    a[i].zero_()
        monkeypatch.setattr(AG.B, name, stand_in)
    return AG


def functions(ag, ck):
    w = torch.ones(N)
    return [lambda x: ag.rms_norm(x, w, checkpoint=ck), lambda x: ag.layer_norm(x, w, w, checkpoint=ck),
            lambda x: ag.fused_add_rms_norm(x, torch.zeros(M, N), w, checkpoint=ck)[0],
            lambda x: ag.block_rms_norm(x, torch.zeros(M, N), w, w, checkpoint=ck)[0],
            lambda x: ag.block_rms_norm(torch.zeros(M, N), x, w, None, checkpoint=ck)[1],
            lambda x: ag.block_rms_norm(torch.zeros(M, N), torch.zeros(M, N), None, w, gate=x, checkpoint=ck)[1]]


@pytest.mark.parametrize("ck", [None, "e4m3", "int8"])
@pytest.mark.parametrize("i", range(6))
def test_tangents_are_refused(ag, ck, i):
    fn = functions(ag, ck)[i]
    x, t = torch.randn(M, N), torch.randn(M, N)
    fn(x)
    for grad in (True, False):
        with torch.set_grad_enabled(grad):
            with fwAD.dual_level(), pytest.raises(RuntimeError):
                fn(fwAD.make_dual(x, t))
            with fwAD.dual_level(), pytest.raises(RuntimeError):
                fn(fwAD.make_dual(x.clone().requires_grad_(), t))
    with pytest.raises(RuntimeError):
        torch.func.jvp(fn, (x,), (t,))


@pytest.mark.parametrize("ck", [None, "e4m3", "int8"])
def test_a_call_without_gradients_keeps_nothing(ag, ck, monkeypatch):
    seen = []
    monkeypatch.setattr(ag.B, "norm_block_rms_fwd", lambda *a, **kw: seen.append((a, kw)))
    x, w = torch.randn(2, 2, N), torch.ones(N)
    y, h = ag.block_rms_norm(x, x, w, w, gate=w, checkpoint=ck)
    with torch.no_grad():
        ag.block_rms_norm(x.clone().requires_grad_(), x, w, w, gate=w, checkpoint=ck)
    assert y.shape == h.shape == x.shape and not y.requires_grad and len(seen) == 2
    for a, kw in seen:
        assert all(t is None for t in a[6:8])                       # the statistics
        assert kw.get("x_ckpt") is None and kw.get("h_ckpt") is None and not kw.get("ckpt_format", 0)
    assert ag.block_rms_norm(x, x, w, None)[0] is None


@pytest.mark.parametrize("shape", [(4, N), (2, 2, N), (N,)])
@pytest.mark.parametrize("i", [0, 1])
def test_outputs_without_gradients_may_be_written_over(ag, shape, i):
    """With what requires a gradient, too: they are no views."""
    x, w, p = torch.randn(shape), torch.ones(N), torch.ones(N, requires_grad=True)
    for keep_graph in (True, False):
        with torch.set_grad_enabled(keep_graph):
            o = ag.block_rms_norm(x, x, w, w)[i]
        assert o.shape == shape and o.is_contiguous()
        o.add_(p)
        o.sum().backward()
    assert torch.equal(p.grad, torch.full((N,), 2.0 * x.numel() / N))
