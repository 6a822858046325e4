"""A single row may come with any row stride (a column turned on its side, a row
of an expanded tensor): the functions take it, in both directions."""
import pytest
import torch

N = 40


def odd_rows(like):
    """[1, N] tensors whose row stride is less than N, of like's values."""
    out = {"column": like.reshape(N, 1).clone().t(), "expanded": like.reshape(N).clone().expand(5, N)[:1]}
    assert all(t.shape == (1, N) and t.stride(0) < N and t.is_contiguous() for t in out.values())
    return out


def test_rows_of_their_own_stride():
    from conftest import built_package
    built_package()
    from row_normalization_rmsnorm_gb300 import autograd as AG
    for t in odd_rows(torch.arange(float(N))).values():
        r = AG._rows(t)
        assert r.stride() == (N, 1) and torch.equal(r, t) and r.data_ptr() == t.data_ptr()
    one = torch.zeros(()).expand(1, 1)
    assert AG._rows(one).stride(0) == AG._rows(one[None]).stride(0) == 1 and AG._rows(torch.zeros(0, N)).shape == (0, N)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["column", "expanded"])
@pytest.mark.parametrize("ck", [None, "e4m3", "int8"])
def test_single_rows(kind, ck):
    from conftest import built_package
    built_package()
    from row_normalization_rmsnorm_gb300 import autograd as AG
    g = torch.Generator(device="cuda").manual_seed(5)
    x, r, dy, w, gate = (torch.randn(1, N, generator=g, device="cuda") for _ in range(5))
    w, b = w[0], gate[0].clone()

    def run(x, r, dy, gate):
        x, r, gate = (t.detach().requires_grad_() for t in (x, r, gate))
        outs = [AG.rms_norm(x, w, checkpoint=ck), AG.layer_norm(x, w, b, checkpoint=ck),
                *AG.fused_add_rms_norm(x, r, w, checkpoint=ck),
                *AG.block_rms_norm(x, r, w, w, gate=gate, checkpoint=ck)]
        return outs + list(torch.autograd.grad(outs, (x, r, gate), [dy] * len(outs)))

    plain = run(x, r, dy, gate)
    got = run(*(odd_rows(t)[kind] for t in (x, r, dy, gate)))
    for a, b2 in zip(got, plain):
        assert torch.equal(a, b2)
