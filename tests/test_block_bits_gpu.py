"""A gradient of the block boundary has the same bits whichever others are
wanted: how rows are split and dealt out does not depend on that.  Without a
norm after the block, x is read for the gate's gradient alone; these sizes are
ones where its room in shared memory decides the split (6144 columns) or the
number of row groups (4096)."""
import pytest
import torch

from gpu_util import bits_equal
from test_block_gpu import check, make, run

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def g():
    from conftest import built_package
    return built_package()


@pytest.mark.parametrize("T,N,gate", [(F32, 4096, "channel"), (F32, 4096, "sequence"), (F32, 4096, "token"),
                                      (F32, 6144, "token"), (F32, 4098, "channel"), (F32, 6145, "token"),
                                      (BF, 8192, "channel"), (BF, 12288, "token"), (BF, 200, "sequence")])
@pytest.mark.parametrize("fmt", [0, 1], ids=["full", "e4m3"])
def test_bits_do_not_depend_on_the_gradients_wanted(g, T, N, gate, fmt):
    M = 2 * torch.cuda.get_device_properties(0).multi_processor_count + 37
    c = make(M, N, T, post=False, gate=gate, R=50)
    full = run(g, c, T, 0.9, 1.1, 0.0, fmt)
    check(c, full, 0.9, 1.1, 0.0, fmt)
    for trainable in (True, False):
        for want in (("dx", "dr"), ("dr",), ("dx", "dgate"), ("dgate",), ()):
            o = run(g, c, T, 0.9, 1.1, 0.0, fmt, trainable=trainable, want=want)
            for k in want:
                assert bits_equal(o[k].view, full[k].view), (k, want, trainable)
            if trainable:
                assert bits_equal(o["dw_pre"], full["dw_pre"]), want
