"""Row lengths whose backward has the most streams to keep in shared memory:
fp32 rows with a gate per token, both norms and a gradient of h, at lengths that
the slices of a cluster do not divide."""
import pytest
import torch

from test_block_gpu import go

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def g():
    from conftest import built_package
    return built_package()


@pytest.mark.parametrize("N,lead", [(24576, 1), (24577, 0), (24580, 0), (24833, 0), (25088, 1), (25089, 0), (21504, 1),
                                    (32764, 0), (32768, 1)])
@pytest.mark.parametrize("gate", ["token", "sequence"])
def test_five_streams_of_wide_rows(g, N, lead, gate):
    go(g, 5, N, F32, gate=gate, R=2, lead=lead)


@pytest.mark.parametrize("N", [1793, 8193, 8225, 12289, 16385, 40961, 49153, 57345])
def test_uneven_slices(g, N):
    """The last slice of a row much shorter than the others, or of one column
    more than the chunks take."""
    go(g, 3, N, BF, gate="token")
    go(g, 3, N, BF, gate="token", fmt=1)
    go(g, 3, min(N, 32767), F32, gate="none", lead=1)
