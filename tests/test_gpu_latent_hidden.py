"""spec_latent_attention: a node's finite row, however large its scores, leaves the
outputs of nodes that do not see it bit for bit."""

import pytest
import torch

import test_gpu_latent_attention as att
from rejection_sampling_verifier_amd import binding

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    binding.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("C,dv", [(576, 512), (288, 256)])
@pytest.mark.parametrize("N,H", [(6, 4), (20, 3), (12, 16), (40, 2)])  # rows that fill 32, 64 and more than 64; two tiles of nodes
@pytest.mark.parametrize("by", [3.0, 40.0])
@pytest.mark.parametrize("lens", [(60, 33, 48), (700,) * 40])  # one workgroup a sequence; several tiles of each in one
def test_large_rows_of_hidden_nodes(N, H, C, dv, dtype, by, lens):
    """Node 1 is on nobody's path but its own; its row is a multiple of a query of its own, so that its score
    lies far above all others."""
    s = att.make(N=N, H=H, C=C, dv=dv, lens=lens, B=len(lens), dtype=dtype)
    s["parent"][:, 1] = 0
    s["parent"][:, 2:][s["parent"][:, 2:] == 1] = 0
    want = att.call(s)
    s["rows"][:, 1] = s["q"][:, 1, 0] * by
    got = att.call(s)
    keep = [i for i in range(N) if i != 1]
    assert torch.equal(got[:, keep].contiguous().view(torch.int16), want[:, keep].contiguous().view(torch.int16))
    assert (got[:, 1, 0].float() - s["rows"][:, 1, :dv].float()).abs().max() <= by * 0.1
