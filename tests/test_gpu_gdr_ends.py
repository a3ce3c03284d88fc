"""The ends of the gated delta rule's chains: CTAs that leave right behind their last product (no state gradient
to write, states alone in the first pass over segments), one after another on the same SMs, keep every bit."""
import pytest
import torch

import rwkv_linear_attention_gb300 as wkv7
from tests import gdr_ref

pytestmark = pytest.mark.gpu

IN = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from rwkv_linear_attention_gb300 import build
    build.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("chunks", [1, 2, 3, 4])
def test_many_short_reverse_chains_without_state_gradients(dev, N, chunks):
    """400 chains of each kind, more than the SMs, of one to four chunks."""
    lens = [64 * chunks - 1] * 50
    x = gdr_ref.draw(lens, 4, 8, N, 400 + chunks, dev, torch.bfloat16)
    args = [x[n] for n in IN]
    cu = x["cu"].to(dev)
    want = wkv7.gdr_prefill_backward(*args, cu, x["do"], initial_state=x["s0"], d_final_state=x["dsf"])
    for _ in range(10):
        got = wkv7.gdr_prefill_backward(*args, cu, x["do"], initial_state=x["s0"], d_final_state=x["dsf"], want_d_initial_state=False)
        assert got[5] is None
        assert all(torch.equal(a, b) for a, b in zip(got[:5], want[:5]))
    wkv7.check_device_status()


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("T", [1600, 1930, 2500, 2941])
def test_segments_of_every_length_again_and_again(dev, N, T):
    x = gdr_ref.draw([T], 2, 4, N, 500 + T, dev, torch.bfloat16)
    args = [x[n] for n in IN]
    cu = x["cu"].to(dev)
    want = wkv7.gdr_prefill(*args, cu, initial_state=x["s0"])
    for _ in range(10):
        got = wkv7.gdr_prefill(*args, cu, initial_state=x["s0"])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    wkv7.check_device_status()
