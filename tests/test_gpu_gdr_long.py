"""The gated delta rule at lengths and head groups of real calls: many value heads on a key head,
thousands of tokens, segments in great number.  Bounds as in test_gpu_gdr.py and test_gpu_gdr_backward.py:
a state that decays forgets the roundings of its past, so they do not grow with the length."""
import pytest
import torch

import rwkv_linear_attention_gb300 as wkv7
from tests import gdr_ref
from tests.gpu_util import rel_err
from tests.test_gpu_gdr import CHUNKED, EXACT, HALF, IN
from tests.test_gpu_gdr_backward import BOUND

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from rwkv_linear_attention_gb300 import build
    build.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("lens,Hk,Hv,N", [([1300, 0, 65], 1, 3, 128), ([2000, 700], 2, 8, 128), ([130], 1, 8, 128), ([2500], 1, 5, 64)],
                         ids=lambda v: str(v))
@pytest.mark.parametrize("states", [True, False], ids=["states", "none"])
def test_gradients(dev, lens, Hk, Hv, N, states):
    """Value heads of a group take the gradient kernel's two places in turn: odd and even numbers of them."""
    x = gdr_ref.draw(lens, Hk, Hv, N, 600 + Hv, dev, torch.bfloat16, s0=states)
    if not states:
        x["dsf"] = None
    got = dict(zip(BOUND, wkv7.gdr_prefill_backward(*(x[n] for n in IN), x["cu"].to(dev), x["do"], initial_state=x["s0"],
                                                    d_final_state=x["dsf"], cu_seqlens_host=x["cu"])))
    wkv7.check_device_status()
    ref = dict(zip(BOUND, gdr_ref.gradients(x)))
    for n in BOUND:
        assert rel_err(got[n], ref[n]) <= BOUND[n], n


@pytest.mark.parametrize("lens,Hk,Hv,N", [([20000], 1, 2, 128), ([12000, 5000], 1, 4, 64), ([7000, 7001], 4, 8, 128)], ids=lambda v: str(v))
@pytest.mark.parametrize("st", [torch.float32, torch.bfloat16], ids=["s32", "sbf16"])
def test_prefill(dev, lens, Hk, Hv, N, st):
    x = gdr_ref.draw(lens, Hk, Hv, N, 700 + Hv, dev, torch.bfloat16)
    state = x["s0"].to(st)
    o_ref, s_ref = gdr_ref.run(*(x[n] for n in IN), x["cu"], state)
    o, s = wkv7.gdr_prefill(*(x[n] for n in IN), x["cu"].to(dev), initial_state=state, final_state=state, cu_seqlens_host=x["cu"])
    wkv7.check_device_status()
    assert s is state
    assert rel_err(o, o_ref) <= CHUNKED and rel_err(s, s_ref) <= CHUNKED + HALF[st]


def test_prefill_of_a_long_fp32_prompt(dev):
    x = gdr_ref.draw([9000, 31], 2, 4, 128, 710, dev, torch.float32)
    o_ref, s_ref = gdr_ref.run(*(x[n] for n in IN), x["cu"], x["s0"])
    o, s = wkv7.gdr_prefill(*(x[n] for n in IN), x["cu"].to(dev), initial_state=x["s0"])
    assert rel_err(o, o_ref) <= EXACT and rel_err(s, s_ref) <= EXACT
