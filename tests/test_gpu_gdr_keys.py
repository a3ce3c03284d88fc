"""The gated delta rule where keys repeat and the strength reaches 2 (reflections), against its
definition in 64 bits (tests/gdr_ref.py): the products over a chunk no longer die out with the distance of
two tokens, and the chunk's inverse is far from the identity.

Tolerances, max |x - ref| / max |ref| per tensor, for unit keys and 0 <= beta <= 2.  I - beta k k^T and its
products then have norm at most 1, so no element of a chunk's inverse is above 2, and a token's err is
a sum of at most 64 terms of that size.  The chunked kernels hold each term's vector as a pair of bf16, off by
at most 2^-17 of itself: all 64 together 64 * 2 * 2^-17 = 2^-10 of the largest.  That is the
bound for the outputs and states; where the errors add with random signs, as they do, it leaves
room for sqrt(64) chunks that forget nothing.  A gradient reads such sums twice (err and dv): 2^-9, and
dg, whose sums' terms may be four times the result, 2^-7.  dq, dk and dv are rounded to bf16, half a step 2^-8, more.
fp32 inputs: the same sums in fp32, 128 terms of 2^-24, over a few hundred tokens that forget nothing: 1e-4.
"""
import pytest
import torch

import rwkv_linear_attention_gb300 as wkv7
from tests import gdr_ref
from tests.gpu_util import rel_err

pytestmark = pytest.mark.gpu

SUM64 = 2.0 ** -10
STEP = 2.0 ** -8
BOUND = dict(dq=2 * SUM64 + STEP, dk=2 * SUM64 + STEP, dv=2 * SUM64 + STEP, dg=8 * SUM64, dbeta=2 * SUM64, ds0=2 * SUM64)
IN = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from rwkv_linear_attention_gb300 import build
    build.build()
    return torch.device("cuda:0")


def _draw(keys, beta, decay, lens, Hk, Hv, N, dev, dtype):
    x = gdr_ref.draw(lens, Hk, Hv, N, 17 + sum(lens), dev, torch.float32)
    gen = torch.Generator(device=dev).manual_seed(3)
    T = sum(lens)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if keys == "one":  # every token writes to the same key
        k = normal(1, Hk, N).expand(T, Hk, N)
    elif keys == "near":
        k = normal(1, Hk, N) + 0.1 * normal(T, Hk, N)
    elif keys == "eight":
        k = normal(8, Hk, N)[torch.randint(0, 8, (T,), generator=gen, device=dev)]
    else:  # "walk": neighbours are alike
        k = normal(T, Hk, N).cumsum(0)
    x["k"] = k / k.norm(dim=-1, keepdim=True)
    x["beta"].fill_(beta)
    x["g"].fill_(-decay)
    for n in ("q", "k", "v", "do"):
        x[n] = x[n].to(dtype)
    # rounded to bf16 a key is no longer of length 1: where beta is 2 its length must not pass 1, or the state grows
    if dtype == torch.bfloat16 and beta == 2:
        x["k"] = (x["k"].float() * (1 - 2.0 ** -8)).to(dtype)
    return x


CASES = [("one", 1.0, 1e-3), ("one", 1.99, 1e-3), ("one", 2.0, 0.0), ("near", 1.0, 0.0), ("near", 1.99, 1e-3), ("near", 2.0, 0.0),
         ("eight", 1.99, 0.0), ("walk", 1.0, 0.0), ("walk", 2.0, 0.0)]


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("keys,beta,decay", CASES)
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16], ids=["x32", "xbf16"])
def test_prefill(dev, keys, beta, decay, N, xt):
    x = _draw(keys, beta, decay, [640, 90], 1, 2, N, dev, xt)
    o_ref, s_ref = gdr_ref.run(*(x[n] for n in IN), x["cu"], x["s0"])
    o, s = wkv7.gdr_prefill(*(x[n] for n in IN), x["cu"].to(dev), initial_state=x["s0"])
    wkv7.check_device_status()
    tol = SUM64 if xt == torch.bfloat16 else 1e-4
    assert rel_err(o, o_ref) <= tol and rel_err(s, s_ref) <= tol


@pytest.mark.parametrize("keys,beta,decay", [("one", 1.99, 1e-3), ("near", 2.0, 0.0)])
def test_prefill_in_segments(dev, keys, beta, decay):
    """Long enough to run in segments at once, whose states are carried by products of their own."""
    x = _draw(keys, beta, decay, [2500], 1, 1, 64, dev, torch.bfloat16)
    o_ref, s_ref = gdr_ref.run(*(x[n] for n in IN), x["cu"], x["s0"])
    o, s = wkv7.gdr_prefill(*(x[n] for n in IN), x["cu"].to(dev), initial_state=x["s0"])
    wkv7.check_device_status()
    assert rel_err(o, o_ref) <= SUM64 and rel_err(s, s_ref) <= SUM64


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("keys,beta,decay", CASES)
def test_gradients(dev, keys, beta, decay, N):
    x = _draw(keys, beta, decay, [300, 70], 1, 2, N, dev, torch.bfloat16)
    got = dict(zip(BOUND, wkv7.gdr_prefill_backward(*(x[n] for n in IN), x["cu"].to(dev), x["do"], initial_state=x["s0"],
                                                    d_final_state=x["dsf"])))
    wkv7.check_device_status()
    ref = dict(zip(BOUND, gdr_ref.gradients(x)))
    for n in BOUND:
        assert rel_err(got[n], ref[n]) <= BOUND[n], n
