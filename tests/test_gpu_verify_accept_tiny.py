"""Draft acceptance where the weights lie at the bottom of fp32: u times their sum is no longer a pair of
normal numbers, and the answer still has to be the definition's (tests/gdr_ref.py, in 64 bits)."""
import pytest
import torch

import rwkv_linear_attention_gb300 as wkv7
from tests import gdr_ref
from tests.test_gpu_verify_accept import dev  # noqa: F401

pytestmark = pytest.mark.gpu

TOP = 1 - 2.0 ** -24
THRESHOLDS = [0.0, 1e-45, 2.0 ** -60, 0.25, 0.3, 0.5, 0.6, 0.9, TOP]


def _rows(dev, V, rows, none):
    """One row per (weights, threshold), no drafts: the target's row alone, all-accepted."""
    B = len(rows)
    p = torch.zeros(B, 2, V, device=dev)
    un = torch.empty(B)
    for b, (weights, u) in enumerate(rows):
        for v, w in weights.items():
            p[b, :, v] = w
        un[b] = u
    tok = torch.zeros(B, 1, dtype=torch.int32, device=dev)
    lens = torch.zeros(B, dtype=torch.int32, device=dev) if none else None
    return p, tok, torch.zeros(B, 1, device=dev), un.to(dev), lens


# one CTA a row, and eight
@pytest.mark.parametrize("V", [300, 65536])
def test_tiny_weights(dev, V):  # noqa: F811
    tiny = 2.0 ** -149
    sets = [{V - 3: tiny}, {5: tiny, V - 3: 2 * tiny}, {5: tiny, 6: tiny, V // 2: tiny, V - 1: tiny}, {7: 2.0 ** -126}, {7: 2.0 ** -127, V - 2: 2.0 ** -127},
            {1: 1e-40, V - 2: 2e-40}, {3: 2.0 ** -100, V - 1: 2.0 ** -110}, {3: 2.0 ** -149, 4: 1.0}, {3: 2.0 ** -149, V - 2: 2.0 ** 100}]
    rows = [(w, u) for w in sets for u in THRESHOLDS]
    p, tok, u, un, lens = _rows(dev, V, rows, True)
    n_out = torch.full((len(rows),), -7, dtype=torch.int32, device=dev)
    t_out = torch.full((len(rows),), -7, dtype=torch.int32, device=dev)
    wkv7.verify_accept(tok, p, u, un, draft_lens=lens, accept_len=n_out, next_token=t_out)
    wkv7.check_device_status()
    n_ref, t_ref = gdr_ref.accept(tok.cpu().numpy(), p.cpu().numpy(), u.cpu().numpy(), un.cpu().numpy(), None, lens.cpu().numpy())
    assert n_out.tolist() == n_ref.tolist()
    assert t_out.tolist() == t_ref.tolist()


def test_tiny_residual_of_a_refused_draft(dev):  # noqa: F811
    """What the target has above the draft is a single subnormal weight."""
    V = 1000
    q = torch.zeros(3, 1, V, device=dev)
    q[:, 0, 10] = 1.0
    p = torch.zeros(3, 2, V, device=dev)
    p[:, 0, 10] = 0.5
    p[:, 0, 700] = 2.0 ** -149
    p[:, 1] = 1.0 / V
    tok = torch.full((3, 1), 10, dtype=torch.int32, device=dev)
    out = torch.full((3,), -7, dtype=torch.int32, device=dev)
    n, t = wkv7.verify_accept(tok, p, torch.full((3, 1), 0.75, device=dev), torch.tensor([0.0, 0.6, TOP], device=dev), draft_probs=q, next_token=out)
    assert n.tolist() == [1, 1, 1] and t.tolist() == [700, 700, 700]
