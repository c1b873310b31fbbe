"""Tokens drawn where a cut lies next to the largest logit: rows so flat that most of
them weigh as much as the maximum within a few thousandths."""

import numpy as np
import pytest
import torch

from online_softmax_attention_rf_gb300 import api
from tests.test_gpu_sample import _check, _expo

pytestmark = pytest.mark.gpu

# top_p from the largest alone to a few hundred of the logits, whose weights (about
# 1 / V, 16 times a border's tolerance at V = 8191) stay apart
SMALL_P = [0.0, 0.002, 0.005, 0.01, 0.05, -1.0, 0.0004, 0.03]


def _near_flat(kind, rows, V, gen):
    """Rows of more than 512 logits that lie within 1/16 of the maximum in units of
    ln 2, and few of them within the first 1024th of that."""
    i = torch.arange(V, dtype=torch.float64).expand(rows, V)
    if kind == "ramp":
        x = -1e-6 * i
    elif kind == "shuffled":
        x = -1e-6 * torch.argsort(torch.rand(rows, V, generator=gen), -1).double()
    elif kind == "maxima":                 # several logits equal the maximum
        x = -1e-6 * (i // 7 * 7)
        x = x.gather(1, torch.argsort(torch.rand(rows, V, generator=gen), -1))
    elif kind == "offset":                 # the maximum is not zero
        x = 0.25 - 3e-6 * torch.argsort(torch.rand(rows, V, generator=gen), -1).double()
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["ramp", "shuffled", "maxima", "offset"])
@pytest.mark.parametrize("V", [600, 4096, 8191])
def test_top_p_of_nearly_flat_rows(cuda_device, dtype, kind, V):
    gen = torch.Generator().manual_seed(V)
    x = _near_flat(kind, 8, V, gen).to(dtype).cuda()
    _, lp = _check(x, _expo(8, V, gen).cuda(), None, None, SMALL_P, None, least=0.7)
    # the largest alone (rows 0 and 5): drawn with certainty
    assert lp[0] == 0 and lp[5] == 0
    assert api.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["shuffled", "maxima"])
@pytest.mark.parametrize("V", [600, 4096])
def test_top_k_of_nearly_flat_rows(cuda_device, dtype, kind, V):
    # every count of the first few logits, and counts that take most of the row
    gen = torch.Generator().manual_seed(V + 1)
    k = [1, 2, 3, 7, 8, 50, 400, V - 50]
    x = _near_flat(kind, 8, V, gen).to(dtype).cuda()
    expo = _expo(8, V, gen).cuda()
    _, lp = _check(x, expo, None, k, None, None, least=1.0)
    assert lp[0] == 0
    _check(x, expo, None, k, [0.5] * 8, None, least=0.7)
    assert api.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_top_p_at_high_temperatures(cuda_device, dtype):
    gen = torch.Generator().manual_seed(3)
    x = (2 * torch.randn(8, 5000, generator=gen)).to(dtype).cuda()
    expo = _expo(8, 5000, gen).cuda()
    for temp in (300.0, 1e4, 1e6):
        _check(x, expo, [temp] * 8, None, SMALL_P, None, least=0.7)
        _check(x, expo, [temp] * 8, [1, 2, 5, 100, 600, 4000, 0, 4999], SMALL_P, None, least=0.6)
    assert api.device_status() == 0


def test_tokens_and_probabilities_are_saved_together(cuda_device, tmp_path):
    x = torch.zeros(3, 40, device="cuda")
    got = api.sample_rows(x, torch.ones_like(x))
    torch.save(got, tmp_path / "drawn")
    assert all(torch.equal(a, b) for a, b in zip(torch.load(tmp_path / "drawn"), got))
