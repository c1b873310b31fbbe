"""Tokens drawn from batches whose rows shared memory does not hold: each pass reads them
again, one CTA a row or two. All rows are drawn in one call, a few of them compared with
the float64 oracle."""

import numpy as np
import pytest
import torch

from online_softmax_attention_rf_gb300 import api
from oracle import tree
from tests.helpers import f64
from tests.test_gpu_sample import LOGPROB, NEAR, _f32, _i32

pytestmark = pytest.mark.gpu

# 200 rows of 50001 float32: a CTA a row; the other two: two CTAs a row (rows resident
# together would not fit L2; a thread would have more than 200 logits)
SIZES = [(200, 50001, torch.float32), (512, 131072, torch.float32), (200, 131072, torch.bfloat16)]


def _rows(kind, B, V, gen):
    def normal():
        return torch.randn(B, V, generator=gen, device="cuda")

    if kind == "normal":
        return 2 * normal()
    if kind == "levels":      # every cut falls among equal logits
        return (3 * normal()).round() / 2
    if kind == "near flat":   # most rows' logits in the first step, cuts next to the maximum
        return 1e-3 * normal()
    if kind == "masked":
        hide = torch.rand(B, V, generator=gen, device="cuda") < 0.6
        return torch.where(hide, -float("inf"), 2 * normal())


@pytest.mark.parametrize("kind", ["normal", "levels", "near flat", "masked"])
@pytest.mark.parametrize("B,V,dtype", SIZES)
def test_rows_that_are_read_again(cuda_device, B, V, dtype, kind):
    gen = torch.Generator(device="cuda").manual_seed(B + V)
    rng = np.random.default_rng(B + V)
    x = _rows(kind, B, V, gen).to(dtype)
    expo = torch.empty(B, V, device="cuda").exponential_(generator=gen).clamp_(min=1e-20)
    i = np.arange(B)
    temp = np.where(i % 16 == 15, 0.0, 0.5 + rng.random(B)).tolist()
    k = np.where(i % 2 == 0, np.exp(rng.uniform(0, np.log(V), B)).astype(int), 0).tolist()
    p = np.where(i % 4 <= 1, 0.05 + 0.94 * rng.random(B), 1.0).tolist()
    m = np.where(i % 8 >= 6, 0.5 * rng.random(B) ** 3, 0.0).tolist()
    token, lp = api.sample_rows(x, expo, _f32(temp), _i32(k), _f32(p), _f32(m))
    assert api.device_status() == 0
    again = api.sample_rows(x, expo, _f32(temp), _i32(k), _f32(p), _f32(m))
    assert torch.equal(again[0], token) and torch.equal(again[1], lp)
    pick = sorted(rng.choice(B, 32, replace=False).tolist())
    xs, es = f64(x[pick]), f64(expo[pick])
    seen = 0
    for a, e, b in zip(xs, es, pick):
        f = [float(np.float32(v[b])) for v in (temp, p, m)]
        want, lp_ref, margin = tree.sample(a, e, f[0], k[b], f[1], f[2])
        lps = [lp_ref]
        if margin < NEAR:    # as test_gpu_sample: a border that errors may move
            near = [tree.sample(a, e, f[0], k[b], f[1] * s if f[1] < 1 else 1.0, f[2] * s,
                                draw_alone=True) for s in (1 - NEAR, 1 + NEAR)]
            if any(t != want or mg < NEAR for t, _, mg in near):
                continue
            lps += [q for _, q, _ in near]
        seen += 1
        assert token[b].item() == want, (b, k[b], f)
        tol = LOGPROB * (1 + abs(lp_ref))
        assert min(lps) - tol <= lp[b].item() <= max(lps) + tol, (b, k[b], f)
    assert seen >= 24
