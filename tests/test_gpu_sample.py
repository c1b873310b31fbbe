"""Tokens drawn with temperature, top-k, top-p and min-p on the GPU against the
float64 oracle."""

import numpy as np
import pytest
import torch

from online_softmax_attention_rf_gb300 import api
from oracle import tree
from tests.helpers import f64

pytestmark = pytest.mark.gpu

# A weight's exponent, (max - x) log2(e) / T, has four roundings in float32
# (difference, quotient, constant, product): a weight of e^-s is off by 4 * 2^-24 s
# relatively, 2^-17 at s = 32, where weights count no more; the exponential, the
# quotient by expo and the sums add less than 2^-20. A border nearer than that
# may be passed.
NEAR = 2.0 ** -17 + 2.0 ** -20
# the same of the token's own exponent (s <= 32 nats), and the logarithm of the sum
LOGPROB = 2.0 ** -17 + 2.0 ** -19


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _f32(x):
    return None if x is None else torch.tensor(x, dtype=torch.float32, device="cuda")


def _expo(B, V, gen):
    return torch.empty(B, V).exponential_(generator=gen).clamp_(1e-20)


def _check(logits, expo, temp=None, k=None, p=None, m=None, least=0.9):
    """Draws, compared row by row with the oracle's where no border is too near (of at
    least a share `least` of the rows)."""
    B = logits.shape[0]
    token, lp = api.sample_rows(logits, expo, _f32(temp), _i32(k), _f32(p), _f32(m))
    x, e, token, lp = f64(logits), f64(expo), token.cpu().tolist(), f64(lp)
    f = lambda v, i, d: d if v is None else float(np.float32(v[i]))  # noqa: E731
    seen = 0
    for b in range(B):
        t_ref, lp_ref, margin = tree.sample(x[b], e[b], f(temp, b, 1.0), 0 if k is None else k[b],
                                            f(p, b, 1.0), f(m, b, 0.0))
        if margin < NEAR:
            # a cut of top_p or min_p that errors may move lies between those of the
            # limits moved by as much: where both draw this token, so does it
            near = [tree.sample(x[b], e[b], f(temp, b, 1.0), 0 if k is None else k[b],
                                f(p, b, 1.0) * s if f(p, b, 1.0) < 1 else 1.0, f(m, b, 0.0) * s,
                                draw_alone=True) for s in (1 - NEAR, 1 + NEAR)]
            if any(t != t_ref or mg < NEAR for t, _, mg in near):
                continue
            lps = [q for _, q, _ in near] + [lp_ref]
        else:
            lps = [lp_ref]
        seen += 1
        assert token[b] == t_ref, (b, token[b], t_ref, margin)
        if t_ref < 0:
            assert np.isnan(lp[b])
        else:
            tol = LOGPROB * (1 + abs(lp_ref))
            assert min(lps) - tol <= lp[b] <= max(lps) + tol, (b, lp[b], lp_ref)
    assert seen >= least * B
    return token, lp


LIMITS = {
    "none": (None, None, None),
    "k": (True, None, None),
    "p": (None, True, None),
    "m": (None, None, True),
    "kp": (True, True, None),
    "pm": (None, True, True),
    "kpm": (True, True, True),
}


def _limits(kind, B, V, rng):
    k, p, m = LIMITS[kind]
    return (rng.integers(0, max(2, V + 2), B).tolist() if k else None,
            (0.02 + 1.03 * rng.random(B)).tolist() if p else None,
            (0.6 * rng.random(B) ** 3).tolist() if m else None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", list(LIMITS))
@pytest.mark.parametrize("B,V,sharp", [
    (5, 1, 1.0), (6, 2, 1.0), (7, 7, 1.0), (9, 33, 2.0), (40, 257, 3.0), (33, 1000, 0.1),
    (20, 2048, 2.0), (12, 4099, 4.0), (16, 8191, 2.0), (9, 32000, 2.5), (3, 50001, 1.0),
])
def test_sample_rows(cuda_device, dtype, kind, B, V, sharp):
    gen = torch.Generator().manual_seed(V + B)
    rng = np.random.default_rng(V)
    logits = (sharp * torch.randn(B, V, generator=gen)).to(dtype).cuda()
    temp = (0.5 + rng.random(B)).tolist()
    k, p, m = _limits(kind, B, V, rng)
    _check(logits, _expo(B, V, gen).cuda(), temp, k, p, m, least=0.5 if V < 50 else 0.8)
    assert api.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_rows_small_limits_of_large_rows(cuda_device, dtype):
    # k of a few, of a thousand, and of most of the row; p and min_p from a token to all
    V = 131072
    gen = torch.Generator().manual_seed(3)
    k = [1, 2, 5, 50, 1000, 100000, 131071, 131072, 0, -3, 7, 40]
    p = [1.0, 0.5, 0.9, 0.95, 0.999, 0.3, 0.99999, 1.5, 1e-6, 0.0, -1.0, 0.7]
    m = [0.0, 0.1, 0.0, 0.01, 0.0, 0.001, 0.0, 0.0, 0.0, 0.0, 0.5, 2.0]
    logits = (2.5 * torch.randn(12, V, generator=gen)).to(dtype).cuda()
    expo = _expo(12, V, gen).cuda()
    temp = (0.3 + torch.rand(12, generator=gen)).tolist()
    _check(logits, expo, temp, k, p, m)
    _check(logits, expo, None, k, None, None)
    _check(logits, expo, temp, None, p, m)
    assert api.device_status() == 0


def test_sample_rows_of_the_largest_vocabulary(cuda_device):
    # rows that shared memory does not hold; equal numbers in great numbers
    gen = torch.Generator().manual_seed(4)
    for dtype, V in [(torch.float32, 1 << 20), (torch.bfloat16, (1 << 20) - 5)]:
        logits = torch.randn(3, V, generator=gen).to(dtype).cuda()
        expo = _expo(3, V, gen).cuda()
        _check(logits, expo, [1.0, 0.5, 2.0], [0, 300000, 5], [0.5, 0.9, 1.0], None)
        flat = torch.zeros(2, V, dtype=dtype, device="cuda")
        _check(flat, expo[:2], None, [0, V - 1], [0.75, 1.0], None)
        _check(flat, expo[:2], None, None, None, None)
    assert api.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [24, 5000, 40000])
def test_sample_rows_ties_go_to_the_lowest_index(cuda_device, dtype, V):
    # a few values only: every cut falls among equal logits; expo that prefers high
    # indices, so that a token too many would show
    gen = torch.Generator().manual_seed(V)
    x = torch.randint(-3, 4, (24, V), generator=gen).to(dtype)
    x[::2] = x[::2] * 0.0          # zeros of both signs
    x[::4] = -x[::4]
    expo = (torch.arange(V, 0, -1).float() / V).expand(24, V).contiguous()
    k = [1 + i * V // 24 for i in range(24)]
    _check(x.cuda(), expo.cuda(), None, k, None, None, least=1.0)
    # half a token's weight over a border of a flat row (every second one)
    p = [(i + 0.5) / V if V < 100 else 0.04 * i + 0.01 + 0.3 / V for i in range(24)]
    _check(x.cuda(), expo.cuda(), None, None, p, None, least=0.4)
    _check(x.cuda(), expo.cuda(), None, k, p, None, least=0.4)
    # all the same and no limit: the lowest index
    token, lp = api.sample_rows(torch.ones(2, V, dtype=dtype, device="cuda"),
                                torch.ones(2, V, device="cuda"))
    assert token.tolist() == [0, 0]
    assert np.allclose(f64(lp), -np.log(V), atol=1e-5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [9, 3001, 70000])
def test_sample_rows_masked_logits(cuda_device, dtype, V):
    gen = torch.Generator().manual_seed(V)
    x = 3 * torch.randn(16, V, generator=gen)
    low = torch.finfo(dtype).min
    hide = torch.rand(16, V, generator=gen) < 0.7
    x[:8] = torch.where(hide[:8], -float("inf"), x[:8])
    x[8:] = torch.where(hide[8:], low, x[8:])       # the type's lowest value
    x[3] = -float("inf")
    x[3, V // 2] = -2.0                             # one token is left
    x[11] = low                                     # lowest values alone: a flat row
    x = x.to(dtype).cuda()
    expo = _expo(16, V, gen).cuda()
    for k, p in [(None, None), ([V // 2] * 16, None), (None, [0.9] * 16), ([5] * 16, [0.5] * 16)]:
        token, _ = _check(x, expo, None, k, p, None, least=0.6)
        assert token[3] == V // 2
        # nothing hidden is drawn while anything else is there
        assert all(x[b, t] > low for b, t in enumerate(token) if (x[b] > low).any())
    assert api.device_status() == 0


@pytest.mark.parametrize("V", [5, 9000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_sample_rows_refuses_rows_without_probabilities(cuda_device, V, bad):
    x = torch.zeros(4, V, device="cuda")
    x[1, V - 1] = bad
    if bad < 0:
        x[1] = bad
    x[2] = x[1]
    token, lp = api.sample_rows(x, torch.ones_like(x), _f32([1, 1, 0, 1]), None, _f32([0.5] * 4))
    assert token.tolist() == [0, -1, -1, 0]
    assert lp.isnan().tolist() == [False, True, True, False]
    with pytest.raises(api.RFError):
        api.device_status()


def test_sample_rows_greedy(cuda_device):
    gen = torch.Generator().manual_seed(5)
    for dtype, V in [(torch.float32, 32000), (torch.bfloat16, 50001), (torch.bfloat16, 3)]:
        x = torch.randn(6, V, generator=gen).to(dtype).cuda()
        expo = _expo(6, V, gen).cuda()
        token, lp = api.sample_rows(x, expo, _f32([0, -1, float("nan"), 0, 1e-30, 0]),
                                    _i32([5] * 6), _f32([0.9] * 6))
        best = [int(np.argmax(r)) for r in f64(x)]
        assert token.tolist()[:4] == best[:4] and token[5] == best[5]
        assert (f64(lp)[[0, 1, 2, 3, 5]] == 0).all()
    assert api.device_status() == 0


@pytest.mark.parametrize("temp", [1e-44, 2e-39, 1e-3, 1e4, 3e38])
def test_sample_rows_extreme_temperatures(cuda_device, temp):
    gen = torch.Generator().manual_seed(6)
    x = (2 * torch.randn(8, 3000, generator=gen)).cuda()
    expo = _expo(8, 3000, gen).cuda()
    for k, p, m in [(None, None, None), ([40] * 8, None, None), (None, [0.5] * 8, None),
                    ([40] * 8, [0.5] * 8, [0.1] * 8)]:
        _check(x, expo, [temp] * 8, k, p, m, least=0.7)
    assert api.device_status() == 0


def test_sample_rows_large_logits(cuda_device):
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(6, 5000, generator=gen).cuda()
    expo = _expo(6, 5000, gen).cuda()
    x[0] *= 1e37
    x[1] += 1e6                      # few different values
    x[2] *= 1e-37
    x[3, 17] = 3e38
    x[4, ::2] = -3e38
    x[5] = -3.4028234663852886e38
    _check(x, expo, None, [0, 100, 50, 10, 3000, 20], [0.9, 0.5, 1.0, 0.3, 0.9, 0.5], None, 0.6)
    assert api.device_status() == 0


def test_sample_rows_smallest_and_largest_exponentials(cuda_device):
    x = torch.zeros(3, 4000, device="cuda")
    expo = torch.ones(3, 4000, device="cuda")
    expo[0, 3333] = 2.0 ** -126
    expo[1] = 2.0 ** 32
    expo[1, 2222] = 2.0 ** 31
    expo[2] = 2.0 ** 32
    token, _ = api.sample_rows(x, expo)
    assert token.tolist() == [3333, 2222, 0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_rows_strides_and_odd_starts(cuda_device, dtype):
    # rows of a wider tensor, that start anywhere; what lies between them is NaN
    gen = torch.Generator().manual_seed(8)
    for V, lead, width in [(1000, 3, 1011), (8193, 1, 8195), (40000, 5, 40007)]:
        wide = torch.full((7, width), float("nan"), dtype=dtype)
        wide[:, lead:lead + V] = (2 * torch.randn(7, V, generator=gen)).to(dtype)
        x = wide.cuda()[:, lead:lead + V]
        expo = _expo(7, V, gen).cuda()
        a = _check(x, expo, None, [40] * 7, [0.9] * 7, None)
        b = _check(x.contiguous(), expo, None, [40] * 7, [0.9] * 7, None)
        assert a[0] == b[0]
    assert api.device_status() == 0


def test_sample_rows_many_rows(cuda_device):
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(5000, 300, generator=gen).cuda()
    expo = _expo(5000, 300, gen).cuda()
    _check(x, expo, None, [7] * 5000, [0.8] * 5000, None)
    assert api.sample_rows(x[:0], expo[:0])[0].shape == (0,)
    assert api.device_status() == 0


def test_sample_rows_is_deterministic_and_captured(cuda_device):
    gen = torch.Generator().manual_seed(10)
    sets = [((2 * torch.randn(40, 50000, generator=gen)).bfloat16().cuda(),
             _expo(40, 50000, gen).cuda(), _i32([(i * 37) % 4000 for i in range(40)]),
             _f32([0.5 + 0.0124 * i for i in range(40)])) for _ in range(3)]
    want = [api.sample_rows(x, e, None, k, p) for x, e, k, p in sets]
    for (x, e, k, p), w in zip(sets, want):
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(api.sample_rows(x, e, None, k, p), w))
    held = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = api.sample_rows(held[0], held[1], None, held[2], held[3])
    for i in (2, 0, 1):
        for h, t in zip(held, sets[i]):
            h.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))


def test_sample_rows_on_two_streams(cuda_device):
    gen = torch.Generator().manual_seed(11)
    sets = [(torch.randn(20, 60000, generator=gen).cuda(), _expo(20, 60000, gen).cuda())
            for _ in range(2)]
    p = _f32([0.9] * 20)
    want = [api.sample_rows(x, e, None, None, p) for x, e in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [None, None]
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = api.sample_rows(*sets[i], None, None, p)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_sample_rows_draws_follow_the_distribution(cuda_device):
    # 40000 draws from one row: shares within five standard deviations
    gen = torch.Generator().manual_seed(12)
    x = torch.randn(20, generator=gen)
    rows = x.expand(40000, 20).contiguous().cuda()
    token, _ = api.sample_rows(rows, _expo(40000, 20, gen).cuda(), None, _i32([12] * 40000),
                               _f32([0.9] * 40000))
    idx, w, _ = tree.kept(x.numpy(), 1.0, 12, float(np.float32(0.9)))
    p = np.zeros(20)
    p[idx] = w / w.sum()
    share = np.bincount(token.cpu().numpy(), minlength=20) / 40000
    assert np.abs(share - p).max() < 5 * np.sqrt(0.25 / 40000)


def test_sample_rows_refusals(cuda_device):
    x, e = torch.zeros(2, 8, device="cuda"), torch.ones(2, 8, device="cuda")
    for bad in [dict(logits=x[0]), dict(logits=x.t()), dict(logits=x.half()), dict(expo=e[:1]),
                dict(expo=e.double()), dict(logits=x.cpu()), dict(expo=e.t().contiguous().t()),
                dict(top_k=_f32([1, 1])), dict(top_k=_i32([1])), dict(top_p=_f32([1])),
                dict(min_p=_f32([1, 1, 1])), dict(temperature=_f32([1]))]:
        with pytest.raises((ValueError, TypeError)):
            api.sample_rows(**dict(dict(logits=x, expo=e), **bad))
    with pytest.raises(api.RFError):        # rows that overlap
        api.sample_rows(torch.zeros(20, device="cuda").as_strided((2, 8), (4, 1)), e)
