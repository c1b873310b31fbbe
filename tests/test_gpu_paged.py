"""The paged-cache serving operators on the GPU against the float64 oracle:
slots, append with head norm and rotation, attention over pages, verification
of drafted tokens, and a run of them together."""

import math

import numpy as np
import pytest
import torch

from online_softmax_attention_rf_gb300 import api
from oracle import paged
from tests.helpers import f64

pytestmark = pytest.mark.gpu

BF16_STEP = 2.0 ** -8    # half a step of bf16, relative
F32_STEP = 2.0 ** -24


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _pool(pages, page, Hkv, d, head_major, dtype, gen):
    shape = (pages, Hkv, page, d) if head_major else (pages, page, Hkv, d)
    c = torch.randn(shape, generator=gen).to(dtype).cuda()
    return c.permute(0, 2, 1, 3) if head_major else c


def _step(lengths, page, gen, spare=3):
    """(cu_q, kv_len, table rows, pages) of a batch of (new, cached) lengths over
    a shuffled pool."""
    need = [-(-kv // page) for _, kv in lengths]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=gen).tolist()
    cu, rows, at = [0], [], 0
    width = max(need + [1])
    for (n, _), m in zip(lengths, need):
        cu.append(cu[-1] + n)
        rows.append(perm[at:at + m] + [0] * (width - m))
        at += m
    return cu, [kv for _, kv in lengths], rows, pages


# ---------------------------------------------------------------- slots

@pytest.mark.parametrize("page,lengths,pad", [
    (16, [(1, 1)], 0),
    (16, [(1, 17), (0, 5), (3, 3), (40, 100)], 0),
    (8, [(5, 3), (2, 0), (1, 64)], 4),          # rows before the cache, padded rows
    (48, [(100, 130), (1, 48), (1, 49)], 1),
])
def test_paged_slots(cuda_device, page, lengths, pad):
    gen = torch.Generator().manual_seed(1)
    cu, kv, rows, pages = _step(lengths, page, gen)
    T = cu[-1] + pad
    pos, slots = api.paged_slots(_i32(cu), _i32(kv), _i32(rows), page, pages, T)
    p_ref, s_ref = paged.slots(cu, kv, rows, page, T)
    assert pos.cpu().tolist() == p_ref.tolist() and slots.cpu().tolist() == s_ref.tolist()
    assert api.device_status() == 0


def test_paged_slots_reports_a_table_entry_out_of_range(cuda_device):
    _, slots = api.paged_slots(_i32([0, 2]), _i32([17]), _i32([[3, 99]]), 16, 9, 2)
    assert slots.cpu().tolist() == [3 * 16 + 15, -1]
    with pytest.raises(api.RFError):
        api.device_status()


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,Hkv,d,rot,page,norm,interleaved,head_major", [
    (1, 4, 1, 128, 128, 16, True, False, False),
    (33, 7, 7, 64, 32, 8, True, True, True),
    (50, 8, 2, 128, 64, 48, False, False, False),
    (9, 3, 3, 80, 48, 16, True, False, False),      # lanes of a row left over
    (5, 2, 1, 256, 256, 1, True, True, False),
    (4, 6, 2, 16, 16, 64, True, False, True),
    (3, 4, 4, 32, 0, 16, True, False, False),       # no rotation
    (70, 0, 5, 64, 64, 32, True, False, False),     # no queries
])
def test_kv_append_paged(cuda_device, dtype, T, H, Hkv, d, rot, page, norm, interleaved,
                         head_major):
    gen = torch.Generator().manual_seed(T * 1000 + d)
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=gen).to(dtype).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    pages = -(-T // page) + 2
    kc = _pool(pages, page, Hkv, d, head_major, dtype, gen)
    vc = _pool(pages, page, Hkv, d, head_major, dtype, gen)
    slots = torch.randperm(pages * page, generator=gen)[:T]
    slots[T // 2] = -1 if T > 2 else slots[T // 2]   # one token without a place
    pos = torch.randint(0, 5000, (T,), generator=gen, dtype=torch.int32)
    ang = torch.rand(5000, max(rot // 2, 1), generator=gen, dtype=torch.float64) * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    w = [(1 + 0.2 * torch.randn(d, generator=gen)).to(dtype) if norm else None for _ in range(2)]
    eps = 1e-5
    k_old, v_old = f64(kc), f64(vc)
    q_out = torch.full((T, H, d), 7.0, dtype=dtype, device="cuda") if H else None
    got = api.kv_append_paged(q if H else None, k, v, kc, vc, slots.cuda(),
                              pos.cuda() if rot else None, cs.cuda() if rot else None,
                              w[0].cuda() if norm and H else None, w[1].cuda() if norm else None,
                              eps, interleaved, q_out)
    assert api.device_status() == 0
    cs_rows = f64(cs)[pos.numpy()] if rot else np.zeros((T, 0))

    def reference(x, weight):
        y = paged.head_norm(f64(x), None if weight is None else f64(weight), eps)
        # of each rotated pair both members' rounding errors reach either result
        size = np.abs(y)
        if rot:
            i = np.arange(rot // 2)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            both = size[..., a] + size[..., b]
            size[..., a] = size[..., b] = both
        return paged.rotate(y, cs_rows, interleaved), size

    # float32 steps: the mean of d squares (d / 2 on average, d at most), root,
    # quotient, two products of the norm, two products and a sum of the rotation
    steps = (d / 2 if norm else 0) + 8
    last = BF16_STEP if dtype == torch.bfloat16 else F32_STEP

    def check(x, ref, size):
        assert (np.abs(f64(x) - ref) <= steps * F32_STEP * size + 1.01 * last * np.abs(ref)
                + 1e-30).all()

    live = slots.numpy() >= 0
    if H:
        ref, size = reference(q, w[0])
        check(got[live], ref[live], size[live])
        assert (got.cpu()[~live] == 7.0).all()
    ref, size = reference(k, w[1])
    at = slots.numpy()[live]
    check(kc[at // page, at % page], ref[live], size[live])
    k_new, v_new = f64(kc), f64(vc)
    assert np.array_equal(v_new[at // page, at % page], f64(v)[live])
    k_old[at // page, at % page] = k_new[at // page, at % page]
    v_old[at // page, at % page] = v_new[at // page, at % page]
    assert np.array_equal(k_old, k_new) and np.array_equal(v_old, v_new)   # nothing else moved


@pytest.mark.parametrize("T,H,Hkv,d,dtype,skip", [
    (1500, 4, 2, 64, torch.bfloat16, 7),       # several tokens a block, some skipped
    (2000, 1, 1, 16, torch.float32, 0),
    (457, 40, 8, 256, torch.float32, 3),       # a token's heads take several stages
    (5000, 0, 1, 128, torch.bfloat16, 2),
])
def test_kv_append_paged_many_tokens(cuda_device, T, H, Hkv, d, dtype, skip):
    gen = torch.Generator().manual_seed(T)
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=gen).to(dtype).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    pages = -(-T // 16) + 1
    kc, vc = torch.zeros(2, pages, 16, Hkv, d, dtype=dtype, device="cuda")
    slots = torch.randperm(pages * 16, generator=gen)[:T].cuda()
    if skip:
        slots[::skip] = -1
    pos = torch.randint(0, 300, (T,), generator=gen, dtype=torch.int32).cuda()
    ang = torch.rand(300, d // 2, generator=gen).cuda() * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1)
    got = api.kv_append_paged(q if H else None, k, v, kc, vc, slots, pos, cs)
    assert api.device_status() == 0
    live = slots >= 0
    c, s = cs[pos.long()].double().chunk(2, 1)

    def turned(x):
        a, b = x.double().chunk(2, -1)
        return torch.cat([a * c[:, None] - b * s[:, None], b * c[:, None] + a * s[:, None]], -1)

    last = BF16_STEP if dtype == torch.bfloat16 else F32_STEP
    at = slots[live] // 16, slots[live] % 16
    for have, x in [(kc[at], k)] + ([(got[live], q)] if H else []):
        want = turned(x)[live]
        size = x[live].double().abs().unfold(-1, d // 2, d // 2).sum(-2).repeat(1, 1, 2)
        assert ((have.double() - want).abs() <= 3 * F32_STEP * size + 1.01 * last * want.abs()).all()
    assert torch.equal(vc[at], v[live])
    assert (kc != 0).any(-1).any(-1).sum() == live.sum()       # and nothing else was written


def test_kv_append_paged_in_place(cuda_device):
    gen = torch.Generator().manual_seed(5)
    q = torch.randn(20, 4, 128, generator=gen).bfloat16().cuda()
    k, v = torch.randn(2, 20, 2, 128, generator=gen).bfloat16().cuda()
    kc, vc = torch.zeros(2, 3, 8, 2, 128, dtype=torch.bfloat16, device="cuda")
    cs = torch.randn(64, 128, generator=gen).cuda()
    slots = torch.arange(20, device="cuda")
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    a = api.kv_append_paged(q, k, v, kc, vc, slots, pos, cs)
    b = api.kv_append_paged(q, k, v, kc, vc, slots, pos, cs, q_out=q)
    assert b.data_ptr() == q.data_ptr() and torch.equal(a, b)


def test_kv_append_paged_reports_places_out_of_range(cuda_device):
    k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    kc, vc = torch.zeros(2, 2, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    cs = torch.cat([torch.ones(10, 32), torch.zeros(10, 32)], 1).cuda()
    for slots, pos in [([0, 32, 1], [0, 0, 0]), ([0, 5, 1], [0, 10, 0]), ([0, 5, 1], [0, -1, 0])]:
        kc.zero_(), vc.zero_()
        api.kv_append_paged(None, k, k, kc, vc, torch.tensor(slots, device="cuda"), _i32(pos), cs)
        with pytest.raises(api.RFError):
            api.device_status()
        assert (kc.sum().item(), vc.sum().item()) == (128.0, 128.0)
        assert (kc[0, :2] == 1).all()


# ---------------------------------------------------------------- plan

def _spans(plan, cu, kv, H, Hkv, causal):
    """The plan's spans as lists of (seq, head, pair, first step, end step, steps)
    and its merge entries, decoded from device memory."""
    w = plan.buf.cpu().numpy().view(np.int32)
    ctas, n_merge, units = w[8], w[9], w[10]
    start = w[16:16 + 153 * 8].reshape(153, 8)
    merge = w[16 + 153 * 8:16 + 305 * 8].reshape(152, 8)[:n_merge]
    for s in start[:ctas]:
        assert (s[4], s[5], s[6]) == (cu[s[0]], cu[s[0] + 1], kv[s[0]])
    start = start[:, :4]
    tt = 128 // (H // Hkv)
    items = []
    for b in range(len(kv)):
        n = cu[b + 1] - cu[b]
        for h in range(Hkv):
            for p in range(-(-n // (2 * tt))):
                i1 = min(n, (p + 1) * 2 * tt)
                seen = max(0, kv[b] - n + i1) if causal else kv[b]
                items.append((b, h, p, -(-seen // 128), (i1 - p * 2 * tt) * (H // Hkv)))
    where = {it[:3]: i for i, it in enumerate(items)}
    where[(len(kv), 0, 0)] = len(items)
    spans = []
    for c in range(ctas):
        a, b = start[c], start[c + 1]
        i, j = where[tuple(a[:3])], where[tuple(b[:3])]
        assert (i, a[3]) <= (j, b[3])
        span, k0 = [], int(a[3])
        while i < j:
            span.append((i, k0, items[i][3]))
            i, k0 = i + 1, 0
        if k0 < b[3]:
            span.append((i, k0, int(b[3])))
        spans.append(span)
    assert ctas == 0 or (tuple(start[0]) == items[0][:3] + (0,)
                         and tuple(start[ctas]) == (len(kv), 0, 0, 0))
    return items, spans, merge, units


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths,H,Hkv", [
    ([(1, 1)], 1, 1), ([(1, 100000)], 8, 8), ([(1, 5000)] * 3, 32, 8), ([(2048, 32768)], 64, 8),
    ([(0, 5), (3, 1), (0, 0), (700, 900), (1, 4000), (0, 9)], 28, 4),
    ([(1 + i % 5, 40 * i + 6) for i in range(1100)], 8, 2), ([(130, 130)] * 7, 128, 1),
    ([(0, 3)], 4, 4), ([(9000, 9000), (1, 60000)], 4, 4),
    ([(1, 100), (1, 9000)] * 9, 64, 8), ([(1, 40000)], 4, 4), ([(130, 9000)], 8, 1),
])
def test_paged_plan_covers_every_step_once(cuda_device, lengths, H, Hkv, causal):
    cu = [0]
    for n, _ in lengths:
        cu.append(cu[-1] + n)
    kv = [m for _, m in lengths]
    plan = api.PagedPlan(_i32(cu), _i32(kv), cu[-1] + 3, H, Hkv, 16, 6250, causal)
    assert api.device_status() == 0
    items, spans, merge, units = _spans(plan, cu, kv, H, Hkv, causal)
    parts = {}
    for cta, span in enumerate(spans):
        for i, k0, k1 in span:
            parts.setdefault(i, []).append((cta, k0, k1))
    assert sorted(parts) == list(range(len(items)))
    cut = {}
    for i, pieces in parts.items():
        # contiguous steps from 0 to the item's end, one piece a CTA
        assert pieces[0][1] == 0 and pieces[-1][2] == items[i][3]
        assert all(x[2] == y[1] for x, y in zip(pieces, pieces[1:]))
        if len(pieces) > 1:
            cut[i] = pieces
    where = {it[:3]: i for i, it in enumerate(items)}
    assert sorted(where[tuple(m[:3])] for m in merge) == sorted(cut)
    unit0, G = 0, H // Hkv
    for m in merge:
        i = where[tuple(m[:3])]
        assert [c for c, _, _ in cut[i]] == list(range(m[3], m[3] + m[4]))
        assert m[5] == items[i][4] and m[6] == unit0
        first = min(m[5], 128 // G * G)        # rows of the first tile, in units of 32
        unit0 += -(-first // 32) + -(-(m[5] - first) // 32)
    assert unit0 == units
    pair = [it[4] > 128 // G * G for it in items]
    by_item = len(items) <= 152 and all(len(span) == 1 for span in spans)
    worth = sum(it[3] * (6 if p else 5) for it, p in zip(items, pair))
    if by_item:   # each CTA has a part of one item, none much larger than an even span
        assert all((k1 - k0) * (6 if pair[i] else 5) <= max(10, worth / 152 + 12) + 6
                   for span in spans for i, k0, k1 in span)
    else:         # the spans are even: a cut moves by up to a step, or by the fixed
        # part of the item that it falls into
        cost = [sum((22 if pair[i] else 12) * (k0 == 0) + (k1 - k0) * (6 if pair[i] else 5)
                    for i, k0, k1 in span) for span in spans]
        assert max(cost) <= sum(cost) / len(cost) + 28


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", [
    [(1, 2 ** 31 - 8)], [(200, 2 ** 31 - 8)], [(1, 2 ** 31 - 9), (0, 2 ** 31 - 8), (3, 5)],
    [(1, 2 ** 31 - 128 + i) for i in (-1, 0, 1, 120)] * 50,
])
def test_paged_plan_of_the_longest_caches(cuda_device, lengths, causal):
    H, Hkv, page = 8, 4, 8
    cu = [0]
    for n, _ in lengths:
        cu.append(cu[-1] + n)
    kv = [m for _, m in lengths]
    plan = api.PagedPlan(_i32(cu), _i32(kv), cu[-1], H, Hkv, page, (2 ** 31 - 8) // page, causal)
    assert api.device_status() == 0
    items, spans, _, _ = _spans(plan, cu, kv, H, Hkv, causal)
    at = [0] * len(items)
    for span in spans:
        for i, k0, k1 in span:
            assert at[i] == k0
            at[i] = k1
    assert at == [it[3] for it in items]
    steps = [sum(k1 - k0 for _, k0, k1 in span) for span in spans]
    # an item cut by itself has a whole number of parts, 37 at least here
    assert len(spans) == 152 and max(steps) <= 38 / 37 * sum(steps) / 152 + 2


# ---------------------------------------------------------------- attention

def _attention_case(lengths, H, Hkv, d, page, seed=0, causal=True, head_major=False, pad=0, amp=1.0,
                    fused=False, scale=None):
    gen = torch.Generator().manual_seed(seed)
    cu, kv, rows, pages = _step(lengths, page, gen)
    T = cu[-1] + pad
    kc = _pool(pages, page, Hkv, d, head_major, torch.bfloat16, gen)
    vc = _pool(pages, page, Hkv, d, head_major, torch.bfloat16, gen)
    heads = H + 2 * Hkv if fused else H
    q = (amp * torch.randn(T, heads, d, generator=gen)).bfloat16().cuda()[:, :H]
    return dict(q=q, kc=kc, vc=vc, cu=cu, kv=kv, rows=rows, T=T, H=H, Hkv=Hkv, d=d, page=page,
                causal=causal, scale=scale or 1.0 / math.sqrt(d))


def _attend(c, plan=None, **kw):
    table = _i32(c["rows"])
    if plan is None:
        plan = api.PagedPlan(_i32(c["cu"]), _i32(c["kv"]), c["T"], c["H"], c["Hkv"], c["page"],
                             table.shape[1], c["causal"])
    return api.attn_paged(c["q"], c["kc"], c["vc"], table, plan, c["scale"], **kw)


def _check_attention(c, o, lse, sequences=None):
    q, kc, vc = f64(c["q"]), f64(c["kc"]), f64(c["vc"])
    o, lse = f64(o), f64(lse)
    d = c["d"]
    for b in sequences if sequences is not None else range(len(c["kv"])):
        t0, t1, kv = c["cu"][b], c["cu"][b + 1], c["kv"][b]
        keys = paged.gather(kc, c["rows"][b], c["page"], kv)
        values = paged.gather(vc, c["rows"][b], c["page"], kv)
        o_ref, lse_ref, w, reach = paged.attention(q[t0:t1], keys, values, c["scale"], c["causal"])
        # a score is a float32 sum of d exact products, scaled to log2 units: at
        # most d + 3 half steps of its terms' absolute sum; the exponential's
        # error (2 steps) and the float32 sums over keys (their rounding errors
        # do not line up: 64 steps) on top
        score = (d + 3) * F32_STEP * reach
        tol_lse = score + 64 * F32_STEP * (1 + np.abs(np.where(np.isfinite(lse_ref), lse_ref, 0)))
        none = ~np.isfinite(lse_ref)
        assert np.array_equal(none, ~np.isfinite(lse[t0:t1])), b
        assert (np.abs(lse[t0:t1][~none] - lse_ref[~none]) <= tol_lse[~none]).all(), b
        assert (lse[t0:t1][none] == -np.inf).all() and (o[t0:t1][none] == 0).all()
        # P is rounded to bf16 (half a step of each term), then O is
        tol = (BF16_STEP + 2 * score[..., None] + 130 * F32_STEP) * w + BF16_STEP * 1.01 * np.abs(o_ref)
        bad = np.abs(o[t0:t1] - o_ref) > tol + 1e-30
        assert not bad.any(), (b, np.argwhere(bad)[:4].tolist(),
                               np.abs(o[t0:t1] - o_ref)[bad][:4], tol[bad][:4])


SMALL = [
    # lengths, H, Hkv, d, page
    ([(1, 1)], 1, 1, 64, 8),
    ([(1, 1)], 8, 1, 128, 16),
    ([(1, 127), (1, 128), (1, 129), (1, 300)], 8, 2, 128, 16),
    ([(2, 2), (0, 50), (5, 1000), (1, 77)], 4, 4, 64, 32),        # a sequence without new tokens
    ([(5, 3), (3, 0), (130, 100)], 4, 2, 128, 16),                # rows that see no key
    ([(100, 100)], 2, 2, 128, 8),
    ([(129, 140), (64, 64), (17, 300)], 2, 1, 64, 24),            # a page of 3 x 8
    ([(300, 1000), (1, 999), (257, 257)], 4, 2, 128, 128),
    ([(40, 41), (7, 2000)], 7, 1, 128, 256),                      # 7 heads a key head: 126 rows
    ([(33, 500), (1, 500)], 24, 2, 64, 48),                       # 12 heads a key head
    ([(3, 640)], 128, 1, 128, 64),                                # one token a tile
    ([(2, 200)], 130, 2, 64, 16),                                 # 65 heads a key head
    ([(1, 5000)], 8, 8, 64, 16),                                  # one sequence, split over CTAs
    ([(600, 2500)], 8, 2, 128, 40),
]


@pytest.mark.parametrize("lengths,H,Hkv,d,page", SMALL)
@pytest.mark.parametrize("causal", [True, False])
def test_attn_paged_matches_oracle(cuda_device, lengths, H, Hkv, d, page, causal):
    c = _attention_case(lengths, H, Hkv, d, page, seed=len(lengths) + page, causal=causal)
    o, lse = _attend(c)
    assert api.device_status() == 0
    _check_attention(c, o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("amp,scale", [(8.0, None), (1.0, 4.0), (0.01, None)])
def test_attn_paged_large_scores(cuda_device, d, amp, scale):
    # the running maximum moves by more than the lazy rescale allows
    c = _attention_case([(1, 900), (150, 700), (9, 260)], 4, 2, d, 16, seed=3, amp=amp, scale=scale)
    o, lse = _attend(c)
    assert api.device_status() == 0
    _check_attention(c, o, lse)


def test_attn_paged_rising_scores(cuda_device):
    # each key tile's scores exceed the last one's by far, in a split item too
    c = _attention_case([(1, 3000), (70, 1500)], 2, 1, 128, 64, seed=4)
    ramp = torch.arange(3000, device="cuda").float() / 40
    for b in range(2):
        for j in range(c["kv"][b]):
            c["kc"][c["rows"][b][j // 64], j % 64, 0] = (ramp[j] * c["q"][0, 0].float() / 30).bfloat16()
    o, lse = _attend(c)
    assert api.device_status() == 0
    _check_attention(c, o, lse)


@pytest.mark.parametrize("H,Hkv,nq", [(4, 4, 1), (4, 4, 32), (4, 4, 33), (15, 3, 6), (15, 3, 7),
                                      (32, 1, 1), (33, 1, 1), (64, 2, 1), (28, 4, 4), (28, 4, 5)])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_paged_few_rows_of_small_heads(cuda_device, H, Hkv, nq, causal):
    # on both sides of 32 packed rows; whole items, items in parts, tiles whose
    # last keys miss some of the quarters
    for kv in ([nq, 40, 129, 700], [1037, 1, 33, 97, 650], [20011]):
        lengths = [(min(nq, x), x) for x in kv]
        c = _attention_case(lengths, H, Hkv, 64, 16, seed=nq + len(kv), causal=causal)
        o, lse = _attend(c)
        _check_attention(c, o, lse)
    assert api.device_status() == 0


def test_attn_paged_small_heads_in_mixed_batches(cuda_device):
    # short single tokens, long ones and chunks in turn on one SM
    lengths = [(1, 90), (1, 5000), (200, 900), (1, 2000), (3, 2500), (1, 100), (1, 1500), (64, 1000)] * 3
    for H, Hkv in ((8, 8), (16, 4)):
        c = _attention_case(lengths, H, Hkv, 64, 16, seed=23)
        o, lse = _attend(c)
        _check_attention(c, o, lse)
        o2, lse2 = _attend(c)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert api.device_status() == 0


@pytest.mark.parametrize("head_major,fused", [(True, False), (False, True), (True, True)])
def test_attn_paged_layouts(cuda_device, head_major, fused):
    c = _attention_case([(65, 200), (1, 333)], 8, 2, 64, 16, seed=6, head_major=head_major,
                        fused=fused)
    o, lse = _attend(c)
    _check_attention(c, o, lse)


def test_attn_paged_other_orders_of_the_pool(cuda_device):
    # pages between the tokens ([page, pages, Hkv, d]), and keys and values of a
    # page side by side ([pages, 2, page, Hkv, d]); K and V in different orders
    c = _attention_case([(40, 300), (1, 150)], 8, 2, 128, 16, seed=17)
    o, lse = _attend(c)
    _check_attention(c, o, lse)
    inner = c["kc"].permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
    both = torch.stack([c["kc"], c["vc"]], 1)
    for kc, vc in [(inner, c["vc"]), (both[:, 0], both[:, 1]),
                   (c["kc"], c["vc"].transpose(1, 2).contiguous().transpose(1, 2))]:
        o2, lse2 = _attend(dict(c, kc=kc, vc=vc))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert api.device_status() == 0


def test_attn_paged_output_on_a_16_byte_boundary(cuda_device):
    # O takes 32-byte stores only where they are aligned
    for lengths in ([(70, 300), (1, 150)], [(1, 9000)]):
        c = _attention_case(lengths, 8, 2, 64, 16, seed=18)
        o, lse = _attend(c)
        room = torch.zeros(o.numel() + 16, dtype=o.dtype, device="cuda")
        odd = room[8:8 + o.numel()].view(o.shape)
        assert odd.data_ptr() % 32 == 16
        _attend(c, out=odd)
        assert torch.equal(o, odd) and (room[:8] == 0).all() and (room[-8:] == 0).all()


def test_attn_paged_rows_before_the_first_sequence(cuda_device):
    # cu_q may start above 0
    c = _attention_case([(3, 40), (1, 9)], 4, 2, 64, 8, seed=19, pad=5)
    shifted = dict(c, cu=[x + 5 for x in c["cu"]],
                   q=torch.cat([torch.full_like(c["q"][:5], float("nan")), c["q"][:4]]))
    o, lse = _attend(c)
    out = torch.full_like(o, 3.0)
    o2, lse2 = _attend(shifted, out=out)
    assert torch.equal(o2[5:], o[:4]) and torch.equal(lse2[5:], lse[:4]) and (o2[:5] == 3).all()
    _check_attention(c, o, lse)


def test_paged_calls_of_nothing(cuda_device):
    # no sequences, no tokens, sequences without new tokens, no drafts to judge
    pool = torch.full((2, 4, 16, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    for B, T in ((0, 0), (0, 3), (3, 0), (3, 2)):
        cu, kv = _i32([0] * (B + 1)), _i32([20] * B)
        table = _i32([[0, 1]] * B).view(B, 2)
        plan = api.PagedPlan(cu, kv, T, 4, 2, 16, 2)
        pos, slots = api.paged_slots(cu, kv, table, 16, 4, T)
        assert pos.tolist() == [0] * T and slots.tolist() == [-1] * T
        x = torch.full((T, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
        o = torch.full_like(x, 3.0)
        assert api.attn_paged(x, pool[0], pool[1], table, plan, out=o)[1].shape == (T, 4)
        assert (o == 3).all()
        out = torch.full_like(x, 7.0)
        api.kv_append_paged(x, x[:, :2], x[:, 2:], pool[0], pool[1], slots, q_out=out)
        assert (out == 7).all() and (pool == 5).all()
    none = torch.empty(0, 3, 10, device="cuda")
    tokens, accepted = api.draft_verify(none, None, _i32([]).view(0, 2),
                                        torch.empty(0, 2, device="cuda"),
                                        torch.empty(0, 10, device="cuda"))
    assert tokens.shape == (0, 3) and accepted.shape == (0,)
    assert api.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_attn_paged_a_whole_tile_of_heads(cuda_device, d):
    # 128 and 100 query heads of one key head: a tile holds one token
    for H in (128, 100):
        c = _attention_case([(1, 700), (3, 40), (2, 1)], H, 1, d, 16, seed=H)
        o, lse = _attend(c)
        _check_attention(c, o, lse)
    assert api.device_status() == 0


def test_append_and_verify_on_another_stream(cuda_device):
    # two streams at once, tensors made on the current one
    gen = torch.Generator().manual_seed(3)
    k = torch.randn(50, 2, 64, generator=gen).bfloat16().cuda()
    slots = torch.randperm(64, generator=gen)[:50].cuda()
    logits = torch.randn(4, 4, 5000, generator=gen).cuda()
    drafted = logits[:, :3].argmax(-1).to(torch.int32)
    u, expo = torch.full((4, 3), 0.5, device="cuda"), torch.ones(4, 5000, device="cuda")
    draft = logits[:, :3].contiguous()
    pools = [torch.zeros(2, 4, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    api.kv_append_paged(None, k, k, pools[2][0], pools[2][1], slots)
    want = api.draft_verify(logits, draft, drafted, u, expo)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                api.kv_append_paged(None, k, k, pools[i][0], pools[i][1], slots)
                got[i] = api.draft_verify(logits, draft, drafted, u, expo)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(pools[i], pools[2])
        assert all(torch.equal(x, y) for x, y in zip(got[i], want))
    assert api.device_status() == 0


def test_attn_paged_leaves_padded_rows(cuda_device):
    c = _attention_case([(3, 40), (1, 9)], 4, 2, 64, 8, seed=7, pad=5)
    o = torch.full((c["T"], 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c["T"], 4), 3.0, device="cuda")
    _attend(c, out=o, lse=lse)
    _check_attention(c, o, lse)
    assert (o[4:] == 3).all() and (lse[4:] == 3).all()
    o2, none = _attend(c, with_lse=False)
    assert none is None and torch.equal(o2[:4], o[:4])


@pytest.mark.parametrize("page", [8, 16, 64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_attn_paged_ignores_what_lies_past_the_cache(cuda_device, page, value):
    # rows past kv_len in the last page, other pages and the table's unused
    # entries hold anything
    c = _attention_case([(1, 70), (20, 333), (140, 200)], 4, 2, 128, page, seed=8)
    kc, vc = c["kc"].clone(), c["vc"].clone()
    live = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b, kv in enumerate(c["kv"]):
        for j in range(kv):
            live[c["rows"][b][j // page], j % page] = True
    kc[~live.cuda()] = value
    vc[~live.cuda()] = value
    o_ref, lse_ref = _attend(c)
    used = [-(-kv // page) for kv in c["kv"]]
    rows = [r[:u] + [1 << 30] * (len(r) - u) for r, u in zip(c["rows"], used)]
    o, lse = _attend(dict(c, kc=kc, vc=vc, rows=rows))
    assert api.device_status() == 0
    assert torch.equal(o, o_ref) and torch.equal(lse, lse_ref)


@pytest.mark.parametrize("lengths", [[(1, 33)], [(1, 640)], [(1, 9000)], [(40, 700)], [(200, 300)]])
def test_attn_paged_a_visible_nan_shows(cuda_device, lengths):
    # in a key that every row sees: that key head's rows are NaN, the others' not
    # touched, whether the item is whole or in parts
    c = _attention_case(lengths, 8, 2, 128, 16, seed=16)
    for at in (0, 31):
        bad = dict(c, kc=c["kc"].clone())
        bad["kc"][c["rows"][0][at // 16], at % 16, 1, 5] = float("nan")
        o, lse = _attend(bad)
        o_ref, lse_ref = _attend(c)
        assert torch.equal(o[:, :4], o_ref[:, :4]) and torch.equal(lse[:, :4], lse_ref[:, :4])
        assert o[:, 4:].isnan().all() and lse[:, 4:].isnan().all()


def test_attn_paged_many_sequences(cuda_device):
    # more items than CTAs, every length of a tile's neighbourhood
    lengths = [(1 + (i % 3), 1 + (i * 37) % 400 + 3) for i in range(300)]
    c = _attention_case(lengths, 4, 2, 64, 16, seed=9)
    o, lse = _attend(c)
    assert api.device_status() == 0
    _check_attention(c, o, lse, range(0, 300, 7))


def test_attn_paged_long_chunk_sampled(cuda_device):
    c = _attention_case([(700, 6000), (1, 6001)], 4, 1, 128, 64, seed=10)
    o, lse = _attend(c)
    assert api.device_status() == 0
    # every row of the second sequence; the first one against the second kernel
    # path of the framework (dense attention, same inputs, gathered)
    _check_attention(c, o, lse, [1])
    k = torch.stack([c["kc"][c["rows"][0][j // 64], j % 64] for j in range(6000)], 1)[None]
    v = torch.stack([c["vc"][c["rows"][0][j // 64], j % 64] for j in range(6000)], 1)[None]
    od, ld = api.attn_fwd(c["q"][:700].transpose(0, 1).contiguous()[None], k.contiguous(),
                          v.contiguous(), c["scale"], True)
    assert (lse[:700].T - ld[0]).abs().max().item() <= 2e-3
    assert (o[:700].transpose(0, 1).float() - od[0].float()).abs().max().item() <= 2e-2


def test_attn_paged_cache_beyond_32_bits(cuda_device):
    # element offsets pass 2^31: a pool of 2.4e9 elements per cache, pages at its end
    page, Hkv, d = 128, 8, 128
    pages = 18400
    kc = torch.empty(pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    gen = torch.Generator().manual_seed(11)
    rows = [[pages - 1, 0, pages - 2], [pages - 3, 16500, 1]]
    for r in sum(rows, []):
        kc[r] = torch.randn(page, Hkv, d, generator=gen).bfloat16().cuda()
        vc[r] = torch.randn(page, Hkv, d, generator=gen).bfloat16().cuda()
    cu, kv = [0, 2, 3], [300, 383]
    q = torch.randn(3, 16, d, generator=gen).bfloat16().cuda()
    plan = api.PagedPlan(_i32(cu), _i32(kv), 3, 16, Hkv, page, 3)
    o, lse = api.attn_paged(q, kc, vc, _i32(rows), plan)
    small = sum(rows, [])
    c = dict(q=q, kc=kc[small], vc=vc[small], cu=cu, kv=kv, rows=[[0, 1, 2], [3, 4, 5]], page=page,
             d=d, causal=True, scale=1.0 / math.sqrt(d))
    _check_attention(c, o, lse)
    # appended rows land there too
    k = torch.randn(2, Hkv, d, generator=gen).bfloat16().cuda()
    at = [(pages - 1) * page + 127, 16500 * page + 3]
    api.kv_append_paged(None, k, k, kc, vc, torch.tensor(at, device="cuda"))
    assert torch.equal(kc[pages - 1, 127], k[0]) and torch.equal(vc[16500, 3], k[1])
    assert api.device_status() == 0


def test_attn_paged_the_longest_cache(cuda_device):
    # one token over 2^31 - 11 keys, most of them in the same five pages. Scores
    # are 0 and values small whole numbers, so that each part's sums are exact; the
    # keys behind the last one would outweigh all others.
    page, d, kv = 8, 64, 2 ** 31 - 11
    width = (2 ** 31 - 8) // page
    gen = torch.Generator().manual_seed(12)
    kc = torch.randn(6, page, 1, d, generator=gen).bfloat16().cuda()
    vc = torch.randint(-1, 4, (6, page, 1, d), generator=gen).bfloat16().cuda()
    kc[..., 0] = 0
    kc[5, 5:, 0, 0], vc[5, 5:] = 100.0, 100.0
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    table = torch.randint(0, 5, (1, width), dtype=torch.int32, device="cuda")
    table[0, -1] = 5
    counts = torch.stack([(table == i).sum() for i in range(5)]).double()
    total = (counts[:, None, None] * vc[:5, :, 0].double()).sum((0, 1)) + vc[5, :5, 0].double().sum(0)
    plan = api.PagedPlan(_i32([0, 1]), _i32([kv]), 1, 1, 1, page, width)
    o, lse = api.attn_paged(q, kc, vc, table, plan, 1.0)
    assert api.device_status() == 0
    want = total / kv
    # parts are exact; joining 152 of them takes a few float32 steps each
    tol = (1.01 * BF16_STEP + 4 * 152 * F32_STEP) * want.abs()
    assert ((o[0, 0].double() - want).abs() <= tol).all()
    assert abs(lse.item() - math.log(kv)) <= 152 * 4 * F32_STEP * math.log(kv)


def test_attn_paged_bad_table_entry_is_reported(cuda_device):
    c = _attention_case([(2, 100), (1, 60)], 2, 1, 64, 16, seed=12)
    rows = [list(r) for r in c["rows"]]
    rows[0][3] = 10 ** 6
    _, _ = _attend(dict(c, rows=rows))
    with pytest.raises(api.RFError):
        api.device_status()
    rows[0][3] = -5
    o, lse = _attend(dict(c, rows=rows))
    with pytest.raises(api.RFError):
        api.device_status()
    _check_attention(c, o, lse, [1])     # the other sequence is unharmed


def test_attn_paged_another_plan_is_reported(cuda_device):
    c = _attention_case([(2, 100), (1, 60)], 2, 1, 64, 16, seed=13)
    plan = api.PagedPlan(_i32(c["cu"]), _i32(c["kv"]), 3, 4, 2, 16, 7)
    plan.H, plan.Hkv = 2, 1
    out = torch.full((3, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    _attend(c, plan=plan, out=out)
    with pytest.raises(api.RFError):
        api.device_status()
    assert (out == 5).all()


@pytest.mark.parametrize("cu,kv", [([0, 2, 1], [5, 5]), ([0, 2, 9], [5, 5]), ([-1, 1, 2], [5, 5]),
                                   ([0, 1, 2], [5, 200]), ([0, 1, 2], [-1, 5])])
def test_paged_plan_refuses_lengths_that_contradict_themselves(cuda_device, cu, kv):
    plan = api.PagedPlan(_i32(cu), _i32(kv), 8, 2, 1, 16, 7)
    with pytest.raises(api.RFError):
        api.device_status()
    q = torch.ones(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.ones(16, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    api.attn_paged(q, kc, kc, _i32([[0] * 7] * 2), plan, out=out)
    assert api.device_status() == 0 and (out == 5).all()


def test_attn_paged_captured_step_follows_its_lengths(cuda_device):
    # a captured decode step: slots, append, plan and attention, replayed for
    # growing lengths, and for lengths in another order of the batch
    H, Hkv, d, page, B, width = 8, 2, 128, 16, 4, 40
    gen = torch.Generator().manual_seed(14)
    pages = B * width + 1
    table = torch.randperm(pages, generator=gen)[:B * width].view(B, width)
    kc = _pool(pages, page, Hkv, d, False, torch.bfloat16, gen)
    vc = _pool(pages, page, Hkv, d, False, torch.bfloat16, gen)
    qkv = torch.zeros(B, H + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
    kv_len, cu = _i32([1] * B), _i32(range(B + 1))
    tab = table.int().cuda()
    cs = torch.cat([torch.ones(1000, 64), torch.zeros(1000, 64)], 1).cuda()
    plan = api.PagedPlan(cu, kv_len, B, H, Hkv, page, width)
    ws = api.attn_paged_workspace(d)

    def step():
        pos, slots = api.paged_slots(cu, kv_len, tab, page, pages, B)
        q = api.kv_append_paged(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kc, vc, slots, pos,
                                cs)
        plan.update(cu, kv_len)
        return (q,) + api.attn_paged(q, kc, vc, tab, plan, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, o, lse = step()
    for kv in ([5, 600, 33, 1], [6, 601, 34, 2], [639, 1, 128, 127], [640, 640, 640, 640]):
        kv_len.copy_(_i32(kv))
        qkv.copy_(torch.randn(qkv.shape, generator=gen).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        assert api.device_status() == 0
        c = dict(q=q, kc=kc, vc=vc, cu=list(range(B + 1)), kv=kv, rows=table.tolist(), page=page,
                 d=d, causal=True, scale=1.0 / math.sqrt(d))
        assert torch.equal(q, qkv[:, :H])
        _check_attention(c, o, lse)


def test_paged_steps_one_behind_the_other(cuda_device):
    # steps enqueued without the host waiting for any of them: the inputs are
    # rewritten by kernels directly ahead of each, the plan and the workspace are
    # the same ones, and each step's results are those of the step by itself
    H, Hkv, d, page, B, width = 8, 2, 64, 16, 6, 200
    gen = torch.Generator().manual_seed(31)
    pages = B * width
    table = torch.randperm(pages, generator=gen).view(B, width).int().cuda()
    filled = torch.randn(2, pages, page, Hkv, d, generator=gen).bfloat16().cuda()
    cs = torch.randn(width * page, d, generator=gen).cuda()
    steps = []
    for i in range(6):
        n = torch.randint(0, 4, (B,), generator=gen) if i % 2 else torch.ones(B, dtype=torch.long)
        kv = torch.randint(4, width * page, (B,), generator=gen)
        steps.append((_i32([0] + n.cumsum(0).tolist()), _i32(kv), torch.randn(
            4 * B, H + 2 * Hkv, d, generator=gen).bfloat16().cuda()))
    cu, kv_len, qkv = (torch.zeros_like(x) for x in steps[0])
    pool = torch.empty_like(filled)

    def step(cu, kv_len, qkv, plan, ws):
        pos, slots = api.paged_slots(cu, kv_len, table, page, pages, 4 * B)
        o = torch.zeros(4 * B, H, d, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(4 * B, H, device="cuda")
        q = torch.zeros_like(o)
        api.kv_append_paged(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], pool[0], pool[1], slots,
                            pos, cs, q_out=q)
        plan.update(cu, kv_len)
        api.attn_paged(q, pool[0], pool[1], table, plan, out=o, lse=lse, workspace=ws)
        return q, o, lse

    def plan_of(cu, kv_len):
        return api.PagedPlan(cu, kv_len, 4 * B, H, Hkv, page, width)

    want = []
    for s in steps:
        pool.copy_(filled)
        torch.cuda.synchronize()
        want.append(step(*s, plan_of(*s[:2]), api.attn_paged_workspace(d)))
        torch.cuda.synchronize()
    plan, ws = plan_of(*steps[0][:2]), api.attn_paged_workspace(d)
    got, order = [], [(i * i) % 6 for i in range(60)]
    torch.cuda.synchronize()
    for i in order:
        torch.add(filled, 0, out=pool)
        for x, y in zip((cu, kv_len, qkv), steps[i]):
            torch.add(y, 0, out=x)
        got.append(step(cu, kv_len, qkv, plan, ws))
    torch.cuda.synchronize()
    assert api.device_status() == 0
    for i, g in zip(order, got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i]))


def test_attn_paged_two_streams(cuda_device):
    # two calls in flight, a workspace each, on streams other than the tensors'
    cases = [_attention_case([(1, 4000), (3, 2500)], 8, 2, 128, 16, seed=20 + i) for i in range(2)]
    want = [_attend(c) for c in cases]
    plans = [api.PagedPlan(_i32(c["cu"]), _i32(c["kv"]), c["T"], 8, 2, 16, len(c["rows"][0]))
             for c in cases]
    spaces = [api.attn_paged_workspace(128) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = _attend(cases[i], plan=plans[i], workspace=spaces[i])
    torch.cuda.synchronize()
    assert api.device_status() == 0
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


def test_attn_paged_is_deterministic(cuda_device):
    c = _attention_case([(1, 9000), (40, 3000), (300, 1000)], 8, 2, 128, 32, seed=30)
    o, lse = _attend(c)
    for _ in range(3):
        o2, lse2 = _attend(c)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attn_paged_refusals(cuda_device):
    c = _attention_case([(2, 100)], 2, 1, 64, 16, seed=15)
    with pytest.raises(ValueError):
        _attend(dict(c, vc=c["vc"][:-1]))
    with pytest.raises(ValueError):
        _attend(dict(c, q=c["q"].transpose(0, 1).contiguous().transpose(0, 1)))
    with pytest.raises(ValueError):
        _attend(dict(c, q=c["q"].float()))
    with pytest.raises(api.RFError):
        _attend(dict(c, q=c["q"].float(), kc=c["kc"].float(), vc=c["vc"].float()))
    with pytest.raises(api.RFError):
        _attend(c, workspace=torch.empty(100, device="cuda"))
    with pytest.raises(ValueError):
        _attend(c, out=torch.empty(2, 2, 64, device="cuda"))
    with pytest.raises(ValueError):
        api.attn_paged(c["q"].cpu(), c["kc"], c["vc"], _i32(c["rows"]), api.PagedPlan(
            _i32(c["cu"]), _i32(c["kv"]), 2, 2, 1, 16, len(c["rows"][0])))


# ---------------------------------------------------------------- verification

# Relative error of a float32 probability: the exponent's argument carries three
# half steps of at most 64, the exponential and the sum a few more.
P_ERROR = (3 * 64 + 64) * F32_STEP


def _verify_case(B, S, V, dtype, seed, certain=False, ragged=False, greedy=False, agree=0.5,
                 sharp=2.5):
    gen = torch.Generator().manual_seed(seed)
    shared = sharp * torch.randn(B, S + 1, V, generator=gen)
    c = dict(target=(shared + agree * torch.randn(B, S + 1, V, generator=gen)).to(dtype))
    c["draft"] = None if certain else \
        (shared[:, :S] + agree * torch.randn(B, S, V, generator=gen)).to(dtype)
    temp = 0.5 + torch.rand(B, generator=gen)
    if greedy:
        temp[::2] = 0
    c["temperature"] = temp
    src = c["target"][:, :S] if certain else c["draft"]
    drawn = torch.argmax(torch.softmax(src.double(), -1) /
                         torch.empty(B, S, V, dtype=torch.float64).exponential_(generator=gen), -1)
    best = torch.argmax(c["target"][:, :S].float(), -1)
    c["tokens"] = torch.where(torch.rand(B, S, generator=gen) < 0.6, best, drawn).int()
    c["u"] = torch.rand(B, S, generator=gen)
    c["expo"] = torch.empty(B, V).exponential_(generator=gen).clamp_min_(1e-20)
    c["n_draft"] = torch.randint(0, S + 1, (B,), generator=gen, dtype=torch.int32) if ragged else None
    return c


def _verify(c, **kw):
    return api.draft_verify(*(None if c[n] is None else c[n].cuda() for n in
                              ("target", "draft", "tokens", "u", "expo", "n_draft",
                               "temperature")), **kw)


def _check_verify(c, out, n_acc):
    out, n_acc = out.cpu().numpy(), n_acc.cpu().numpy()
    B, S = c["tokens"].shape
    close = 0
    for b in range(B):
        n = S if c["n_draft"] is None else int(c["n_draft"][b])
        want, acc, margin = paged.verify(
            f64(c["target"][b]), None if c["draft"] is None else f64(c["draft"][b]),
            c["tokens"][b].tolist(), f64(c["u"][b]).tolist(), f64(c["expo"][b]), n,
            1.0 if c["temperature"] is None else float(c["temperature"][b]))
        if margin <= P_ERROR:      # within rounding of another answer: not decided in float32
            close += 1
            continue
        assert n_acc[b] == acc and out[b].tolist() == want.tolist(), (b, out[b], want, margin)
    assert close <= B // 8


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (3, 1, 2), (5, 4, 33), (2, 3, 1000), (9, 5, 2049),
                                   (16, 2, 8192), (2, 64, 257), (33, 7, 4099)])
@pytest.mark.parametrize("certain,ragged,greedy", [(False, False, False), (True, True, True),
                                                   (False, True, True)])
def test_draft_verify(cuda_device, dtype, B, S, V, certain, ragged, greedy):
    c = _verify_case(B, S, V, dtype, B * 100 + S, certain, ragged, greedy)
    out, n_acc = _verify(c)
    assert api.device_status() == 0
    _check_verify(c, out, n_acc)


@pytest.mark.parametrize("agree,sharp", [(0.0, 2.5), (0.05, 1.0), (3.0, 2.5), (0.5, 12.0)])
def test_draft_verify_agreement(cuda_device, agree, sharp):
    c = _verify_case(40, 6, 5000, torch.float32, 7, agree=agree, sharp=sharp)
    out, n_acc = _verify(c)
    assert api.device_status() == 0
    _check_verify(c, out, n_acc)
    if agree == 0.0:     # the draft is the target: u < 1 accepts everything
        assert (n_acc == 6).all()


def test_draft_verify_large_vocabulary(cuda_device):
    c = _verify_case(3, 2, 131072, torch.bfloat16, 8)
    out, n_acc = _verify(c)
    assert api.device_status() == 0
    _check_verify(c, out, n_acc)
    c["temperature"] = None
    out, n_acc = _verify(c)
    _check_verify(c, out, n_acc)


def test_draft_verify_masked_logits(cuda_device):
    # filtered vocabularies: most entries -inf, some at the type's lowest value,
    # a drafted token without any probability
    c = _verify_case(12, 3, 700, torch.float32, 9)
    gen = torch.Generator().manual_seed(1)
    for name in ("target", "draft"):
        cut = torch.rand(c[name].shape, generator=gen)
        c[name][cut < 0.8] = float("-inf")
        c[name][(cut >= 0.8) & (cut < 0.85)] = torch.finfo(torch.float32).min
        c[name][..., 5] = 1.0
    out, n_acc = _verify(c)
    assert api.device_status() == 0
    _check_verify(c, out, n_acc)
    assert ((out.cpu() >= -1) & (out.cpu() < 700)).all()


def test_draft_verify_nothing_to_draw_from(cuda_device):
    for bad in (float("-inf"), float("nan")):
        c = _verify_case(3, 2, 100, torch.float32, 10)
        c["target"][1] = bad
        out, n_acc = _verify(c)
        with pytest.raises(api.RFError):
            api.device_status()
        assert out[1].cpu().tolist() == [-1, -1, -1] and n_acc[1].item() == 0
        ok = {k: None if v is None else v[[0, 2]] for k, v in c.items()}
        _check_verify(ok, out[[0, 2]], n_acc[[0, 2]])


def test_draft_verify_token_out_of_range(cuda_device):
    for x in (-1, 100, 2 ** 31 - 1):
        c = _verify_case(2, 2, 100, torch.bfloat16, 11)
        c["tokens"][0, 0] = x
        out, n_acc = _verify(c)
        with pytest.raises(api.RFError):
            api.device_status()
        assert n_acc[0].item() == 0 and 0 <= out[0, 0].item() < 100


@pytest.mark.parametrize("temp", [1e-45, 1e-40, 4e-39, 5e-39, 1e-37, 1e37, 3.4e38])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_draft_verify_extreme_temperatures(cuda_device, dtype, temp):
    # subnormal ones among them: the largest logits share all the probability; at
    # the other end every entry but -inf weighs the same
    c = _verify_case(6, 3, 3000, dtype, 23)
    c["temperature"] = torch.full((6,), temp)
    c["target"][::2, :, [40, 2999]] = 20.0       # two largest logits
    c["target"][:, :, 7] = float("-inf")
    c["draft"][:, :, 8] = float("-inf")
    out, n_acc = _verify(c)
    assert api.device_status() == 0
    _check_verify(c, out, n_acc)


def test_draft_verify_smallest_and_largest_exponentials(cuda_device):
    c = _verify_case(8, 2, 2000, torch.float32, 24, sharp=1.0)
    c["expo"][0::4] = 2.0 ** 32
    c["expo"][0::4, 100] = 2.0 ** 31.5
    c["expo"][1::4, [50, 60]] = torch.tensor([2.0 ** -125, 2.0 ** -126])
    c["target"][1::4, :, [50, 60]] = 0.0                 # equal weights, the second one wins
    c["draft"][1::4, :, [50, 60]] = -4.0
    c["expo"][2::4] = 2.0 ** -126
    out, n_acc = _verify(c)
    assert api.device_status() == 0
    _check_verify(c, out, n_acc)
    refused = [b for b in (1, 5) if n_acc[b] < 2]
    assert all(out[b, n_acc[b]].item() == 60 for b in refused)


def test_draft_verify_ties_go_to_the_lowest_index(cuda_device):
    V = 10000
    target = torch.zeros(2, 2, V)
    target[1, 0, [77, 4000, 9999]] = 3.0
    c = dict(target=target, draft=None, tokens=torch.tensor([[0], [4000]], dtype=torch.int32),
             u=torch.tensor([[0.999], [0.0]]), expo=torch.ones(2, V), n_draft=None,
             temperature=torch.tensor([1.0, 0.0]))
    out, n_acc = _verify(c)
    # refused: all weights but the draft's own are equal; greedy: 77, not the drafted 4000
    assert out.cpu().tolist() == [[1, -1], [77, -1]] and n_acc.cpu().tolist() == [0, 0]


def test_draft_verify_captured(cuda_device):
    c = {k: None if v is None else v.cuda() for k, v in
         _verify_case(4, 3, 3001, torch.bfloat16, 12).items()}
    ws = api.draft_verify_workspace(4, 3)
    names = ("target", "draft", "tokens", "u", "expo", "n_draft", "temperature")
    call = lambda: api.draft_verify(*[c[n] for n in names], workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, n_acc = call()
    for seed in (13, 14):
        new = _verify_case(4, 3, 3001, torch.bfloat16, seed)
        for n in names:
            if c[n] is not None:
                c[n].copy_(new[n])
        g.replay()
        torch.cuda.synchronize()
        _check_verify(new, out, n_acc)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 101), (torch.bfloat16, 9000)])
@pytest.mark.parametrize("bad", ["-inf", "nan", "inf", "all nan"])
def test_draft_verify_greedy_row_without_probabilities(cuda_device, dtype, V, bad):
    # greedy sequences whose judging row (the first, a middle one, the extra one)
    # has no finite maximum or a NaN: the row refuses its draft and draws -1
    c = _verify_case(4, 3, V, dtype, 21)
    c["temperature"] = torch.tensor([0.0, 0.0, 0.0, 1.0])
    c["target"][:3, torch.arange(3), torch.arange(3)] = 30.0
    c["tokens"][:3] = torch.arange(3, dtype=torch.int32)    # what the rows choose
    good = {k: None if v is None else v.clone() for k, v in c.items()}
    for b, row in enumerate((0, 2, 3)):
        if bad in ("-inf", "all nan"):
            c["target"][b, row] = float(bad.split()[-1])
        else:
            c["target"][b, row, V - 7] = float(bad)
    out, n_acc = _verify(c)
    with pytest.raises(api.RFError):
        api.device_status()
    want, want_acc = _verify(good)
    assert api.device_status() == 0
    _check_verify(good, want, want_acc)
    assert want_acc[:3].cpu().tolist() == [3, 3, 3]
    # the accepted drafts ahead of the bad row, then -1
    assert n_acc[:3].cpu().tolist() == [0, 2, 3]
    assert out[:3].cpu().tolist() == [[-1] * 4, [0, 1, -1, -1], [0, 1, 2, -1]]
    assert torch.equal(out[3], want[3]) and n_acc[3] == want_acc[3]
    # a bad row behind the first refusal is not looked at
    c["tokens"][:, 0] = V - 1
    c["target"][:, 0] = good["target"][:, 0]
    out, _ = _verify(c)
    assert api.device_status() == 0 and (out[:, 0] >= 0).all()


@pytest.mark.parametrize("dtype,V", [(torch.float32, 101), (torch.bfloat16, 9000)])
@pytest.mark.parametrize("bad", ["-inf", "nan", "inf", "all nan"])
def test_draft_verify_draft_row_without_probabilities(cuda_device, dtype, V, bad):
    # a draft row that is no distribution refuses its draft and draws -1, as a
    # target row does; one behind the first refusal is not looked at
    c = _verify_case(3, 3, V, dtype, 22)
    c["target"][:, torch.arange(3), torch.arange(3)] = 30.0   # accepted with certainty
    c["tokens"][:] = torch.arange(3, dtype=torch.int32)
    good = {k: None if v is None else v.clone() for k, v in c.items()}
    for b, row in enumerate((0, 2)):
        if bad in ("-inf", "all nan"):
            c["draft"][b, row] = float(bad.split()[-1])
        else:
            c["draft"][b, row, V - 7] = float(bad)
    out, n_acc = _verify(c)
    with pytest.raises(api.RFError):
        api.device_status()
    want, want_acc = _verify(good)
    assert api.device_status() == 0
    _check_verify(good, want, want_acc)
    assert n_acc.cpu().tolist() == [0, 2, want_acc[2].item()]
    assert out[:2].cpu().tolist() == [[-1] * 4, [0, 1, -1, -1]] and torch.equal(out[2], want[2])
    c["tokens"][1, 0] = V - 1
    c["draft"][0] = good["draft"][0]
    out, n_acc = _verify(c)
    assert api.device_status() == 0 and n_acc[1] == 0 and out[1, 0] >= 0


def _rewritten_in_place(c, sets, names):
    """Calls one behind the other on one stream, with one workspace: a kernel
    writes the inputs `names` of the next set into the same tensors directly
    ahead of each call, and the host waits for nothing in between. Yields the
    calls' results beside those of calls by themselves."""
    c = {k: None if v is None else v.cuda() for k, v in c.items()}
    sets = [{n: s[n].cuda() for n in names} for s in sets]
    B, S = c["tokens"].shape

    def call(kw, ws):
        return api.draft_verify(*(kw[n] for n in ("target", "draft", "tokens", "u", "expo",
                                                  "n_draft", "temperature")), workspace=ws)

    want = []
    for s in sets:
        want.append(call(dict(c, **s), api.draft_verify_workspace(B, S)))
        torch.cuda.synchronize()
    assert len({str([x.tolist() for x in w]) for w in want}) > 1
    ws = api.draft_verify_workspace(B, S)
    for n in names:
        c[n] = torch.empty_like(sets[0][n])
    torch.cuda.synchronize()
    got, order = [], [i % len(sets) for i in range(200)]
    for i in order:
        for n in names:
            torch.add(sets[i][n], 0, out=c[n])
        got.append(call(c, ws))
    torch.cuda.synchronize()
    assert api.device_status() == 0
    return [(got[k], want[i]) for k, i in enumerate(order)]


@pytest.mark.parametrize("B,S,V", [(1, 4, 600), (4, 3, 20000), (40, 6, 1000)])
def test_draft_verify_statistics_of_this_call(cuda_device, B, S, V):
    # the draw starts under the statistics of its own call: it must not see the
    # last call's, which lie at the same place in the workspace
    cases = [_verify_case(B, S, V, torch.float32, 50 + i) for i in range(5)]
    for got, want in _rewritten_in_place(cases[0], cases, ("target", "draft")):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("B,S,V,certain", [(1, 4, 600, False), (4, 3, 20000, False),
                                           (40, 6, 1000, True), (3, 64, 257, False)])
def test_draft_verify_inputs_of_this_call(cuda_device, B, S, V, certain):
    # the draw reads drafts, their logits, random numbers and temperatures before
    # the statistics are done: they must be this call's too
    cases = [_verify_case(B, S, V, torch.float32, 60 + i, certain, ragged=True, greedy=True,
                          agree=0.3) for i in range(7)]
    for c in cases[::2]:
        c["temperature"] = c["temperature"].flip(0)      # other sequences are greedy
    names = ("target", "tokens", "u", "expo", "n_draft", "temperature") + \
        (() if certain else ("draft",))
    for got, want in _rewritten_in_place(cases[0], cases, names):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------- together

def test_speculative_decoding_over_a_paged_cache(cuda_device):
    """Three verification steps of a small random model's layer: drafted tokens
    are embedded, their keys and values appended, attended over the pages, and
    verified; refused ones are overwritten by the next step. The oracle
    recomputes each step from the whole history without a cache."""
    H, Hkv, d, page, V, S, B = 4, 2, 64, 16, 50, 3, 3
    gen = torch.Generator().manual_seed(40)
    emb = torch.randn(V, (H + 2 * Hkv) * d, generator=gen).bfloat16().cuda()
    head = (torch.randn(H * d, V, generator=gen) / 8).cuda()
    wq, wk = (1 + 0.1 * torch.randn(2, d, generator=gen)).bfloat16().cuda()
    half = d // 2
    ang = torch.arange(200).double()[:, None] * 100.0 ** (-torch.arange(half).double() / half)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    width = 5
    table = torch.randperm(B * width, generator=gen).view(B, width).int().cuda()
    kc, vc = torch.zeros(2, B * width, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    history = [torch.randint(0, V, (n,), generator=gen).tolist() for n in (4, 17, 30)]

    def forward(new, cached):
        """New tokens (lists) of each sequence after `cached` ones -> hidden rows."""
        cu = np.concatenate([[0], np.cumsum([len(x) for x in new])])
        kv = [m + len(x) for m, x in zip(cached, new)]
        T = int(cu[-1])
        tok = torch.tensor(sum(new, []), device="cuda")
        qkv = emb[tok].view(T, H + 2 * Hkv, d)
        pos, slots = api.paged_slots(_i32(cu), _i32(kv), table, page, B * width, T)
        q = api.kv_append_paged(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], kc, vc, slots, pos,
                                cs, wq, wk)
        plan = api.PagedPlan(_i32(cu), _i32(kv), T, H, Hkv, page, width)
        o, _ = api.attn_paged(q, kc, vc, table, plan, with_lse=False)
        return cu, o

    def oracle_rows(tokens):
        x = f64(emb)[tokens].reshape(len(tokens), H + 2 * Hkv, d)
        rows = f64(cs)[:len(tokens)]
        q = paged.rotate(paged.head_norm(x[:, :H], f64(wq), 1e-6), rows, False)
        k = paged.rotate(paged.head_norm(x[:, H:H + Hkv], f64(wk), 1e-6), rows, False)
        return paged.attention(q, k, x[:, H + Hkv:], 1.0 / math.sqrt(d), True)[0]

    forward([h[:-1] for h in history], [0] * B)       # the prompts, but for the last token
    for step in range(3):
        drafts = [torch.randint(0, V, (S,), generator=gen).tolist() for _ in range(B)]
        new = [h[-1:] + x for h, x in zip(history, drafts)]
        cu, o = forward(new, [len(h) - 1 for h in history])
        for b in range(B):
            ref = oracle_rows(history[b] + drafts[b])[-(S + 1):]
            got = f64(o[cu[b]:cu[b + 1]])
            # q and k rounded to bf16 move a score by at most 2^-7 of |q||k| scale,
            # itself at most sqrt(d) * (largest weights)^2 ~ 14: 0.11, hence
            # weights by 2 * 0.11; P and O are rounded once more
            assert np.abs(got - ref).max() <= (0.22 + 2 ** -7) * np.abs(f64(emb)).max()
            assert np.abs(got - ref).mean() <= 0.01
        logits = (o.view(-1, H * d).float() @ head).view(B, S + 1, V)
        u = torch.rand(B, S, generator=gen)
        expo = torch.empty(B, V).exponential_(generator=gen)
        c = dict(target=logits.cpu(), draft=None, tokens=torch.tensor(drafts).int(), u=u * 0.05,
                 expo=expo, n_draft=None, temperature=None)
        out, n_acc = _verify(c)
        _check_verify(c, out, n_acc)
        for b in range(B):
            a = n_acc[b].item()
            history[b] = history[b] + out[b, :a + 1].tolist()
    assert api.device_status() == 0
