"""Trees of drafted tokens on the GPU against the float64 oracle: masks and
positions, attention over a paged cache, the walk along drawn tokens, and steps of
decoding with trees as they would be used."""

import math

import numpy as np
import pytest
import torch

from online_softmax_attention_rf_gb300 import api
from oracle import paged, tree
from tests.helpers import f64

pytestmark = pytest.mark.gpu

BF16_STEP = 2.0 ** -8    # half a step of bf16, relative
F32_STEP = 2.0 ** -24


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _offsets(sizes):
    return [0] + np.cumsum(sizes).tolist()


def _parents(n, rng, reach=6):
    return [-1 if i == 0 else int(rng.integers(max(0, i - reach), i)) for i in range(n)]


# ---------------------------------------------------------------- masks

@pytest.mark.parametrize("sizes,words,lead,pad", [
    ([1], 1, 0, 0), ([64], 1, 0, 0), ([65, 1, 0, 128], 2, 0, 0), ([7, 0, 30], 4, 3, 5),
    ([1024], 16, 0, 0), ([1000, 3], 16, 0, 2), ([200] * 40, 4, 0, 1),
])
def test_tree_mask(cuda_device, sizes, words, lead, pad):
    rng = np.random.default_rng(len(sizes) + words)
    parents = [_parents(n, rng, reach=3) for n in sizes]
    cu = [c + lead for c in _offsets(sizes)]
    kv = [n + int(rng.integers(0, 100)) for n in sizes]
    packed = [-1] * lead + sum(parents, []) + [5] * pad
    mask, pos = api.tree_mask(_i32(packed), _i32(cu), _i32(kv), words)
    assert api.device_status() == 0
    m_ref, p_ref = np.zeros((len(packed), words), np.int64), np.zeros(len(packed), np.int64)
    for b, p in enumerate(parents):
        if p:
            m_ref[cu[b]:cu[b + 1]] = tree.words(tree.mask(p), words)
            p_ref[cu[b]:cu[b + 1]] = kv[b] - len(p) + tree.depths(p)
    assert np.array_equal(mask.cpu().numpy(), m_ref)
    assert pos.cpu().tolist() == p_ref.tolist()


def test_tree_mask_reports_what_is_no_tree(cuda_device):
    # a parent behind its child, itself, or below -1: the node becomes a root
    mask, pos = api.tree_mask(_i32([-1, 2, 0, 3, -2]), _i32([0, 5]), _i32([9]))
    assert mask[:, 0].tolist() == [1, 2, 5, 8, 16] and pos.tolist() == [4, 4, 5, 4, 4]
    with pytest.raises(api.RFError):
        api.device_status()
    # more nodes than the words have bits for; the other sequence's are right
    mask, pos = api.tree_mask(_i32([-1] + [0] * 64 + [-1, 0]), _i32([0, 65, 67]), _i32([70, 2]))
    assert not mask[:65].any() and not pos[:65].any()
    assert mask[65:, 0].tolist() == [1, 3] and pos[65:].tolist() == [0, 1]
    with pytest.raises(api.RFError):
        api.device_status()
    # offsets that contradict themselves: no access outside the rows
    for cu in ([0, 4, 2], [-1, 1, 2], [0, 1, 9]):
        api.tree_mask(_i32([-1, 0, 0]), _i32(cu), _i32([5, 5]))
        api.tree_accept(*[_i32([-1, 0, 0])] * 3, _i32(cu), _i32([5, 5]))
        with pytest.raises(api.RFError):
            api.device_status()


# ---------------------------------------------------------------- attention

def _case(lengths, H, Hkv, d, page, words=1, seed=0, head_major=False, pad=0, amp=1.0, fused=False):
    """Sequences of (nodes, cached tokens with them) over a shuffled pool."""
    gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    need = [-(-kv // page) for _, kv in lengths]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=gen).tolist()
    rows, at, width = [], 0, max(need + [1])
    for m in need:
        rows.append(perm[at:at + m] + [0] * (width - m))
        at += m
    cu = _offsets([n for n, _ in lengths])
    T = cu[-1] + pad

    def pool():
        shape = (pages, Hkv, page, d) if head_major else (pages, page, Hkv, d)
        c = torch.randn(shape, generator=gen).bfloat16().cuda()
        return c.permute(0, 2, 1, 3) if head_major else c

    q = (amp * torch.randn(T, H + 2 * Hkv if fused else H, d, generator=gen)).bfloat16().cuda()
    parents = [_parents(n, rng) for n, _ in lengths]
    return dict(q=q[:, :H], kc=pool(), vc=pool(), cu=cu, kv=[m for _, m in lengths], rows=rows, T=T,
                H=H, Hkv=Hkv, d=d, page=page, words=words, parents=parents,
                packed=_i32(sum(parents, []) + [-1] * pad), scale=1.0 / math.sqrt(d))


def _plan(c, causal=False):
    return api.PagedPlan(_i32(c["cu"]), _i32(c["kv"]), c["T"], c["H"], c["Hkv"], c["page"],
                         len(c["rows"][0]), causal)


def _attend(c, plan=None, mask=None, **kw):
    if mask is None:
        mask, _ = api.tree_mask(c["packed"], _i32(c["cu"]), _i32(c["kv"]), c["words"])
    return api.attn_paged(c["q"], c["kc"], c["vc"], _i32(c["rows"]), plan or _plan(c), c["scale"],
                          tree_mask=mask, **kw)


def _seen(c, b, bits=None):
    n, kv = c["cu"][b + 1] - c["cu"][b], c["kv"][b]
    own = tree.mask(c["parents"][b]) if bits is None else bits
    seen = np.ones((n, kv), bool)
    for i in range(n):
        for j in range(max(0, kv - n), kv):
            seen[i, j] = own[i, j - (kv - n)]
    return seen


def _check(c, o, lse, sequences=None, seen=None):
    q, kc, vc = f64(c["q"]), f64(c["kc"]), f64(c["vc"])
    o, lse, d = f64(o), f64(lse), c["d"]
    for b in sequences if sequences is not None else range(len(c["kv"])):
        t0, t1, kv = c["cu"][b], c["cu"][b + 1], c["kv"][b]
        keys = paged.gather(kc, c["rows"][b], c["page"], kv)
        values = paged.gather(vc, c["rows"][b], c["page"], kv)
        o_ref, lse_ref, w, reach = tree.attention(q[t0:t1], keys, values, c["scale"],
                                                  _seen(c, b) if seen is None else seen[b])
        # a score is a float32 sum of d exact products, scaled to log2 units: at
        # most d + 3 half steps of its terms' absolute sum; the exponential's error
        # (2 steps) and the float32 sums over keys (their rounding errors do not
        # line up: 64 steps) on top
        score = (d + 3) * F32_STEP * reach
        fin = np.isfinite(lse_ref)
        assert np.array_equal(fin, np.isfinite(lse[t0:t1])), b
        tol_lse = score + 64 * F32_STEP * (1 + np.abs(np.where(fin, lse_ref, 0)))
        assert (np.abs(lse[t0:t1][fin] - lse_ref[fin]) <= tol_lse[fin]).all(), b
        assert (lse[t0:t1][~fin] == -np.inf).all() and (o[t0:t1][~fin] == 0).all()
        # P is rounded to bf16 (half a step of each term), then O is
        tol = (BF16_STEP + 2 * score[..., None] + 130 * F32_STEP) * w + \
            BF16_STEP * 1.01 * np.abs(o_ref)
        assert (np.abs(o[t0:t1] - o_ref) <= tol + 1e-30).all(), b


SMALL = [
    # lengths, H, Hkv, d, page, words
    ([(1, 1)], 1, 1, 64, 8, 1),
    ([(5, 5)], 4, 1, 128, 16, 1),                                # nothing before the tree
    ([(25, 1030)], 32, 8, 128, 16, 1),
    ([(64, 127), (64, 128), (64, 129), (63, 300), (1, 77)], 8, 2, 128, 16, 1),
    ([(2, 2), (0, 50), (50, 1000), (1, 77)], 4, 4, 64, 32, 1),   # a sequence without nodes
    ([(200, 333), (130, 131), (129, 140), (65, 500)], 7, 1, 64, 24, 4),
    ([(256, 700)], 2, 2, 128, 128, 4),
    ([(100, 1000), (3, 2000), (40, 41)], 28, 4, 128, 256, 2),
    ([(9, 640)], 128, 1, 128, 64, 1),                            # one token a tile
    ([(12, 200)], 130, 2, 64, 16, 1),
    ([(64, 5000)], 8, 8, 64, 16, 1),                             # split over CTAs
    ([(1000, 1200)], 4, 2, 64, 16, 16),
]


@pytest.mark.parametrize("lengths,H,Hkv,d,page,words", SMALL)
def test_tree_attention_matches_oracle(cuda_device, lengths, H, Hkv, d, page, words):
    c = _case(lengths, H, Hkv, d, page, words, seed=len(lengths) + page)
    o, lse = _attend(c)
    assert api.device_status() == 0
    _check(c, o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("over", range(0, 130, 13))
def test_tree_attention_context_ends_anywhere_in_a_tile(cuda_device, d, over):
    # the mask's words lie at every offset to the key tiles
    c = _case([(61, 128 + over + 61), (130, over + 130)], 4, 2, d, 16, 3, seed=over)
    o, lse = _attend(c)
    _check(c, o, lse)
    assert api.device_status() == 0


@pytest.mark.parametrize("head_major,fused", [(True, False), (False, True)])
def test_tree_attention_layouts(cuda_device, head_major, fused):
    c = _case([(20, 333), (64, 70)], 8, 2, 128, 16, 1, seed=9, head_major=head_major, fused=fused)
    o, lse = _attend(c)
    _check(c, o, lse)


def test_a_chain_is_causal_attention(cuda_device):
    # the same steps and tiles as the causal call's where both have as many keys:
    # equal up to the order in which spans are cut; here a sequence is whole
    c = _case([(40, 1000), (3, 77), (1, 500)], 8, 2, 128, 16, 1, seed=2)
    c["parents"] = [list(range(-1, n - 1)) for n in (40, 3, 1)]
    c["packed"] = _i32(sum(c["parents"], []))
    o, lse = _attend(c)
    _check(c, o, lse)
    table = _i32(c["rows"])
    o2, lse2 = api.attn_paged(c["q"], c["kc"], c["vc"], table, _plan(c, True), c["scale"])
    # both within their tolerance of one value: P's and O's rounding, twice
    assert (o.float() - o2.float()).abs().max() <= 4 * BF16_STEP * c["vc"].float().abs().max()
    assert torch.allclose(lse, lse2, atol=1e-4, rtol=0)


def test_tree_attention_other_masks(cuda_device):
    # any bits do: rows that see no node, later nodes, nothing at all (no context);
    # bits of nodes that there are not change nothing
    rng = np.random.default_rng(3)
    lengths = [(40, 40), (50, 170), (10, 7), (64, 100)]
    c = _case(lengths, 4, 2, 64, 16, 2, seed=3)
    bits = [rng.random((n, 128)) < 0.2 for n, _ in lengths]
    bits[0][5] = bits[1][7] = False
    words = np.concatenate([tree.words(b, 2) for b in bits])
    o, lse = _attend(c, mask=torch.from_numpy(words).cuda())
    assert api.device_status() == 0
    # (of 10 nodes of a cache of 7 tokens the first three have no key)
    seen = [_seen(c, b, bits[b]) for b in range(4)]
    assert not seen[0][5].any()
    _check(c, o, lse, seen=seen)


def test_tree_attention_nodes_behind_the_words_are_not_seen(cuda_device):
    c = _case([(70, 200)], 4, 2, 128, 16, 1, seed=4)
    bits = np.tri(70, 128, dtype=bool)
    bits[:, 64:] = False
    o, lse = _attend(c, mask=torch.from_numpy(tree.words(bits[:, :64], 1)).cuda())
    assert api.device_status() == 0
    _check(c, o, lse, seen=[_seen(c, 0, bits)])


def test_tree_attention_leaves_padded_rows(cuda_device):
    c = _case([(3, 40), (20, 29)], 4, 2, 64, 8, seed=7, pad=5)
    o = torch.full((c["T"], 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c["T"], 4), 3.0, device="cuda")
    _attend(c, out=o, lse=lse)
    _check(c, o, lse)
    assert (o[23:] == 3).all() and (lse[23:] == 3).all()
    o2, none = _attend(c, with_lse=False)
    assert none is None and torch.equal(o2[:23], o[:23])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_tree_attention_ignores_what_lies_past_the_cache(cuda_device, value):
    c = _case([(20, 70), (60, 333), (64, 200)], 4, 2, 128, 16, seed=8)
    kc, vc = c["kc"].clone(), c["vc"].clone()
    live = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b, kv in enumerate(c["kv"]):
        for j in range(kv):
            live[c["rows"][b][j // 16], j % 16] = True
    kc[~live.cuda()] = value
    vc[~live.cuda()] = value
    o_ref, lse_ref = _attend(c)
    o, lse = _attend(dict(c, kc=kc, vc=vc))
    assert api.device_status() == 0
    assert torch.equal(o, o_ref) and torch.equal(lse, lse_ref)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_tree_attention_an_unseen_node_s_key_changes_nothing(cuda_device, value):
    # a node's key that its siblings do not see may hold anything (its value row has
    # to be finite): the rows that do not see it are bit for bit the same
    c = _case([(30, 100)], 4, 2, 64, 16, seed=11)
    o_ref, lse_ref = _attend(c)
    node = 12
    at = 70 + node
    kc = c["kc"].clone()
    kc[c["rows"][0][at // 16], at % 16] = value
    o, lse = _attend(dict(c, kc=kc))
    blind = torch.from_numpy(~tree.mask(c["parents"][0])[:, node]).cuda()
    assert blind.sum() >= 15
    assert torch.equal(o[blind], o_ref[blind]) and torch.equal(lse[blind], lse_ref[blind])


def test_tree_attention_many_sequences_and_long_caches(cuda_device):
    rng = np.random.default_rng(12)
    lengths = [(int(rng.integers(1, 64)), int(rng.integers(64, 900))) for _ in range(150)]
    c = _case(lengths, 8, 2, 64, 16, seed=12)
    o, lse = _attend(c)
    _check(c, o, lse, sequences=[0, 1, 75, 148, 149])
    c = _case([(64, 20000), (17, 30000)], 8, 1, 128, 64, seed=13)
    o, lse = _attend(c)
    _check(c, o, lse, sequences=[1])
    assert api.device_status() == 0


def test_tree_attention_is_deterministic_and_on_two_streams(cuda_device):
    cases = [_case([(40, 3000), (64, 1000)], 8, 2, 128, 16, seed=20 + i) for i in range(2)]
    plans = [_plan(c) for c in cases]
    masks = [api.tree_mask(c["packed"], _i32(c["cu"]), _i32(c["kv"]))[0] for c in cases]
    spaces = [api.attn_paged_workspace(128) for _ in cases]
    want = [_attend(*x) for x in zip(cases, plans, masks)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i] = _attend(cases[i], plans[i], masks[i], workspace=spaces[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])
    assert api.device_status() == 0


def test_tree_attention_refusals(cuda_device):
    c = _case([(4, 100)], 2, 1, 64, 16, seed=15)
    mask, _ = api.tree_mask(c["packed"], _i32(c["cu"]), _i32(c["kv"]))
    for bad in (mask[:3], mask.int(), mask[0], mask.cpu(), mask.float()):
        with pytest.raises(ValueError):
            _attend(c, mask=bad)
    with pytest.raises(api.RFError):
        _attend(c, mask=mask[:, :0])
    with pytest.raises(ValueError):
        _attend(c, plan=_plan(c, True))
    # a causal plan that passed for another: nothing is computed, and it is reported
    plan = _plan(c, True)
    plan.causal = False
    out = torch.full((4, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    _attend(c, plan=plan, mask=mask, out=out)
    with pytest.raises(api.RFError):
        api.device_status()
    assert (out == 5).all()
    with pytest.raises(api.RFError):
        api.tree_mask(c["packed"], _i32(c["cu"]), _i32(c["kv"]), 17)
    with pytest.raises(api.RFError):
        api.tree_mask(c["packed"], _i32(c["cu"]), _i32(c["kv"]), 0)
    with pytest.raises(ValueError):
        api.tree_mask(c["packed"].long(), _i32(c["cu"]), _i32(c["kv"]))


# ---------------------------------------------------------------- the walk

@pytest.mark.parametrize("sizes,lead,pad,vocab", [
    ([1], 0, 0, 3), ([32], 0, 0, 2), ([64, 1, 0, 7, 40], 0, 0, 2), ([5, 0, 9], 2, 6, 2),
    ([300, 2, 1500], 0, 0, 2), ([33] * 200, 0, 0, 3), ([0, 0], 0, 4, 2), ([1200], 0, 0, 1),
])
def test_tree_accept(cuda_device, sizes, lead, pad, vocab):
    rng = np.random.default_rng(sum(sizes) + vocab)
    parents = [_parents(n, rng, 3) for n in sizes]
    T = lead + sum(sizes) + pad
    cu = [c + lead for c in _offsets(sizes)]
    tokens, sampled = rng.integers(0, vocab, (2, T))
    sampled[rng.random(T) < 0.02] = -1
    kv = [n + int(rng.integers(0, 50)) for n in sizes]
    packed = [0] * lead + sum(parents, []) + [0] * pad
    got = api.tree_accept(_i32(packed), _i32(tokens), _i32(sampled), _i32(cu), _i32(kv))
    assert api.device_status() == 0
    path, out, n_path, base, new_len = (t.cpu().tolist() for t in got)
    want_path, want_out = [-1] * T, [-1] * T
    for b, p in enumerate(parents):
        nodes, drawn = tree.accept(p, tokens[cu[b]:cu[b + 1]].tolist(),
                                   sampled[cu[b]:cu[b + 1]].tolist())
        want_path[cu[b]:cu[b] + len(nodes)] = nodes
        want_out[cu[b]:cu[b] + len(nodes)] = drawn
        assert (n_path[b], base[b], new_len[b]) == (len(nodes), kv[b] - len(p),
                                                    kv[b] - len(p) + len(nodes))
    assert path == want_path and out == want_out


def test_tree_accept_parents_that_are_none(cuda_device):
    # numbers out of range, and a parent behind its child, are never followed
    path, out, n_path, _, _ = api.tree_accept(
        _i32([7, 2, 0, -9, 1 << 30]), _i32([1] * 5), _i32([1] * 5), _i32([0, 5]), _i32([5]))
    assert n_path.tolist() == [2] and path.tolist() == [0, 2, -1, -1, -1]
    with pytest.raises(ValueError):
        api.tree_accept(_i32([-1]), _i32([1]).long(), _i32([1]), _i32([0, 1]), _i32([1]))
    with pytest.raises(ValueError):
        api.tree_accept(_i32([-1]), _i32([1, 2]), _i32([1]), _i32([0, 1]), _i32([1]))


# ---------------------------------------------------------------- steps

def _model(vocab, gen):
    """A layer of weights: embeddings, and projections to q, k, v and back."""
    H, Hkv, d = 4, 2, 64
    emb = torch.randn(vocab, 128, generator=gen).cuda()
    w = (torch.randn(128, (H + 2 * Hkv) * d, generator=gen) / 11).bfloat16().cuda()
    back = (torch.randn(H * d, vocab, generator=gen) / 4).cuda()
    ang = torch.arange(200)[:, None] / 30.0 ** (torch.arange(32) / 32)
    return emb, w, back, torch.cat([ang.cos(), ang.sin()], 1).cuda()


def test_decoding_with_trees_over_a_paged_cache(cuda_device):
    """Greedy decoding with trees of drafts, some of them right, emits the tokens of
    decoding one by one: nodes appended and attended to, tokens drawn, the walk, rows
    moved together, pages taken and given back."""
    vocab, B, page, width, H, Hkv, d = 50, 3, 8, 20, 4, 2, 64
    gen = torch.Generator().manual_seed(40)
    rng = np.random.default_rng(40)
    emb, w, back, cs = _model(vocab, gen)
    ones = torch.ones(200, vocab, device="cuda")

    def forward(tokens, pos, slots, pool, attend):
        qkv = (emb[tokens.long()].bfloat16() @ w).view(-1, H + 2 * Hkv, d)
        q = api.kv_append_paged(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], pool[0], pool[1],
                                slots, pos, cs)
        o, _ = attend(q)
        return (o.float().view(-1, H * d) @ back)

    # one by one
    start = [3, 7, 11]
    pool = torch.zeros(2, B * width, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    cu1 = _i32(range(B + 1))
    now, plain, sure = _i32(start), [[] for _ in range(B)], [24] * B
    for step in range(24):
        kv = _i32([step + 1] * B)
        pos, slots = api.paged_slots(cu1, kv, table, page, B * width, B)
        plan = api.PagedPlan(cu1, kv, B, H, Hkv, page, width)
        logits = forward(now, pos, slots, pool, lambda q: api.attn_paged(q, *pool, table, plan))
        # a tree's roundings (bf16 outputs, 256 of them a logit) draw the same token
        # where the best two are well apart
        best = logits.topk(2).values
        for b, gap in enumerate((best[:, 0] - best[:, 1]).tolist()):
            if gap < 0.05:
                sure[b] = min(sure[b], step)
        now, _ = api.sample_rows(logits, ones[:B], torch.zeros(B, device="cuda"))
        for b, t in enumerate(now.tolist()):
            plain[b].append(t)

    # with trees: the root is the last token; drafts are the right ones or others
    refs = torch.zeros(40, dtype=torch.int32, device="cuda")
    pool = torch.zeros(2, 1, 40, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    length = _i32([0] * B)
    got, now, steps = [[] for _ in range(B)], list(start), 0
    while min(map(len, got)) < 20:
        steps += 1
        parents, tokens = [], []
        for b in range(B):
            n = int(rng.integers(1, 12))
            p = _parents(n, rng, 4)
            depth = tree.depths(p)
            t = [now[b]]
            for i in range(1, n):
                k = len(got[b]) + depth[i] - 1
                right = k < len(plain[b]) and rng.random() < 0.7
                t.append(plain[b][k] if right else int(rng.integers(0, vocab)))
            parents.append(p)
            tokens.append(t)
        cu = _i32(_offsets([len(p) for p in parents]))
        par, tok = _i32(sum(parents, [])), _i32(sum(tokens, []))
        T = par.numel()
        grown = length + cu[1:] - cu[:-1]
        src, dst, left = api.pages_grow(table, length, grown, refs, page)
        assert left.item() >= 0 and (src == -1).all()
        mask, pos = api.tree_mask(par, cu, grown)
        _, slots = api.paged_slots(cu, grown, table, page, 40, T)
        plan = api.PagedPlan(cu, grown, T, H, Hkv, page, width, causal=False)
        logits = forward(tok, pos, slots, pool[:, 0],
                         lambda q: api.attn_paged(q, *pool[:, 0], table, plan, tree_mask=mask))
        drawn, _ = api.sample_rows(logits, ones[:T], torch.zeros(T, device="cuda"))
        path, out, n_path, base, new_len = api.tree_accept(par, tok, drawn, cu, grown)
        api.kv_compact_paged(pool[0], pool[1], table, path, cu, n_path, base)
        api.pages_release(table, grown, refs, page, new_len)
        length = new_len
        for b, c in enumerate(cu.tolist()[:-1]):
            got[b] += out.tolist()[c:c + n_path[b]]
            now[b] = got[b][-1]
        assert api.device_status() == 0
        used = sum(-(-n // page) for n in length.tolist())
        assert refs.sum().item() == used == (refs > 0).sum().item()
    for b in range(B):
        n = min(len(got[b]), sure[b])
        assert got[b][:n] == plain[b][:n]
    assert sum(sure) > 20 and steps < 20       # several tokens a step


def test_a_tree_step_captured_and_replayed_with_other_trees(cuda_device):
    """One graph of a whole step, padded to T nodes, replayed with other trees, lengths
    and tables, gives what the calls give one by one, to the bit."""
    B, T, H, Hkv, d, page, width, vocab = 3, 48, 8, 2, 64, 16, 20, 97
    gen, rng = torch.Generator().manual_seed(50), np.random.default_rng(50)
    pools = torch.randn(2, 2, B * width + 1, page, Hkv, d, generator=gen).bfloat16().cuda()
    back = torch.randn(H * d, vocab, generator=gen).cuda()
    expo = torch.empty(T, vocab).exponential_(generator=gen).clamp_(1e-20).cuda()
    limits = [torch.full((T,), 0.8, device="cuda"), _i32([20] * T),
              torch.full((T,), 0.9, device="cuda"), torch.full((T,), 0.02, device="cuda")]
    ws = api.attn_paged_workspace(d)

    def inputs():
        sizes = [int(rng.integers(1, 17)) for _ in range(B)]
        kv = [n + int(rng.integers(0, width * page - n + 1)) for n in sizes]
        parents = sum((_parents(n, rng) for n in sizes), [])
        pad = T - len(parents)
        return (torch.randn(T, H, d, generator=gen).bfloat16().cuda(), _i32(_offsets(sizes)),
                _i32(kv), _i32(parents + [-1] * pad), _i32(rng.integers(0, vocab, T)),
                _i32(rng.permutation(B * width).reshape(B, width)))

    def step(state, pool, plan, out):
        q, cu, kv, parent, tokens, table = state
        mask, pos = api.tree_mask(parent, cu, kv)
        plan.update(cu, kv)
        o, lse = api.attn_paged(q, pool[0][0], pool[1][0], table, plan, out=out, workspace=ws,
                                tree_mask=mask)
        drawn, logprob = api.sample_rows(o.float().view(T, -1) @ back, expo, *limits)
        path, emitted, n_path, base, new_len = api.tree_accept(parent, tokens, drawn, cu, kv)
        api.kv_compact_paged(pool[0], pool[1], table, path, cu, n_path, base)
        return o, mask, pos, drawn, logprob, path, emitted, n_path, base, new_len

    static = inputs()
    out = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
    plan = api.PagedPlan(static[1], static[2], T, H, Hkv, page, width, causal=False)
    pool = pools.clone()
    step(static, pool, plan, out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(static, pool, plan, out)
    walked = 0
    for turn in range(4):
        new = inputs()
        if turn > 1:  # drafts that are drawn: every node's is its parent's draw
            first = step(new, pools.clone(), plan, torch.zeros_like(out))[3].tolist()
            cu, parent = new[1].tolist(), new[3].tolist()
            for c0, c1 in zip(cu, cu[1:]):
                for i in range(c0 + 1, c1):
                    new[4][i] = first[c0 + parent[i]]
        for a, b in zip(static, new):
            a.copy_(b)
        pool.copy_(pools)
        out.zero_()
        other = pools.clone()
        want = step(new, other, plan, torch.zeros_like(out))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(pool, other)
        assert api.device_status() == 0
        walked += want[7].sum().item()
    assert walked > 4 * B


def _poison(*sizes):
    """What torch's allocator hands out next for int32 outputs of these sizes holds
    numbers that no call gives."""
    held = [torch.full((n,), 0x55555555, dtype=torch.int32, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    del held


BAD_OFFSETS = [
    ([0, 4, 20], 10), ([-1, 1, 2], 3), ([0, 20, 5, 8], 8), ([0, 3, 12, 3, 7], 9), ([5, 1, 3], 6),
    ([-5, -3, 2, 4], 6), ([9, 9, 9], 6), ([3, -1], 5), ([0, 1 << 30, -(1 << 30), 2], 4),
    ([600] + list(range(0, 600, 2)), 605),
    ([1000 if i % 10 == 3 else 2 * i for i in range(301)], 640),
    ([-7 if i % 50 == 49 else 3 * i + 4 for i in range(400)], 1300),
]


@pytest.mark.parametrize("cu,T", BAD_OFFSETS)
def test_rows_of_no_sequence_where_offsets_contradict_themselves(cuda_device, cu, T):
    # rows that no sequence with good offsets has hold 0 in masks and positions, -1 in
    # paths and tokens; the others' are theirs
    B = len(cu) - 1
    rng = np.random.default_rng(T)
    good = [0 <= a <= b <= T for a, b in zip(cu, cu[1:])]
    parent, token = np.full(T, -1), rng.integers(0, 2, T)
    kv = [0] * B
    m_ref, p_ref = np.zeros((T, 16), np.int64), np.zeros(T, np.int64)
    path, out, n_path = np.full(T, -1), np.full(T, -1), [0] * B
    for b in range(B):
        n, rows = cu[b + 1] - cu[b], slice(cu[b], cu[b + 1])
        kv[b] = 20 + b
        if good[b] and n:
            p = _parents(n, rng)
            parent[rows] = p
            m_ref[rows] = tree.words(tree.mask(p), 16)
            p_ref[rows] = kv[b] - n + tree.depths(p)
            nodes, drawn = tree.accept(p, token[rows].tolist(), token[rows].tolist())
            path[cu[b]:cu[b] + len(nodes)], out[cu[b]:cu[b] + len(nodes)] = nodes, drawn
            n_path[b] = len(nodes)
    assert not all(good)
    args = [_i32(x) for x in (parent, token, token, cu, kv)]
    _poison(32 * T, T)
    mask, pos = api.tree_mask(args[0], args[3], args[4], 16)
    with pytest.raises(api.RFError):
        api.device_status()
    assert np.array_equal(mask.cpu().numpy(), m_ref) and pos.tolist() == p_ref.tolist()
    _poison((T + 3) // 4 * 8 + (B + 3) // 4 * 12)
    got = api.tree_accept(*args)
    with pytest.raises(api.RFError):
        api.device_status()
    assert got[0].tolist() == path.tolist() and got[1].tolist() == out.tolist()
    assert got[2].tolist() == n_path


@pytest.mark.parametrize("T", [0, 1, 37])
def test_trees_of_no_sequences(cuda_device, T):
    # a padded step in which no sequence takes part
    x, cu, none = _i32([0] * T), _i32([0]), _i32([])
    _poison(4 * T, T)
    mask, pos = api.tree_mask(x, cu, none, 2)
    assert mask.shape == (T, 2) and not mask.any() and pos.tolist() == [0] * T
    _poison((T + 3) // 4 * 8)
    path, out, n_path, base, new_len = api.tree_accept(x, x, x, cu, none)
    assert path.tolist() == out.tolist() == [-1] * T
    assert n_path.shape == base.shape == new_len.shape == (0,)
    assert api.device_status() == 0
