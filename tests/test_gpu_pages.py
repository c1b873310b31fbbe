"""Housekeeping of a paged cache on the GPU against the oracle: kept rows moved
together, pages copied, forked, handed out and taken back."""

import numpy as np
import pytest
import torch

from online_softmax_attention_rf_gb300 import api
from oracle import tree
from tests.helpers import f64

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _pool(layers, pages, page, Hkv, d, dtype, order, gen):
    """A pool [layers, pages, page, Hkv, d] (layers None: without them) whose
    dimensions lie in another order in memory."""
    dims = dict(l=layers or 1, p=pages, t=page, h=Hkv)
    c = torch.randn(*(dims[x] for x in order), d, generator=gen).to(dtype).cuda()
    c = c.permute(*(order.index(x) for x in "lpth"), 4)
    return c[0] if layers is None else c


def _tables(lens, page, spare, gen):
    need = [tree.pages(n, page) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=gen).tolist()
    rows, at, width = [], 0, max(need + [1]) + 1
    for m in need:
        rows.append(perm[at:at + m] + [0] * (width - m))
        at += m
    return rows, pages


ORDERS = ["lpth", "lpht", "hlpt", "tplh"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,share,page,layers,Hkv,d,order", [
    ([1], 1.0, 8, None, 1, 64, "lpth"),
    ([40, 0, 7, 100], 0.5, 16, 3, 2, 64, "lpth"),
    ([300, 5], 0.9, 24, 2, 8, 128, "lpht"),
    ([1000], 0.3, 1, None, 3, 16, "lpth"),
    ([700, 699, 3], 0.05, 64, 2, 4, 8, "hlpt"),
    ([500] * 9, 0.7, 32, 1, 5, 80, "tplh"),
    ([4000], 0.6, 128, 1, 8, 128, "lpth"),
    ([90, 200], 0.5, 16, None, 20, 1024, "lpth"),       # a row of 20 heads takes several CTAs
])
def test_kv_compact_paged(cuda_device, dtype, lens, share, page, layers, Hkv, d, order):
    gen, rng = torch.Generator().manual_seed(sum(lens)), np.random.default_rng(sum(lens))
    rows, pages = _tables(lens, page, 3, gen)
    pools = [_pool(layers, pages, page, Hkv, d, dtype, order, gen) for _ in range(2)]
    keep = [sorted(rng.choice(n, int(round(share * n)), replace=False).tolist()) for n in lens]
    want = [f64(p) for p in pools]
    for p in want:
        for cache in (p if layers else [p]):
            for r, k in zip(rows, keep):
                tree.compact(cache, r, page, k, 0)
    cu = np.cumsum([0] + [len(k) for k in keep])
    assert api.kv_compact_paged(*pools, _i32(rows), _i32(sum(keep, [])), _i32(cu)) is None
    assert api.device_status() == 0
    for p, w in zip(pools, want):
        assert np.array_equal(f64(p), w)


def test_kv_compact_paged_bases_and_counts(cuda_device):
    # lists longer than what is kept of them, bases inside a page, tables with room
    # between their rows
    gen, rng = torch.Generator().manual_seed(1), np.random.default_rng(1)
    lens, page = [90, 33, 64, 12], 16
    rows, pages = _tables(lens, page, 2, gen)
    pools = [_pool(2, pages, page, 2, 64, torch.bfloat16, "lpth", gen) for _ in range(2)]
    base = [50, 0, 63, 5]
    keep = [sorted(rng.choice(n - b, min(n - b, 20), replace=False).tolist())
            for n, b in zip(lens, base)]
    counts = [7, 20, 1, 0]
    want = [f64(p) for p in pools]
    for p in want:
        for cache in p:
            for b in range(4):
                tree.compact(cache, rows[b], page, keep[b][:counts[b]], base[b])
    wide = torch.full((4, 40), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :len(rows[0])] = _i32(rows)
    api.kv_compact_paged(*pools, wide[:, :len(rows[0])], _i32(sum(keep, [])),
                         _i32(np.cumsum([0] + [len(k) for k in keep])), _i32(counts), _i32(base))
    assert api.device_status() == 0
    for p, w in zip(pools, want):
        assert np.array_equal(f64(p), w)


@pytest.mark.parametrize("keep,cu,n_keep,base,moved", [
    ([1, 1, 5], [0, 3], None, None, [(1, 0), (5, 2)]),          # one twice
    ([4, 2, 6], [0, 3], None, None, [(4, 0), (6, 2)]),          # does not ascend
    ([-1, 3, 6], [0, 3], None, None, [(3, 1), (6, 2)]),
    ([1, 3, 99], [0, 3], None, None, [(1, 0), (3, 1)]),         # behind the table
    ([1, 3, 20], [0, 3], None, None, [(1, 0), (3, 1)]),         # an entry that is no page
    ([1, 3, 5], [0, 4], None, None, []),                        # offsets out of range
    ([1, 3, 5], [-1, 3], None, None, []),
    ([1, 3, 5], [2, 1], None, None, []),
    ([1, 3, 5], [0, 3], [4], None, []),
    ([1, 3, 5], [0, 3], [-1], None, []),
    ([1, 3, 5], [0, 3], None, [-2], [(3, 0)]),                  # rows before the first
])
def test_kv_compact_paged_reports_what_it_skips(cuda_device, keep, cu, n_keep, base, moved):
    kc = torch.arange(32.0, device="cuda").view(4, 8, 1, 1).expand(4, 8, 1, 64).contiguous()
    vc, old = kc + 100, kc.clone()
    table = _i32([[2, 0, 77]])
    api.kv_compact_paged(kc, vc, table, _i32(keep), _i32(cu),
                         None if n_keep is None else _i32(n_keep),
                         None if base is None else _i32(base))
    with pytest.raises(api.RFError):
        api.device_status()
    want = old.clone()
    place = lambda p: ([2, 0][p // 8], p % 8)  # noqa: E731
    for a, b in moved:
        want[place(b)] = old[place(a)]
    assert torch.equal(kc, want) and torch.equal(vc, want + 100)


def test_kv_compact_paged_offsets_beyond_32_bits(cuda_device):
    # a pool of 9 GB: rows that move lie behind 2^31 and 2^32 bytes, in both layers
    layers, pages, page, Hkv, d = 2, 4500, 64, 8, 1024
    kc = torch.zeros(layers, pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    rows = [[4499, 3, 4100]]
    for l in range(2):
        for i, p in enumerate(rows[0]):
            kc[l, p] = torch.arange(page, device="cuda").view(page, 1, 1) + 64 * i + 1000 * l
    api.kv_compact_paged(kc, vc, _i32(rows), _i32([0, 70, 130, 191]), _i32([0, 4]))
    assert api.device_status() == 0
    for l in range(2):
        got = kc[l, 4499, :4].float()
        # 1064 and beyond round to eights in bf16
        want = torch.tensor([0., 70, 130, 191]).cuda() + 1000 * l
        assert torch.equal(got, want.bfloat16().float().view(4, 1, 1).expand_as(got))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layers,page,Hkv,d,order", [
    (None, 8, 1, 64, "lpth"), (3, 16, 2, 64, "lpht"), (2, 24, 5, 8, "hlpt"), (2, 1, 3, 128, "tplh"),
    (1, 256, 8, 128, "lpth"),
])
def test_kv_copy_pages(cuda_device, dtype, layers, page, Hkv, d, order):
    gen = torch.Generator().manual_seed(page)
    pools = [_pool(layers, 30, page, Hkv, d, dtype, order, gen) for _ in range(2)]
    want = [p.clone() for p in pools]
    src, dst = [3, -1, 3, 29, 7, 7], [4, 5, 0, 1, -1, 7]
    for p in want:
        for s, t in zip(src, dst):
            if s >= 0 and t >= 0:
                p.select(-4, t).copy_(p.select(-4, s).clone())
    assert api.kv_copy_pages(*pools, _i32(src), _i32(dst)) is None
    assert api.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(pools, want))
    api.kv_copy_pages(*pools, _i32([2, 30, 4, 1 << 30]), _i32([6, 1, 30, 2]))
    with pytest.raises(api.RFError):
        api.device_status()
    for p, w in zip(pools, want):
        w.select(-4, 6).copy_(w.select(-4, 2))
        assert torch.equal(p, w)


def _fork_case(B, width, page, pages, rng, cols):
    lens = [int(rng.integers(0, (cols - 3) * page)) for _ in range(B)]
    perm = rng.permutation(pages).tolist()
    table, at = [[0] * cols for _ in range(B)], 0
    refs = [0] * pages
    for r, n in zip(table, lens):
        m = tree.pages(n, page)
        r[:m] = perm[at:at + m]
        for p in r[:m]:
            refs[p] = 1
        at += m
    for p in perm[at:]:
        if rng.random() < 0.4:
            refs[p] = int(rng.integers(1, 4))      # other sequences' pages
    src = [int(rng.integers(0, B)) for _ in range(width)] if B else []
    return lens, table, refs, src


@pytest.mark.parametrize("B,width,page,pages,cols", [
    (1, 1, 16, 20, 4), (1, 5, 16, 64, 6), (4, 30, 8, 700, 7), (3, 3, 1, 90, 12), (50, 200, 32, 5001, 9),
    (7, 1500, 16, 40003, 20),
])
def test_pages_fork_grow_release(cuda_device, B, width, page, pages, cols):
    rng = np.random.default_rng(pages)
    lens, table, refs, src = _fork_case(B, width, page, pages, rng, cols)
    d_table, d_refs = _i32(table), _i32(refs)
    out = [[-7] * cols for _ in range(width)]
    d_out = _i32(out)
    got = api.pages_fork(d_table, _i32(lens), _i32(src), d_out, d_refs, page)
    new_lens = tree.fork(table, lens, src, out, refs, page)
    assert got.tolist() == new_lens
    assert d_out.tolist() == out and d_refs.tolist() == refs
    # grow: some rows not at all, most by a few tokens, some by pages
    new = [n + int(rng.choice([0, 1, 2, page, 2 * page + 1])) for n in new_lens]
    c_src, c_dst, left = api.pages_grow(d_out, got, _i32(new), d_refs, page)
    want = tree.grow(out, new_lens, new, refs, page)
    assert (c_src.tolist(), c_dst.tolist(), left.item()) == want
    assert d_out.tolist() == out and d_refs.tolist() == refs
    # the parents go (their pages stay as long as they have owners), then the children shrink
    api.pages_release(d_table, _i32(lens), d_refs, page)
    tree.release(table, lens, refs, page)
    assert d_refs.tolist() == refs
    grown = new if want[2] >= 0 else new_lens
    less = [max(0, n - int(rng.integers(0, 3 * page))) for n in grown]
    api.pages_release(d_out, _i32(grown), d_refs, page, _i32(less))
    tree.release(out, grown, refs, page, less)
    assert d_refs.tolist() == refs
    api.pages_release(d_out, _i32(less), d_refs, page)
    tree.release(out, less, refs, page)
    assert d_refs.tolist() == refs and min(refs) >= 0
    assert api.device_status() == 0


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_pages_grow_takes_the_lowest_free_pages(cuda_device, shift):
    # refs at every alignment, counts at every border of a share of the pages
    for pages in (1, 5, 33, 4096, 32768, 32771, 100001):
        rng = np.random.default_rng(pages)
        refs = (rng.random(pages) < 0.7).astype(int).tolist()
        free = refs.count(0)
        held = torch.ones(pages + 4, dtype=torch.int32, device="cuda")
        held[shift:shift + pages] = _i32(refs)
        d_refs = held[shift:shift + pages]
        for want in sorted({0, 1, free // 2, free, free + 1}):
            r, table = list(refs), [[0] * (free + 2)]
            d_r = d_refs.clone() if shift == 0 else held.clone()[shift:shift + pages]
            d_table = _i32(table)
            res = tree.grow(table, [0], [want], r, 1)
            got = api.pages_grow(d_table, _i32([0]), _i32([want]), d_r, 1)
            assert [t.tolist()[0] for t in got] == [res[0][0], res[1][0], res[2]]
            assert d_table.tolist() == table and d_r.tolist() == r
    assert api.device_status() == 0


def test_pages_grow_when_all_owners_write(cuda_device):
    # three rows hold one partly filled page; with a fourth owner elsewhere all
    # three get copies, without one the last keeps it
    for owners in (3, 4):
        refs, table = [owners, 0, 0, 0, 0, 0], [[0, 9], [0, 9], [0, 9]]
        d_refs, d_table = _i32(refs), _i32(table)
        res = tree.grow(table, [2, 2, 2], [3, 9, 4], refs, 8)
        got = api.pages_grow(d_table, _i32([2, 2, 2]), _i32([3, 9, 4]), d_refs, 8)
        assert [t.tolist() for t in got] == [res[0], res[1], [res[2]]]
        assert d_table.tolist() == table and d_refs.tolist() == refs
        assert res[0] == ([0, 0, -1] if owners == 3 else [0, 0, 0])


def test_pages_calls_report_what_they_skip(cuda_device):
    def reported():
        with pytest.raises(api.RFError):
            api.device_status()

    refs = _i32([1, 1, 0, 0])
    table = _i32([[0, 99], [1, -1]])
    out = _i32([[5, 5]] * 4)
    # a source, a length and a page that are none
    got = api.pages_fork(table, _i32([12, 99]), _i32([0, 1, 2, -1]), out, refs, 8)
    assert got.tolist() == [12, 0, 0, 0] and refs.tolist() == [2, 1, 0, 0]
    assert out.tolist() == [[0, 99]] + [[5, 5]] * 3
    reported()
    # pages without an owner, and numbers out of range, are left alone
    api.pages_release(_i32([[2, 1], [99, -5]]), _i32([16, 16]), refs, 8)
    assert refs.tolist() == [2, 0, 0, 0]
    reported()
    api.pages_release(_i32([[0, 0]]), _i32([17]), refs, 8)
    assert refs.tolist() == [2, 0, 0, 0]
    reported()
    # lengths out of range get nothing; the other row its page
    table = _i32([[0, 0], [0, 0], [0, 0]])
    got = api.pages_grow(table, _i32([0, -1, 0]), _i32([17, 8, 8]), refs, 8)
    assert table.tolist() == [[0, 0], [0, 0], [1, 0]] and got[2].item() == 2
    reported()
    # a partly filled page that is none cannot be shared
    got = api.pages_grow(_i32([[50, 0]]), _i32([3]), _i32([4]), refs, 8)
    assert got[0].tolist() == [-1] and got[2].item() == 2
    reported()


def test_pages_calls_of_nothing(cuda_device):
    none, refs = _i32([]), _i32([1, 0, 0])
    table = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    assert api.pages_fork(table, none, none, table, refs, 8).shape == (0,)
    src, dst, left = api.pages_grow(table, none, none, refs, 8)
    assert src.shape == dst.shape == (0,) and left.item() == 2
    api.pages_release(table, none, refs, 8)
    pool = torch.ones(2, 3, 8, 1, 64, device="cuda")
    api.kv_copy_pages(pool[0], pool[1], none, none)
    api.kv_compact_paged(pool[0], pool[1], table, none, _i32([0]))
    api.kv_compact_paged(pool[:0], pool[:0], _i32([[0]]), _i32([1]), _i32([0, 1]))
    assert (pool == 1).all() and refs.tolist() == [1, 0, 0] and api.device_status() == 0


def test_beams_reordered_in_place_of_copies(cuda_device):
    # beam search: each step some beams go on twice and others not at all; what each
    # row holds is followed on the host
    B, page, pages, cols, d = 6, 4, 80, 16, 16
    rng = np.random.default_rng(50)
    kc = torch.zeros(1, pages, page, 1, d, device="cuda")
    vc = torch.zeros_like(kc)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.zeros(B, cols, dtype=torch.int32, device="cuda")
    length, held = _i32([0] * B), [[] for _ in range(B)]
    for step in range(40):
        if step:
            src = rng.integers(0, B, B)
            other = torch.zeros_like(table)
            lens = api.pages_fork(table, length, _i32(src), other, refs, page)
            api.pages_release(table, length, refs, page)
            table, length = other, lens
            held = [list(held[s]) for s in src]
        a, b, left = api.pages_grow(table, length, length + 1, refs, page)
        api.kv_copy_pages(kc, vc, a, b)
        assert left.item() >= 0
        length = length + 1
        cu = _i32(range(B + 1))
        _, slots = api.paged_slots(cu, length, table, page, pages, B)
        value = rng.integers(0, 1000, B)
        x = torch.tensor(value, dtype=torch.float32, device="cuda").view(B, 1, 1).repeat(1, 1, d)
        api.kv_append_paged(None, x, -x, kc[0], vc[0], slots)
        for h, v in zip(held, value):
            h.append(int(v))
    rows = table.tolist()
    for b in range(B):
        got = [kc[0, rows[b][j // page], j % page, 0, 0].item() for j in range(40)]
        assert got == held[b]
        assert [-vc[0, rows[b][j // page], j % page, 0, 0].item() for j in range(40)] == held[b]
    api.pages_release(table, length, refs, page)
    assert refs.sum().item() == 0 and api.device_status() == 0


def test_housekeeping_captured_and_on_another_stream(cuda_device):
    page, pages, cols, n = 8, 200, 6, 12
    rng = np.random.default_rng(60)
    lens, table, refs, src = _fork_case(6, n, page, pages, rng, cols)
    kc0, vc0 = torch.randn(2, 2, pages, page, 2, 64, device="cuda")
    state = [_i32(table), _i32(lens), _i32(src), _i32(refs), _i32([[0] * cols] * n), kc0.clone(),
             vc0.clone(), _i32([1])]
    keep, cu = _i32(list(range(1, 7)) * n), _i32(range(0, 6 * n + 1, 6))

    def step(table, lens, src, refs, out, kc, vc, more):
        got = api.pages_fork(table, lens, src, out, refs, page)
        a, b, left = api.pages_grow(out, got, got + more, refs, page)
        api.kv_copy_pages(kc, vc, a, b)
        api.kv_compact_paged(kc, vc, out, keep, cu, torch.where(got >= 7, 6, 0).int())
        api.pages_release(table, lens, refs, page)
        return got, a, b, left

    def result(st, out):
        torch.cuda.synchronize()
        assert api.device_status() == 0
        return [t.clone() for t in list(out) + [st[3], st[4], st[5], st[6]]]

    # rows share pages, so that moving theirs together would meet: one child a parent
    state[2] = _i32(rng.permutation(6).tolist() + [0] * 6)[:6]
    state[4] = state[4][:6].contiguous()
    keep, cu = keep[:36], cu[:7]
    fresh = [t.clone() for t in state]
    st = [t.clone() for t in fresh]
    want = result(st, step(*st))
    side = torch.cuda.Stream()
    st = [t.clone() for t in fresh]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out = step(*st)
    assert all(torch.equal(a, b) for a, b in zip(result(st, out), want))
    g = torch.cuda.CUDAGraph()
    st = [t.clone() for t in fresh]
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = step(*st)
    for _ in range(2):
        for a, b in zip(st, fresh):
            a.copy_(b)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(result(st, out), want))


def test_housekeeping_refusals(cuda_device):
    pool = torch.zeros(2, 4, 8, 2, 64, device="cuda")
    k, v = pool[0], pool[1]
    t, one, cu = _i32([[0, 1]]), _i32([0]), _i32([0, 1])
    refs = _i32([0] * 4)
    for bad in [lambda: api.kv_compact_paged(k, v[:3], t, one, cu),
                lambda: api.kv_compact_paged(k, v.bfloat16(), t, one, cu),
                lambda: api.kv_compact_paged(k.transpose(2, 3), v.transpose(2, 3), t, one, cu),
                lambda: api.kv_compact_paged(k, v, t.long(), one, cu),
                lambda: api.kv_compact_paged(k, v, t, one, one),
                lambda: api.kv_compact_paged(k, v, t, one, cu, n_keep=cu),
                lambda: api.kv_compact_paged(k, v, t, one, cu, base=one.cpu()),
                lambda: api.kv_compact_paged(k.half(), v.half(), t, one, cu),
                lambda: api.kv_copy_pages(k, v, one, cu),
                lambda: api.kv_copy_pages(k[0], v[0], one, one),
                lambda: api.pages_fork(t, one, one, _i32([[0, 1, 2]]), refs, 8),
                lambda: api.pages_fork(t, cu, one, t.clone(), refs, 8),
                lambda: api.pages_fork(t, one, one, t.clone(), refs.long(), 8),
                lambda: api.pages_grow(t, one, cu, refs, 8),
                lambda: api.pages_grow(t, one, None, refs, 8),
                lambda: api.pages_grow(t, one, one, refs.cpu(), 8),
                lambda: api.pages_release(t, cu, refs, 8),
                lambda: api.pages_release(t, one, refs, 8, new_len=cu)]:
        with pytest.raises((ValueError, TypeError)):
            bad()
    odd = torch.zeros(2, 4, 8, 2, 6, device="cuda")
    for bad in [lambda: api.kv_copy_pages(odd[0], odd[1], one, one),
                lambda: api.pages_fork(t, one, one, t, refs, 8),
                lambda: api.kv_copy_pages(k.flatten()[1:4 * 8 * 2 * 60 + 1].view(4, 8, 2, 60),
                                          v.flatten()[1:4 * 8 * 2 * 60 + 1].view(4, 8, 2, 60), one, one),
                lambda: api.pages_grow(t, one, one, refs, 0),
                lambda: api.pages_grow(t, one, one, refs[:0], 8),
                lambda: api.pages_release(t, one, refs, 1 << 31 - 1)]:
        with pytest.raises(api.RFError):
            bad()


def test_kv_copy_pages_of_a_long_list_and_large_pages(cuda_device):
    # pages of 134 MB and 2^20 pairs, nearly all of them empty: pairs times the parts of
    # a page pass 2^32
    n, page, Hkv, d = 1 << 20, 65552, 8, 128
    pools = []
    for i in range(2):
        c = torch.empty(5, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
        # every 16 bytes of the pool differ, up to a period that no page's length shares
        bits = torch.arange(c.numel(), dtype=torch.int32, device="cuda") % (30011 + 10 * i)
        c.copy_(bits.to(torch.int16).view(torch.bfloat16).view_as(c))
        pools.append(c)
    want = [p[:2].view(torch.int16).clone() for p in pools]
    src = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    dst = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    src[300], dst[300] = 0, 2
    src[n - 1], dst[n - 1] = 1, 4
    api.kv_copy_pages(*pools, src, dst)
    assert api.device_status() == 0
    for p, w in zip(pools, want):
        p = p.view(torch.int16)
        assert torch.equal(p[2], w[0]) and torch.equal(p[4], w[1]) and torch.equal(p[:2], w)
        assert not torch.equal(p[3], w[0])


def test_pages_grow_of_a_row_whose_last_page_has_no_owner(cuda_device):
    # page 0 is free, whatever row 0's entry says: the row gets nothing, the others theirs,
    # that page among them
    for owners in (0, -3):
        refs = _i32([owners, 1, 2, 0, 0])
        table = _i32([[0, 9, 9], [1, 9, 9], [2, 9, 9], [0, 9, 9]])
        src, dst, left = api.pages_grow(table, _i32([3, 5, 4, 6]), _i32([20, 9, 5, 6]), refs, 8)
        with pytest.raises(api.RFError):
            api.device_status()
        free = [p for p in (0, 3, 4) if owners == 0 or p > 0]
        assert table.tolist() == [[0, 9, 9], [1, free[0], 9], [free[1], 9, 9], [0, 9, 9]]
        assert src.tolist() == [-1, -1, 2, -1] and dst.tolist() == [-1, -1, free[1], -1]
        want = [owners, 1, 1, 0, 0]
        want[free[0]] = want[free[1]] = 1
        assert refs.tolist() == want and left.item() == len(free) - 2
    # a row that does not write to it is no matter
    refs, table = _i32([0, 1]), _i32([[0, 0], [0, 0]])
    api.pages_grow(table, _i32([3, 8]), _i32([3, 8]), refs, 8)
    assert api.device_status() == 0 and refs.tolist() == [0, 1]


@pytest.mark.parametrize("length,new", [(17, 5), (17, 17), (1 << 30, 0), (-1, 3), (3, -1), (3, 17)])
def test_pages_calls_report_lengths_out_of_range(cuda_device, length, new):
    # tables of two pages of 8 tokens: 17 tokens are too many, there or to be there
    refs, table = _i32([1, 1, 1, 0]), _i32([[0, 1], [2, 0]])
    api.pages_release(table, _i32([length, 8]), refs, 8, _i32([new, 0]))
    with pytest.raises(api.RFError):
        api.device_status()
    assert refs.tolist() == [1, 1, 0, 0]
    src, dst, left = api.pages_grow(table, _i32([length, 0]), _i32([new, 8]), refs, 8)
    with pytest.raises(api.RFError):
        api.device_status()
    assert table.tolist() == [[0, 1], [2, 0]] and refs.tolist() == [1, 1, 1, 0]
    assert src.tolist() == dst.tolist() == [-1, -1] and left.item() == 1


def test_pages_fork_gives_free_pages_no_owner(cuda_device):
    # pages 1 and 3 have no owner: many rows share them, none becomes theirs
    refs = _i32([1, 0, 2, -1])
    table = _i32([[0, 1, 2, 3], [2, 0, 9, 9]])
    out = torch.full((600, 4), 7, dtype=torch.int32, device="cuda")
    got = api.pages_fork(table, _i32([32, 16]), _i32([0] * 300 + [1] * 300), out, refs, 8)
    with pytest.raises(api.RFError):
        api.device_status()
    assert refs.tolist() == [601, 0, 602, -1]
    assert got.tolist() == [32] * 300 + [16] * 300
    assert out.tolist() == [[0, 1, 2, 3]] * 300 + [[2, 0, 7, 7]] * 300


def test_expanded_pools_are_refused(cuda_device):
    # layers or heads that are one memory: a row would be moved once for each of them
    x = torch.arange(24.0, device="cuda").view(3, 8, 1, 1).expand(3, 8, 1, 64).contiguous()
    for pool in (x.expand(2, 3, 8, 1, 64), x.expand(3, 8, 4, 64), x[:1].expand(3, 8, 1, 64)):
        other = pool.contiguous()
        for k, v in ((pool, other), (other, pool)):
            with pytest.raises(api.RFError):
                api.kv_compact_paged(k, v, _i32([[2, 0]]), _i32([1, 3, 5]), _i32([0, 3]))
            with pytest.raises(api.RFError):
                api.kv_copy_pages(k, v, _i32([0]), _i32([1]))
    assert torch.equal(x[:, :, 0, 0].flatten(), torch.arange(24.0, device="cuda"))


@pytest.mark.parametrize("most", [40, 400])     # lists of one chunk, and of several
@pytest.mark.parametrize("dtype,Hkv,d,order", [(torch.bfloat16, 8, 64, "lpth"),
                                               (torch.float32, 3, 80, "lpht")])
def test_kv_compact_paged_of_many_sequences_in_many_layers(cuda_device, most, dtype, Hkv, d, order):
    # more planes (k and v of a sequence's layers) than are in flight: a CTA takes several
    layers, B, page = 12, 64, 16
    gen, rng = torch.Generator().manual_seed(most), np.random.default_rng(most)
    lens = [int(rng.integers(1, most + 1)) for _ in range(B)]
    lens[0], lens[1] = most, 1
    rows, pages = _tables(lens, page, 5, gen)
    pools = [_pool(layers, pages, page, Hkv, d, dtype, order, gen) for _ in range(2)]
    keep = [sorted(rng.choice(n, int(rng.integers(0, n + 1)), replace=False).tolist())
            for n in lens]
    keep[0] = list(range(1, most))
    want = [p.clone() for p in pools]
    for r, kept in zip(rows, keep):
        place = lambda js: (_i32([r[j // page] for j in js]).long(),  # noqa: E731
                            _i32([j % page for j in js]).long())
        (p0, r0), (p1, r1) = place(kept), place(range(len(kept)))
        for w, p in zip(want, pools):
            w[:, p1, r1] = p[:, p0, r0]
    cu = np.cumsum([0] + [len(x) for x in keep])
    api.kv_compact_paged(*pools, _i32(rows), _i32(sum(keep, [])), _i32(cu))
    assert api.device_status() == 0
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


def test_pages_of_the_most_rows_that_grow_at_once(cuda_device):
    # thousands of rows share each partly filled page
    test_pages_fork_grow_release(cuda_device, 7, 16384, 16, 120011, 8)
    with pytest.raises(api.RFError):
        one = _i32([0] * 16385)
        api.pages_grow(one.view(-1, 1), one, one, _i32([0] * 8), 8)
