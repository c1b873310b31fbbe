"""The entries for drafted trees, sampling and cache pages without a GPU: sizes,
pointers, strides and types that they refuse on the host, and calls with nothing to
do."""

import ctypes

import pytest
import torch

from online_softmax_attention_rf_gb300 import api, build

A = 0x10000        # an aligned fake device address; never dereferenced
MIS = 0x10008
INV, UNS = api.RF_ERR_INVALID, api.RF_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def _call(L, name, ok, kw):
    a = dict(ok)
    assert not set(kw) - set(a), set(kw) - set(a)
    a.update(kw)
    st = getattr(L, name)(*a.values())
    if st != api.RF_OK:
        assert L.rf_last_error().startswith(name.encode()), L.rf_last_error()
    return st


MASK = dict(parent=A, cu_q=A, kv_len=A, B=2, T=5, words=1, mask=A, pos=A, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(words=0), INV), (dict(words=17), UNS),
    (dict(B=(1 << 20) + 1), INV), (dict(T=(1 << 28) + 1), INV), (dict(parent=None), INV),
    (dict(cu_q=None), INV), (dict(kv_len=None), INV), (dict(mask=None), INV),
    (dict(mask=A + 4), INV), (dict(pos=A + 2), INV), (dict(parent=A + 1), INV),
])
def test_tree_mask_rejects(L, kw, expect):
    assert _call(L, "rf_tree_mask", MASK, kw) == expect


ACCEPT = dict(parent=A, tokens=A, sampled=A, cu_q=A, kv_len=A, B=2, T=5, path=A, out=A, n_path=A,
              base=A, new_len=A, stream=None)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(T=-1), dict(B=(1 << 20) + 1), dict(T=(1 << 28) + 1),
    *[{n: None} for n in ACCEPT if ACCEPT[n] == A], *[{n: A + 2} for n in ACCEPT if ACCEPT[n] == A],
])
def test_tree_accept_rejects(L, kw):
    assert _call(L, "rf_tree_accept", ACCEPT, kw) == INV


TREE = dict(q=A, q_stride=4 * 64, k_cache=A, kp=16 * 128, kt=128, kh=64, v_cache=A, vp=16 * 128,
            vt=128, vh=64, page=16, num_pages=9, table=A, table_stride=4, max_pages=4, plan=A, B=2,
            T=5, H=4, Hkv=2, d=64, scale=0.1, o=A, lse=A, ws=A, ws_bytes=1 << 40, tree=A, words=1,
            dt=api.RF_BF16, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(words=0), INV), (dict(words=(1 << 24) + 1), INV), (dict(tree=None), INV),
    (dict(tree=A + 4), INV), (dict(dt=api.RF_F32), UNS), (dict(d=96), UNS), (dict(page=12), UNS),
    (dict(H=5), INV), (dict(scale=0.0), INV), (dict(q=MIS), INV), (dict(kt=0), INV),
    (dict(ws_bytes=0), INV), (dict(plan=None), INV), (dict(table_stride=3), INV),
])
def test_attn_paged_tree_rejects(L, kw, expect):
    assert _call(L, "rf_attn_paged_tree", TREE, kw) == expect


SAMPLE = dict(logits=A, stride=100, expo=A, temperature=A, top_k=A, top_p=A, min_p=A, B=2, V=100,
              token=A, logprob=A, dt=api.RF_BF16, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INV), (dict(V=0), INV), (dict(dt=7), INV), (dict(V=(1 << 20) + 1), UNS),
    (dict(B=(1 << 20) + 1), INV), (dict(stride=99), INV), (dict(stride=1 << 39), INV),
    (dict(logits=None), INV), (dict(expo=None), INV), (dict(token=None), INV),
    (dict(logits=A + 1), INV), (dict(logits=A + 2, dt=api.RF_F32), INV),
    *[({n: A + 2}, INV) for n in ("expo", "temperature", "top_k", "top_p", "min_p", "token",
                                  "logprob")],
])
def test_sample_rows_rejects(L, kw, expect):
    assert _call(L, "rf_sample_rows", SAMPLE, kw) == expect


def _pool(**kw):
    p = dict(k=A, v=A, layers=2, num_pages=9, page=16, Hkv=2, d=64, dt=api.RF_BF16)
    for c in "kv":
        p.update({c + "_layer_stride": 9 * 2048, c + "_page_stride": 2048, c + "_token_stride": 128,
                  c + "_head_stride": 64})
    p.update(kw)
    return ctypes.byref(api.RFKvPool(**p))


COMPACT = dict(pool=None, table=A, table_stride=4, B=2, max_pages=4, keep=A, N=7, cu_keep=A,
               n_keep=A, base=A, stream=None)
COPY = dict(pool=None, src=A, dst=A, n=3, stream=None)
POOLS = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(k=MIS), INV), (dict(v=MIS), INV),
    (dict(layers=-1), INV), (dict(layers=32768), INV), (dict(num_pages=0), INV), (dict(page=0), INV),
    (dict(Hkv=0), INV), (dict(d=0), INV), (dict(d=60), UNS), (dict(d=1032), UNS), (dict(dt=9), INV),
    (dict(page=1 << 16, num_pages=1 << 16), INV), (dict(page=1 << 20, num_pages=1, Hkv=64), INV),
    (dict(k_page_stride=2044), INV), (dict(v_head_stride=-64), INV), (dict(v_layer_stride=4), INV),
    (dict(k_token_stride=1 << 41), INV),
]


@pytest.mark.parametrize("pool,expect", POOLS)
@pytest.mark.parametrize("name,ok", [("rf_kv_compact_paged", COMPACT), ("rf_kv_copy_pages", COPY)])
def test_pools_rejected(L, name, ok, pool, expect):
    assert _call(L, name, ok, dict(pool=_pool(**pool))) == expect
    assert _call(L, name, ok, dict(pool=None)) == INV


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(N=-1), dict(max_pages=0), dict(table_stride=3), dict(table=None),
    dict(keep=None), dict(cu_keep=None), dict(keep=A + 2), dict(n_keep=A + 1), dict(base=A + 2),
    dict(max_pages=1 << 28), dict(N=(1 << 30) + 1),
])
def test_kv_compact_paged_rejects(L, kw):
    assert _call(L, "rf_kv_compact_paged", COMPACT, dict(kw, pool=_pool())) == INV


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n=(1 << 20) + 1), dict(src=None), dict(dst=None),
                                dict(src=A + 2)])
def test_kv_copy_pages_rejects(L, kw):
    assert _call(L, "rf_kv_copy_pages", COPY, dict(kw, pool=_pool())) == INV


FORK = dict(table=A, table_stride=4, len=A, B=2, src=A, n=3, out=2 * A, out_stride=4, len_out=A, refs=A,
            max_pages=4, page=16, num_pages=9, stream=None)
GROW = dict(table=A, table_stride=4, len=A, new_len=A, n=3, refs=A, max_pages=4, page=16,
            num_pages=9, copy_src=A, copy_dst=A, left=A, stream=None)
RELEASE = dict(table=A, table_stride=4, len=A, new_len=A, n=3, refs=A, max_pages=4, page=16,
               num_pages=9, stream=None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(max_pages=0), dict(page=0), dict(num_pages=0), dict(table_stride=3),
    dict(page=1 << 16, num_pages=1 << 16), dict(table=None), dict(len=None), dict(refs=None),
    dict(refs=A + 2), dict(table=A + 1),
])
@pytest.mark.parametrize("name,ok", [("rf_pages_fork", FORK), ("rf_pages_grow", GROW),
                                     ("rf_pages_release", RELEASE)])
def test_pages_calls_reject(L, name, ok, kw):
    assert _call(L, name, ok, kw) == INV


@pytest.mark.parametrize("name,ok,kw,expect", [
    ("rf_pages_fork", FORK, dict(B=-1), INV), ("rf_pages_fork", FORK, dict(src=None), INV),
    ("rf_pages_fork", FORK, dict(out=None), INV), ("rf_pages_fork", FORK, dict(out_stride=3), INV),
    ("rf_pages_fork", FORK, dict(len_out=None), INV), ("rf_pages_fork", FORK, dict(out=A), INV),
    ("rf_pages_fork", FORK, dict(out=A + 4 * 7), INV), ("rf_pages_fork", FORK, dict(out=A - 4), INV),
    ("rf_pages_grow", GROW, dict(new_len=None), INV), ("rf_pages_grow", GROW, dict(left=None), INV),
    ("rf_pages_grow", GROW, dict(copy_src=None), INV), ("rf_pages_grow", GROW, dict(n=16385), UNS),
    ("rf_pages_grow", GROW, dict(page=1, num_pages=(1 << 30) + 1), INV),
    ("rf_pages_release", RELEASE, dict(new_len=A + 2), INV),
])
def test_pages_calls_reject_more(L, name, ok, kw, expect):
    assert _call(L, name, ok, kw) == expect


@pytest.mark.parametrize("name,ok,kw", [
    ("rf_tree_mask", MASK, dict(T=0, parent=None, mask=None)), ("rf_tree_mask", MASK, dict(B=0)),
    ("rf_tree_accept", ACCEPT, dict(B=0, cu_q=None)), ("rf_attn_paged_tree", TREE, dict(T=0, tree=None)),
    ("rf_sample_rows", SAMPLE, dict(B=0, logits=None)),
    ("rf_kv_compact_paged", COMPACT, dict(B=0, table=None)),
    ("rf_kv_compact_paged", COMPACT, dict(N=0, keep=None)), ("rf_kv_copy_pages", COPY, dict(n=0, src=None)),
    ("rf_pages_fork", FORK, dict(n=0, src=None)), ("rf_pages_release", RELEASE, dict(n=0, table=None)),
])
def test_calls_of_nothing(L, name, ok, kw):
    if "pool" in ok:
        kw = dict(kw, pool=_pool())
    assert _call(L, name, ok, kw) == api.RF_OK


def test_python_refuses_host_tensors_and_causal_plans():
    build.build()
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(2, 4)
    pool = torch.zeros(1, 8, 1, 64)
    for call in [lambda: api.tree_mask(i, i, i), lambda: api.tree_accept(i, i, i, i, i),
                 lambda: api.sample_rows(f, f), lambda: api.kv_copy_pages(pool, pool, i, i),
                 lambda: api.kv_compact_paged(pool, pool, i.view(1, 2), i, i),
                 lambda: api.pages_fork(i.view(1, 2), i, i, i.view(1, 2), i, 8),
                 lambda: api.pages_grow(i.view(1, 2), i, i, i, 8),
                 lambda: api.pages_release(i.view(1, 2), i, i, 8)]:
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("kw,hkv,expect", [
    (dict(N=1 << 30), 2, api.RF_OK), (dict(N=(1 << 30) + 1), 2, INV),
    (dict(N=(1 << 28) + 1), 2, api.RF_OK), (dict(B=(1 << 20) + 1), 2, api.RF_OK),
    (dict(B=(1 << 30) - 1), 2, api.RF_OK), (dict(B=1 << 30), 2, INV),
    (dict(B=(1 << 31) - 1), 1, api.RF_OK),
])
def test_kv_compact_paged_largest_lists(L, kw, hkv, expect):
    # (without layers nothing is launched)
    pool = _pool(layers=0, Hkv=hkv)
    assert _call(L, "rf_kv_compact_paged", COMPACT, dict(kw, pool=pool)) == expect


@pytest.mark.parametrize("name,ok,nothing", [("rf_kv_compact_paged", COMPACT, dict(N=0)),
                                             ("rf_kv_copy_pages", COPY, dict(n=0))])
@pytest.mark.parametrize("pool,expect", [
    (dict(k_head_stride=0), INV), (dict(v_token_stride=0), INV), (dict(k_page_stride=0), INV),
    (dict(v_layer_stride=0), INV),                       # an expanded pool
    (dict(k_head_stride=56), INV), (dict(v_token_stride=120), INV), (dict(k_page_stride=1024), INV),
    (dict(v_layer_stride=8 * 2048), INV), (dict(k_layer_stride=128), INV),
    # a dimension of one has no stride
    (dict(layers=1, k_layer_stride=0, v_layer_stride=0), api.RF_OK),
    (dict(Hkv=1, k_head_stride=0, v_head_stride=8), api.RF_OK),
    # other orders, and room between the rows
    (dict(k_head_stride=1024, k_token_stride=64), api.RF_OK),
    (dict(k_layer_stride=64, k_head_stride=128, k_token_stride=256, k_page_stride=4096), api.RF_OK),
    (dict(k_head_stride=72, k_token_stride=144, k_page_stride=1 << 39, k_layer_stride=1 << 39,
          num_pages=1), api.RF_OK),
    (dict(num_pages=1 << 26, k_page_stride=1 << 39, k_layer_stride=(1 << 40) - 8), INV),
    (dict(num_pages=1 << 26, k_layer_stride=2048, k_page_stride=1 << 39, v_layer_stride=2048,
          v_page_stride=4096), api.RF_OK),
])
def test_pools_whose_rows_overlap(L, name, ok, nothing, pool, expect):
    assert _call(L, name, ok, dict(nothing, pool=_pool(**pool))) == expect
