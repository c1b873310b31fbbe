"""The paged-cache serving entries without a GPU: sizes, pointers, strides and
types that they refuse on the host, and calls with nothing to do."""

import math
import subprocess

import pytest

from online_softmax_attention_rf_gb300 import api, build

A = 0x10000        # an aligned fake device address; never dereferenced
MIS = 0x10008


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def _call(fn, names, defaults, kw):
    a = dict(defaults)
    assert not set(kw) - set(a), set(kw) - set(a)
    a.update(kw)
    return fn(*[a[n] for n in names])


SLOTS = ["cu_q", "kv_len", "table", "table_stride", "B", "T", "max_pages", "page", "num_pages",
         "pos", "slots", "stream"]
SLOTS_OK = dict(cu_q=A, kv_len=A, table=A, table_stride=4, B=2, T=3, max_pages=4, page=16,
                num_pages=9, pos=A, slots=A, stream=None)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(T=-1), dict(page=0), dict(num_pages=0), dict(max_pages=0),
    dict(page=1 << 16, num_pages=1 << 16), dict(page=1 << 16, max_pages=1 << 16),
    dict(B=(1 << 20) + 1), dict(T=(1 << 28) + 1), dict(table_stride=3),
    dict(cu_q=None), dict(kv_len=None), dict(table=None), dict(pos=None), dict(slots=None),
    dict(slots=A + 4), dict(pos=A + 2), dict(cu_q=A + 1),
])
def test_paged_slots_rejects(L, kw):
    assert _call(L.rf_paged_slots, SLOTS, SLOTS_OK, kw) == api.RF_ERR_INVALID
    assert L.rf_last_error().startswith(b"rf_paged_slots")


def test_paged_slots_without_rows_is_a_no_op(L):
    assert _call(L.rf_paged_slots, SLOTS, SLOTS_OK, dict(T=0, cu_q=None, pos=None)) == api.RF_OK


APPEND = ["q", "q_stride", "k", "k_stride", "v", "v_stride", "q_out", "k_cache", "kp", "kt", "kh",
          "v_cache", "vp", "vt", "vh", "T", "H", "Hkv", "d", "page", "num_pages", "slots", "pos",
          "cos_sin", "max_pos", "rot", "interleaved", "q_weight", "k_weight", "eps", "dt", "stream"]
APPEND_OK = dict(q=A, q_stride=4 * 64, k=A, k_stride=2 * 64, v=A, v_stride=2 * 64, q_out=2 * A,
                 k_cache=A, kp=16 * 128, kt=128, kh=64, v_cache=A, vp=16 * 128, vt=128, vh=64, T=3,
                 H=4, Hkv=2, d=64, page=16, num_pages=9, slots=A, pos=A, cos_sin=A, max_pos=100,
                 rot=64, interleaved=0, q_weight=A, k_weight=A, eps=1e-6, dt=api.RF_BF16,
                 stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), api.RF_ERR_INVALID), (dict(H=0), api.RF_ERR_INVALID),
    (dict(Hkv=0), api.RF_ERR_INVALID), (dict(d=0), api.RF_ERR_INVALID),
    (dict(rot=-16), api.RF_ERR_INVALID), (dict(rot=80), api.RF_ERR_INVALID),
    (dict(page=0), api.RF_ERR_INVALID), (dict(num_pages=0), api.RF_ERR_INVALID),
    (dict(page=1 << 16, num_pages=1 << 16), api.RF_ERR_INVALID),
    (dict(d=72), api.RF_ERR_UNSUPPORTED), (dict(d=272), api.RF_ERR_UNSUPPORTED),
    (dict(rot=24), api.RF_ERR_UNSUPPORTED), (dict(dt=5), api.RF_ERR_INVALID),
    (dict(interleaved=2), api.RF_ERR_INVALID), (dict(eps=-1.0), api.RF_ERR_INVALID),
    (dict(eps=math.nan), api.RF_ERR_INVALID), (dict(max_pos=0), api.RF_ERR_INVALID),
    (dict(k=None), api.RF_ERR_INVALID), (dict(v=None), api.RF_ERR_INVALID),
    (dict(k_cache=None), api.RF_ERR_INVALID), (dict(v_cache=None), api.RF_ERR_INVALID),
    (dict(q_out=None), api.RF_ERR_INVALID), (dict(slots=None), api.RF_ERR_INVALID),
    (dict(pos=None), api.RF_ERR_INVALID), (dict(cos_sin=None), api.RF_ERR_INVALID),
    (dict(q=MIS), api.RF_ERR_INVALID), (dict(k=MIS), api.RF_ERR_INVALID),
    (dict(v_cache=MIS), api.RF_ERR_INVALID), (dict(q_weight=MIS), api.RF_ERR_INVALID),
    (dict(cos_sin=MIS), api.RF_ERR_INVALID), (dict(slots=A + 4), api.RF_ERR_INVALID),
    (dict(kt=132), api.RF_ERR_INVALID), (dict(vh=-64), api.RF_ERR_INVALID),
    (dict(q_stride=3 * 64), api.RF_ERR_INVALID), (dict(k_stride=64), api.RF_ERR_INVALID),
    (dict(q_out=A, q_stride=8 * 64), api.RF_ERR_INVALID),
])
def test_kv_append_paged_rejects(L, kw, expect):
    assert _call(L.rf_kv_append_paged, APPEND, APPEND_OK, kw) == expect
    assert L.rf_last_error().startswith(b"rf_kv_append_paged")


def test_kv_append_paged_without_rows_is_a_no_op(L):
    assert _call(L.rf_kv_append_paged, APPEND, APPEND_OK, dict(T=0, k=None)) == api.RF_OK


PLAN = ["cu_q", "kv_len", "B", "T", "H", "Hkv", "page", "max_pages", "causal", "plan", "bytes",
        "stream"]


def test_paged_plan_rejects(L):
    n = L.rf_paged_plan_bytes(3)
    assert n > 0 and n % 256 == 0 and L.rf_paged_plan_bytes(-1) == 0
    ok = dict(cu_q=A, kv_len=A, B=3, T=5, H=8, Hkv=2, page=16, max_pages=4, causal=1, plan=A,
              bytes=n, stream=None)
    for kw in [dict(B=-1), dict(T=-1), dict(H=0), dict(Hkv=3), dict(Hkv=0), dict(page=0),
               dict(max_pages=0), dict(page=1 << 16, max_pages=1 << 16), dict(causal=2),
               dict(cu_q=None), dict(kv_len=None), dict(plan=None), dict(plan=A + 128),
               dict(cu_q=A + 2), dict(bytes=n - 1)]:
        assert _call(L.rf_paged_plan, PLAN, ok, kw) == api.RF_ERR_INVALID, kw
        assert L.rf_last_error().startswith(b"rf_paged_plan")
    assert _call(L.rf_paged_plan, PLAN, ok, dict(H=258, Hkv=2)) == api.RF_ERR_UNSUPPORTED


def test_plan_steps_up_to_the_longest_cache(tmp_path):
    # the plan's arithmetic over lengths, compiled for the host: caches of up to
    # 2^31 - 1 tokens
    (tmp_path / "steps.cpp").write_text("""
#include <cstddef>
#define __host__
#define __device__
#include "paged_plan.h"
#include <cstdio>
#include <initializer_list>
int main() {
  for (long long keys : {0LL, 1LL, 127LL, 128LL, 129LL, 2147483519LL, 2147483520LL, 2147483521LL,
                         2147483640LL, 2147483647LL}) {
    const int kv = static_cast<int>(keys);
    std::printf("%lld %d %d %d\\n", keys, rf::plan_steps(kv), rf::plan_visible(0, 1, kv, 1),
                rf::plan_visible(2, 3, kv, 0));
  }
}
""")
    exe = str(tmp_path / "steps")
    subprocess.run(["g++", "-std=c++17", "-ftrapv", "-I", build.CSRC, str(tmp_path / "steps.cpp"),
                    "-o", exe], check=True)
    rows = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    rows = [[int(x) for x in r.split()] for r in rows if r]
    assert len(rows) == 10
    for keys, steps, last, every in rows:
        assert steps == -(-keys // 128) and last == every == keys


ATTN = ["q", "q_stride", "k", "kp", "kt", "kh", "v", "vp", "vt", "vh", "page", "num_pages", "table",
        "table_stride", "max_pages", "plan", "B", "T", "H", "Hkv", "d", "scale", "o", "lse", "ws",
        "ws_bytes", "dt", "stream"]


def _attn_ok(L):
    return dict(q=A, q_stride=8 * 128, k=A, kp=16 * 256, kt=256, kh=128, v=A, vp=16 * 256, vt=256,
                vh=128, page=16, num_pages=9, table=A, table_stride=4, max_pages=4, plan=A, B=3,
                T=5, H=8, Hkv=2, d=128, scale=0.1, o=A, lse=A, ws=A,
                ws_bytes=L.rf_attn_paged_workspace_bytes(128), dt=api.RF_BF16, stream=None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), api.RF_ERR_INVALID), (dict(T=-1), api.RF_ERR_INVALID),
    (dict(Hkv=3), api.RF_ERR_INVALID), (dict(H=512), api.RF_ERR_UNSUPPORTED),
    (dict(d=96), api.RF_ERR_UNSUPPORTED), (dict(dt=api.RF_F32), api.RF_ERR_UNSUPPORTED),
    (dict(dt=9), api.RF_ERR_INVALID), (dict(page=12), api.RF_ERR_UNSUPPORTED),
    (dict(page=1), api.RF_ERR_UNSUPPORTED), (dict(scale=0.0), api.RF_ERR_INVALID),
    (dict(scale=math.inf), api.RF_ERR_INVALID), (dict(scale=math.nan), api.RF_ERR_INVALID),
    (dict(q=None), api.RF_ERR_INVALID), (dict(k=None), api.RF_ERR_INVALID),
    (dict(table=None), api.RF_ERR_INVALID), (dict(plan=None), api.RF_ERR_INVALID),
    (dict(o=None), api.RF_ERR_INVALID), (dict(ws=None), api.RF_ERR_INVALID),
    (dict(q=MIS), api.RF_ERR_INVALID), (dict(v=MIS), api.RF_ERR_INVALID),
    (dict(lse=A + 2), api.RF_ERR_INVALID), (dict(ws=A + 16), api.RF_ERR_INVALID),
    (dict(q_stride=8 * 128 - 8), api.RF_ERR_INVALID), (dict(kt=260), api.RF_ERR_INVALID),
    (dict(vh=0), api.RF_ERR_INVALID), (dict(table_stride=3), api.RF_ERR_INVALID),
    (dict(ws_bytes=1024), api.RF_ERR_INVALID), (dict(kp=1 << 38), api.RF_ERR_INVALID),
])
def test_attn_paged_rejects(L, kw, expect):
    assert _call(L.rf_attn_paged, ATTN, _attn_ok(L), kw) == expect
    assert L.rf_last_error().startswith(b"rf_attn_paged")


def test_attn_paged_without_rows_is_a_no_op(L):
    assert _call(L.rf_attn_paged, ATTN, _attn_ok(L), dict(T=0, q=None, o=None)) == api.RF_OK
    assert _call(L.rf_attn_paged, ATTN, _attn_ok(L), dict(B=0, table=None)) == api.RF_OK
    assert L.rf_attn_paged_workspace_bytes(96) == 0


VERIFY = ["target", "draft", "tokens", "u", "expo", "n_draft", "temperature", "B", "S", "V", "out",
          "n_accepted", "ws", "ws_bytes", "dt", "stream"]


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), api.RF_ERR_INVALID), (dict(S=0), api.RF_ERR_INVALID),
    (dict(S=65), api.RF_ERR_UNSUPPORTED), (dict(V=0), api.RF_ERR_INVALID),
    (dict(V=(1 << 30) + 1), api.RF_ERR_INVALID), (dict(B=(1 << 20) + 1), api.RF_ERR_INVALID),
    (dict(dt=3), api.RF_ERR_INVALID), (dict(target=None), api.RF_ERR_INVALID),
    (dict(tokens=None), api.RF_ERR_INVALID), (dict(u=None), api.RF_ERR_INVALID),
    (dict(expo=None), api.RF_ERR_INVALID), (dict(out=None), api.RF_ERR_INVALID),
    (dict(n_accepted=None), api.RF_ERR_INVALID), (dict(ws=None), api.RF_ERR_INVALID),
    (dict(ws=MIS), api.RF_ERR_INVALID), (dict(ws_bytes=16), api.RF_ERR_INVALID),
    (dict(target=A + 1), api.RF_ERR_INVALID), (dict(u=A + 2), api.RF_ERR_INVALID),
    (dict(target=A + 2, dt=api.RF_F32), api.RF_ERR_INVALID),
])
def test_draft_verify_rejects(L, kw, expect):
    ok = dict(target=A, draft=A, tokens=A, u=A, expo=A, n_draft=None, temperature=None, B=2, S=4,
              V=100, out=A, n_accepted=A, ws=A, ws_bytes=L.rf_draft_verify_workspace_bytes(2, 4),
              dt=api.RF_BF16, stream=None)
    assert _call(L.rf_draft_verify, VERIFY, ok, kw) == expect
    assert L.rf_last_error().startswith(b"rf_draft_verify")
    assert _call(L.rf_draft_verify, VERIFY, ok, dict(B=0, target=None)) == api.RF_OK
    assert L.rf_draft_verify_workspace_bytes(0, 4) == 0
    assert L.rf_draft_verify_workspace_bytes(2, 65) == 0
