"""Cases and plain forms of the paged-cache serving operators.

One step of speculative decoding over a paged key/value cache:

* ``append``: queries and keys normalised per head and rotated by position,
  keys and values written into their pages (``api.kv_append_paged``);
* ``attn``: attention of each sequence's new tokens (one token, a few drafted
  ones, or a long chunk) over its paged cache (``api.attn_paged``);
* ``verify``: the drafted tokens judged against the target's probabilities
  from given random numbers (``api.draft_verify``).

``run`` computes a pass in plain torch operations, or, where ``own`` is true,
through the package's public calls.
"""

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user, one new token, a short cache: latency of a decode step
        dict(name="attn_decode_one", op="attn", H=32, Hkv=8, d=128, page=16, head_major=False,
             B=1, q_min=1, q_max=1, kv_min=515, kv_max=515, lens=0),
        # a serving batch of one new token each, lengths from a few to many thousands
        dict(name="attn_decode_batch", op="attn", H=32, Hkv=8, d=128, page=16, head_major=False,
             B=64, q_min=1, q_max=1, kv_min=9, kv_max=16384, lens=1),
        # four drafted tokens and the last accepted one, long caches
        dict(name="attn_verify_batch", op="attn", H=64, Hkv=8, d=128, page=64, head_major=False,
             B=16, q_min=5, q_max=5, kv_min=1024, kv_max=32768, lens=2),
        # chunked prefill at the end of a long prompt
        dict(name="attn_chunk_long", op="attn", H=64, Hkv=8, d=128, page=128, head_major=False,
             B=1, q_min=2048, q_max=2048, kv_min=32768, kv_max=32768, lens=3),
        # several prompts' chunks of odd lengths, 7 query heads a key head, head-major pages
        dict(name="attn_chunk_ragged", op="attn", H=28, Hkv=4, d=128, page=32, head_major=True,
             B=6, q_min=100, q_max=1000, kv_min=1000, kv_max=8192, lens=4),
        # a mixed batch (chunks between single tokens), small heads, one key head per query head
        dict(name="attn_mixed_d64", op="attn", H=16, Hkv=16, d=64, page=16, head_major=False,
             B=24, q_min=1, q_max=700, kv_min=700, kv_max=4096, lens=5),
        # one token for each of 32 users: latency of the write before a decode step
        dict(name="append_decode", op="append", H=32, Hkv=8, d=128, rot=128, page=16,
             head_major=False, T=32, norm=True, interleaved=False, dtype="bf16"),
        # a long chunk out of a fused projection
        dict(name="append_chunk", op="append", H=64, Hkv=8, d=128, rot=128, page=64,
             head_major=False, T=8192, norm=True, interleaved=False, dtype="bf16"),
        # float32, neighbouring pairs, half of the head rotated, no norm, head-major pages
        dict(name="append_f32_d64", op="append", H=16, Hkv=16, d=64, rot=32, page=32,
             head_major=True, T=1001, norm=False, interleaved=True, dtype="f32"),
        # one user, four drafted tokens: latency of a verification
        dict(name="verify_one", op="verify", B=1, S=4, V=32000, dtype="f32", drafts="logits",
             ragged=False, greedy=False),
        # a serving batch, large vocabulary
        dict(name="verify_batch", op="verify", B=64, S=4, V=131072, dtype="bf16", drafts="logits",
             ragged=False, greedy=False),
        # drafts copied from the prompt (no draft probabilities), of different lengths,
        # some users decoding greedily, a vocabulary of odd size
        dict(name="verify_copied", op="verify", B=16, S=7, V=50001, dtype="f32", drafts="fixed",
             ragged=True, greedy=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _seconds(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.8e15)


def _largest():
    return max(_seconds(c) for c in listed())


def draw(rng):
    """One more case: sizes spread over the listed cases' ranges."""
    op = rng.choice(["attn", "attn", "append", "verify"])
    limit = _largest()
    while True:
        if op == "attn":
            H, Hkv = rng.choice([(32, 8), (64, 8), (28, 4), (16, 16), (8, 1), (12, 4), (8, 8)])
            q_max = rng.choice([1, _log_int(rng, 2, 16), _log_int(rng, 17, 2048)])
            kv_max = _log_int(rng, max(q_max, 100), 32768)
            case = dict(op=op, H=H, Hkv=Hkv, d=rng.choice([64, 128]),
                        page=rng.choice([16, 32, 48, 64, 128, 256]),
                        head_major=rng.random() < 0.3, B=_log_int(rng, 1, 64),
                        q_min=rng.choice([1, q_max]), q_max=q_max,
                        kv_min=rng.randint(q_max, kv_max), kv_max=kv_max,
                        lens=rng.randrange(1 << 30))
        elif op == "append":
            d = rng.choice([64, 128])
            H, Hkv = rng.choice([(32, 8), (64, 8), (28, 4), (16, 16), (8, 1)])
            case = dict(op=op, H=H, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2]),
                        page=rng.choice([16, 32, 48, 64, 128]), head_major=rng.random() < 0.3,
                        T=_log_int(rng, 1, 8192), norm=rng.random() < 0.6,
                        interleaved=rng.random() < 0.3, dtype=rng.choice(["bf16", "bf16", "f32"]))
        else:
            case = dict(op=op, B=_log_int(rng, 1, 64), S=rng.randint(1, 8),
                        V=_log_int(rng, 1000, 131072), dtype=rng.choice(["bf16", "f32"]),
                        drafts=rng.choice(["logits", "logits", "fixed"]),
                        ragged=rng.random() < 0.5, greedy=rng.random() < 0.3)
        if _seconds(case) <= limit:
            return case


def _lengths(case):
    """New tokens and cache lengths (the new tokens among them) of an attention case."""
    rng = random.Random(case["lens"])
    nq = [rng.randint(case["q_min"], case["q_max"]) for _ in range(case["B"])]
    if case["q_min"] == 1 and case["q_max"] > 16:  # most users decode, some prefill
        nq = [n if i % 4 == 0 else 1 for i, n in enumerate(nq)]
    kv = [rng.randint(max(case["kv_min"], n), max(case["kv_max"], n)) for n in nq]
    return nq, kv


def work(case):
    op = case["op"]
    if op == "attn":
        nq, kv = _lengths(case)
        T, H, Hkv, d = sum(nq), case["H"], case["Hkv"], case["d"]
        pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(nq, kv))
        table = sum(-(-m // case["page"]) for m in kv) * 4
        return {"bytes": 2 * T * H * d * 2 + 4 * T * H + 2 * sum(kv) * Hkv * d * 2 + table,
                "flops": 4 * d * H * pairs}
    if op == "append":
        T, H, Hkv, d, e = case["T"], case["H"], case["Hkv"], case["d"], _BYTES[case["dtype"]]
        per_token = 2 * (H + 2 * Hkv) * d * e + case["rot"] * 4 + 12
        weights = 2 * d * e if case["norm"] else 0
        return {"bytes": T * per_token + weights,
                "flops": T * (H + Hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    B, S, V, e = case["B"], case["S"], case["V"], _BYTES[case["dtype"]]
    rows = (2 * S + 1) if case["drafts"] == "logits" else S + 1
    # every logit: a running maximum and a sum of exponentials; one row more for the choice
    return {"bytes": B * (rows * V * e + 4 * V + 12 * S + 8), "flops": B * V * (4 * rows + 6)}


# ------------------------------------------------------------------ inputs

def _pages(needed, device, g):
    """Block table rows (python lists) over a shuffled pool with a few spare pages."""
    total = sum(needed) + 8
    perm = torch.randperm(total, generator=g, device=device).tolist()
    rows, at = [], 0
    for n in needed:
        rows.append(perm[at:at + n])
        at += n
    return rows, total


def _cache(num_pages, page, Hkv, d, dtype, head_major, device, g):
    """A [num_pages, page, Hkv, d] cache, stored page- or head-major inside a page."""
    shape = (num_pages, Hkv, page, d) if head_major else (num_pages, page, Hkv, d)
    c = torch.randn(shape, generator=g, device=device, dtype=torch.float32).to(dtype)
    return c.permute(0, 2, 1, 3) if head_major else c


def prepare(case, seed):
    device = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=device).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "attn":
        _prepare_attn(case, st, device, g)
    elif case["op"] == "append":
        _prepare_append(case, st, device, g)
    else:
        _prepare_verify(case, st, device, g)
    return st


def _prepare_attn(case, st, device, g):
    nq, kv = _lengths(case)
    B, H, Hkv, d, page = case["B"], case["H"], case["Hkv"], case["d"], case["page"]
    T = sum(nq)
    needed = [-(-m // page) for m in kv]
    rows, total = _pages(needed, device, g)
    width = max(needed)
    st["table"] = torch.tensor([r + [0] * (width - len(r)) for r in rows], dtype=torch.int32,
                               device=device)
    st["k_cache"] = _cache(total, page, Hkv, d, torch.bfloat16, case["head_major"], device, g)
    st["v_cache"] = _cache(total, page, Hkv, d, torch.bfloat16, case["head_major"], device, g)
    st["q"] = torch.randn(T, H, d, generator=g, device=device).to(torch.bfloat16)
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    st["nq"], st["kv"], st["cu"] = nq, kv, cu
    st["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=device)
    st["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=device)
    st["scale"] = 1.0 / math.sqrt(d)
    if own:
        from online_softmax_attention_rf_gb300 import api
        # made once a step, used by every layer
        st["plan"] = api.PagedPlan(st["cu_q"], st["kv_len"], T, H, Hkv, page, width)
        st["ws"] = api.attn_paged_workspace(d, device)


def _prepare_append(case, st, device, g):
    T, H, Hkv, d, page = case["T"], case["H"], case["Hkv"], case["d"], case["page"]
    dt = _DT[case["dtype"]]
    # a step's tokens come out of one fused projection: q, k and v are views of it
    qkv = torch.randn(T, H + 2 * Hkv, d, generator=g, device=device).to(dt)
    st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    num_pages = -(-T // page) + 8
    st["k_cache"] = _cache(num_pages, page, Hkv, d, dt, case["head_major"], device, g)
    st["v_cache"] = _cache(num_pages, page, Hkv, d, dt, case["head_major"], device, g)
    # each token its own slot; runs of a page stay together, as a chunk's do
    first = torch.randperm(num_pages, generator=g, device=device)[:-(-T // page)]
    slots = (first[:, None] * page + torch.arange(page, device=device)[None, :]).reshape(-1)[:T]
    st["slots"] = slots.contiguous()
    max_pos = 65536
    st["pos"] = torch.randint(0, max_pos, (T,), generator=g, device=device, dtype=torch.int32)
    half = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    ang = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq[None, :]
    st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    st["eps"] = 1e-6
    st["qw"] = st["kw"] = None
    if case["norm"]:
        st["qw"] = (1 + 0.1 * torch.randn(d, generator=g, device=device)).to(dt)
        st["kw"] = (1 + 0.1 * torch.randn(d, generator=g, device=device)).to(dt)


def _prepare_verify(case, st, device, g):
    B, S, V = case["B"], case["S"], case["V"]
    dt = _DT[case["dtype"]]
    shared = 2.5 * torch.randn(B, S + 1, V, generator=g, device=device)
    st["target"] = (shared + 0.5 * torch.randn(B, S + 1, V, generator=g, device=device)).to(dt)
    temp = 0.6 + 0.6 * torch.rand(B, generator=g, device=device)
    if case["greedy"]:
        temp = torch.where(torch.arange(B, device=device) % 3 == 1, torch.zeros_like(temp), temp)
    st["temp"] = temp
    t = torch.where(temp > 0, temp, torch.ones_like(temp))[:, None, None]
    noise = torch.empty(B, S, V, device=device).exponential_(generator=g)
    if case["drafts"] == "logits":
        st["draft"] = (shared[:, :S] + 0.5 * torch.randn(B, S, V, generator=g,
                                                         device=device)).to(dt)
        drawn = torch.argmax(torch.softmax(st["draft"].float() / t, -1) / noise, -1)
        best = torch.argmax(st["draft"].float(), -1)
    else:
        st["draft"] = None
        drawn = torch.argmax(torch.softmax(st["target"][:, :S].float() / t, -1) / noise, -1)
        best = torch.argmax(st["target"][:, :S].float(), -1)
    pick = torch.rand(B, S, generator=g, device=device) < 0.5
    st["tokens"] = torch.where(pick, best, drawn).to(torch.int32)
    st["u"] = torch.rand(B, S, generator=g, device=device)
    st["expo"] = torch.empty(B, V, device=device).exponential_(generator=g).clamp_min_(1e-20)
    st["n_draft"] = None
    if case["ragged"]:
        st["n_draft"] = torch.randint(0, S + 1, (B,), generator=g, device=device,
                                      dtype=torch.int32)
    if own:
        from online_softmax_attention_rf_gb300 import api
        st["ws"] = api.draft_verify_workspace(B, S, device)


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _own(op, st)
    if op == "attn":
        return _plain_attn(st)
    if op == "append":
        return _plain_append(st)
    return _plain_verify(st)


def _own(op, st):
    from online_softmax_attention_rf_gb300 import api
    if op == "attn":
        return api.attn_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["plan"],
                              scale=st["scale"], workspace=st["ws"])
    if op == "append":
        q_out = api.kv_append_paged(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                                    st["slots"], pos=st["pos"], cos_sin=st["cos_sin"],
                                    q_weight=st["qw"], k_weight=st["kw"], eps=st["eps"],
                                    interleaved=st["case"]["interleaved"])
        return q_out, st["k_cache"], st["v_cache"]
    return api.draft_verify(st["target"], st["draft"], st["tokens"], st["u"], st["expo"],
                            n_draft=st["n_draft"], temperature=st["temp"], workspace=st["ws"])


def _plain_attn(st):
    case, q = st["case"], st["q"]
    T, H, d = q.shape
    Hkv, page = case["Hkv"], case["page"]
    G = H // Hkv
    o = torch.empty_like(q)
    lse = torch.empty(T, H, dtype=torch.float32, device=q.device)
    for b in range(case["B"]):
        n, m, t0 = st["nq"][b], st["kv"][b], st["cu"][b]
        pages = st["table"][b, :-(-m // page)].long()
        k = st["k_cache"][pages].reshape(-1, Hkv, d)[:m].float()
        v = st["v_cache"][pages].reshape(-1, Hkv, d)[:m].float()
        step = max(1, (1 << 28) // (G * m))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            qb = q[t0 + i0:t0 + i1].float().view(i1 - i0, Hkv, G, d)
            hidden = torch.arange(m, device=q.device)[None, :] > \
                torch.arange(m - n + i0, m - n + i1, device=q.device)[:, None]
            for h in range(Hkv):
                s = torch.matmul(qb[:, h], k[:, h].t()) * st["scale"]  # [tokens, G, m]
                s = torch.where(hidden[:, None, :], float("-inf"), s)
                mx = s.max(-1, keepdim=True).values
                p = torch.exp(s - mx)
                l = p.sum(-1, keepdim=True)
                o[t0 + i0:t0 + i1, h * G:(h + 1) * G] = (torch.matmul(p, v[:, h]) / l).to(q.dtype)
                lse[t0 + i0:t0 + i1, h * G:(h + 1) * G] = (mx + torch.log(l))[..., 0]
    return o, lse


def _plain_norm_rotate(x, w, eps, cos, sin, interleaved):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    half = cos.shape[-1]
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        head = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        head = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([head, x[..., 2 * half:]], -1)


def _plain_append(st):
    case, page = st["case"], st["case"]["page"]
    rows = st["cos_sin"][st["pos"].long()]
    cos, sin = rows.chunk(2, -1)
    q = _plain_norm_rotate(st["q"], st["qw"], st["eps"], cos, sin, case["interleaved"])
    k = _plain_norm_rotate(st["k"], st["kw"], st["eps"], cos, sin, case["interleaved"])
    dt = st["q"].dtype
    at = st["slots"] // page, st["slots"] % page
    st["k_cache"][at] = k.to(dt)
    st["v_cache"][at] = st["v"]
    return q.to(dt), st["k_cache"], st["v_cache"]


def _plain_verify(st):
    # 64 bits: a value next to a border decides a whole number
    target, draft, tokens = st["target"], st["draft"], st["tokens"].long()
    B, S1, V = target.shape
    S = S1 - 1
    dev = target.device
    out = torch.full((B, S1), -1, dtype=torch.int32, device=dev)
    n_acc = torch.zeros(B, dtype=torch.int32, device=dev)
    n_draft = st["n_draft"] if st["n_draft"] is not None else \
        torch.full((B,), S, dtype=torch.int32, device=dev)
    greedy = st["temp"] == 0
    t = torch.where(greedy, 1.0, st["temp"].double())
    x = torch.arange(V, device=dev)

    def softmax(row):
        z = row.double() / t[:, None]
        e = torch.exp(z - z.max(-1, keepdim=True).values)
        return e / e.sum(-1, keepdim=True)

    alive = torch.ones(B, dtype=torch.bool, device=dev)
    for i in range(S1):
        p = softmax(target[:, i])
        best = target[:, i].double().max(-1, keepdim=True).values == target[:, i].double()
        best = torch.where(best, x, V).min(-1).values
        p = torch.where(greedy[:, None], (x[None] == best[:, None]).double(), p)
        weights = p
        accept = torch.zeros_like(alive)
        if i < S:
            tok = tokens[:, i]
            px = p.gather(1, tok[:, None])[:, 0]
            if draft is not None:
                q = softmax(draft[:, i])
                qx = q.gather(1, tok[:, None])[:, 0]
            else:
                q = (x[None] == tok[:, None]).double()
                qx = torch.ones_like(px)
            drafted = i < n_draft
            accept = torch.where(greedy, px > 0, st["u"][:, i].double() * qx < px) & drafted
            rest = torch.clamp(p - q, min=0)
            usable = (rest.sum(-1) > 0) & drafted & ~greedy
            weights = torch.where(usable[:, None], rest, p)
        score = weights / st["expo"].double()
        chosen = torch.where(score == score.max(-1, keepdim=True).values, x, V).min(-1).values
        stop = alive & ~accept
        if i < S:
            out[:, i] = torch.where(alive & accept, tok.to(torch.int32), out[:, i])
        out[:, i] = torch.where(stop, chosen.to(torch.int32), out[:, i])
        n_acc += (alive & accept).to(torch.int32)
        alive = alive & accept
    return out, n_acc


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(st)
    if case["op"] == "append":
        return _exact_append(st)
    return _exact_verify(st)


def _exact_attn(st):
    case, q = st["case"], st["q"]
    if work(case)["flops"] > 6e12:
        return None
    T, H, d = q.shape
    o = torch.empty(T, H, d, dtype=torch.float64, device=q.device)
    lse = torch.empty(T, H, dtype=torch.float64, device=q.device)
    group = H // case["Hkv"]
    for b, (n, m) in enumerate(zip(st["nq"], st["kv"])):
        j = torch.arange(m, device=q.device)
        page = st["table"][b].long()[j // case["page"]]
        for h in range(H):
            k = st["k_cache"][page, j % case["page"], h // group].double()
            v = st["v_cache"][page, j % case["page"], h // group].double()
            rows = slice(st["cu"][b], st["cu"][b] + n)
            z = st["scale"] * (q[rows, h].double() @ k.T)
            last = m - n + torch.arange(n, device=q.device)
            z.masked_fill_(j[None] > last[:, None], float("-inf"))
            lse[rows, h] = torch.logsumexp(z, 1)
            o[rows, h] = torch.exp(z - lse[rows, h][:, None]) @ v
    return o, lse


def _exact_append(st):
    case = st["case"]
    rot, d = case["rot"], case["d"]
    i = torch.arange(rot // 2, device=st["q"].device)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    row = st["cos_sin"].double()[st["pos"].long()]

    def turned(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + st["eps"]) * w.double()
        z = torch.complex(y[..., first], y[..., second])
        z = z * torch.complex(row[:, : rot // 2], row[:, rot // 2:])[:, None]
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    page, off = st["slots"].div(case["page"], rounding_mode="floor"), st["slots"] % case["page"]
    k_cache[page, off] = turned(st["k"], st["kw"])
    v_cache[page, off] = st["v"].double()
    return turned(st["q"], st["qw"]), k_cache, v_cache


def _exact_verify(st):
    target, draft = st["target"], st["draft"]
    B, S = target.shape[0], target.shape[1] - 1
    out = torch.full((B, S + 1), -1, dtype=torch.int32)
    n_acc = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        temp = float(st["temp"][b])
        drafted = S if st["n_draft"] is None else int(st["n_draft"][b])
        tokens, u = st["tokens"][b].tolist(), st["u"][b].double().tolist()
        at = 0
        while True:
            z = target[b, at].double()
            if temp == 0:
                choice = int((z == z.max()).nonzero()[0, 0])
                accepted = at < drafted and tokens[at] == choice
            else:
                z = z / temp
                p = torch.exp(z - torch.logsumexp(z, 0))
                accepted, rest = False, p
                if at < drafted:
                    if draft is None:
                        q = torch.zeros_like(p)
                        q[tokens[at]] = 1
                    else:
                        y = draft[b, at].double() / temp
                        q = torch.exp(y - torch.logsumexp(y, 0))
                    accepted = u[at] * float(q[tokens[at]]) < float(p[tokens[at]])
                    if bool((p > q).any()):
                        rest = torch.where(p > q, p - q, torch.zeros_like(p))
                if not accepted:
                    race = rest / st["expo"][b].double()
                    choice = int((race == race.max()).nonzero()[0, 0])
            if not accepted:
                out[b, at] = choice
                n_acc[b] = at
                break
            out[b, at] = tokens[at]
            at += 1
    return out.to(target.device), n_acc.to(target.device)
