"""Cases and plain forms of the operators around a tree of drafted tokens.

A step of speculative decoding with a tree of drafts over a paged key/value
cache, and what a serving loop does to the cache between steps:

* ``attn``: attention of each sequence's drafted nodes, a node seeing the cached
  context and its own ancestors (``api.attn_paged`` with a tree mask);
* ``sample``: a token drawn from each row of logits by temperature, top-k, top-p
  and min-p, from given random numbers (``api.sample_rows``);
* ``commit``: the walk down the tree along the drawn tokens, and the accepted
  nodes' cache rows moved together (``api.tree_accept``, ``api.kv_compact_paged``);
* ``evict``: the kept tokens of a long cache moved together
  (``api.kv_compact_paged``);
* ``fork``: sequences forked by sharing pages, given pages to write to, the pages
  that are written to by one of several owners copied, and freed again
  (``api.pages_fork``, ``api.pages_grow``, ``api.kv_copy_pages``,
  ``api.pages_release``).

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
        # one user, a small tree, a short cache: latency of a verification step
        dict(name="tree_one", op="attn", H=32, Hkv=8, d=128, page=16, head_major=False, B=1,
             n_min=25, n_max=25, kv_min=1030, kv_max=1030, words=1, lens=0),
        # a serving batch of full one-word trees over long caches
        dict(name="tree_batch", op="attn", H=64, Hkv=8, d=128, page=64, head_major=False, B=16,
             n_min=64, n_max=64, kv_min=16384, kv_max=32768, words=1, lens=1),
        # trees of all sizes up to four words, odd group, head-major pages, small heads
        dict(name="tree_ragged_d64", op="attn", H=28, Hkv=4, d=64, page=32, head_major=True, B=24,
             n_min=1, n_max=200, kv_min=700, kv_max=8192, words=4, lens=2),
        # one user's next token: latency
        dict(name="sample_one", op="sample", B=1, V=32000, dtype="f32", mix="all"),
        # the nodes of a few users' trees, each user with limits of their own
        dict(name="sample_batch", op="sample", B=64, V=131072, dtype="bf16", mix="each"),
        # a batch with top-p alone, a vocabulary of odd size
        dict(name="sample_top_p", op="sample", B=200, V=50001, dtype="f32", mix="top_p"),
        # the nodes of many trees in one call
        dict(name="sample_many", op="sample", B=512, V=131072, dtype="f32", mix="each"),
        # one user: latency of the walk and of the move in all layers
        dict(name="commit_one", op="commit", B=1, n_min=32, n_max=32, ctx_max=1000, L=16, page=16,
             Hkv=8, d=128, head_major=False, dtype="bf16", lens=3),
        # a serving batch in all layers, trees of all sizes
        dict(name="commit_batch", op="commit", B=64, n_min=1, n_max=64, ctx_max=150, L=16, page=16,
             Hkv=8, d=128, head_major=False, dtype="bf16", lens=4),
        # half of long caches dropped, all layers
        dict(name="evict_half", op="evict", B=8, kv_min=2000, kv_max=8000, share=0.5, L=4, page=64,
             Hkv=8, d=128, head_major=False, dtype="bf16", lens=5),
        # one prompt, four answers
        dict(name="fork_one", op="fork", B=1, width=4, len_min=500, len_max=500, grow=1, P=1024,
             L=8, page=16, Hkv=8, d=128, head_major=False, dtype="bf16", lens=6),
        # a batch of prompts with several answers each, most of the pool in use
        dict(name="fork_batch", op="fork", B=48, width=4, len_min=1, len_max=1200, grow=40, P=4096,
             L=4, page=32, Hkv=8, d=128, head_major=False, dtype="bf16", lens=7),
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
    op = rng.choice(["attn", "sample", "sample", "commit", "evict", "fork"])
    limit = _largest()
    while True:
        lens = rng.randrange(1 << 30)
        Hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        page, hm = rng.choice([16, 32, 64]), rng.random() < 0.3
        if op == "attn":
            words = rng.choice([1, 1, 2, 4])
            n_max = _log_int(rng, 1, 64 * words)
            kv_max = _log_int(rng, n_max + 1, 32768)
            case = dict(op=op, H=Hkv * rng.choice([1, 4, 7, 8]), Hkv=Hkv, d=d, page=page,
                        head_major=hm, B=_log_int(rng, 1, 32), n_min=rng.choice([1, n_max]),
                        n_max=n_max, kv_min=rng.randint(n_max, kv_max), kv_max=kv_max,
                        words=words, lens=lens)
            size = case["B"] * case["H"] * n_max * kv_max
        elif op == "sample":
            case = dict(op=op, B=_log_int(rng, 1, 512), V=_log_int(rng, 1000, 131072),
                        dtype=rng.choice(["bf16", "f32"]),
                        mix=rng.choice(["all", "each", "top_k", "top_p", "min_p", "plain"]))
            size = 0
        elif op == "commit":
            n_max = _log_int(rng, 1, 200)
            case = dict(op=op, B=_log_int(rng, 1, 64), n_min=rng.choice([1, n_max]), n_max=n_max,
                        ctx_max=_log_int(rng, 1, 1000), L=_log_int(rng, 1, 16), page=page, Hkv=Hkv,
                        d=d, head_major=hm, dtype=rng.choice(["bf16", "bf16", "f32"]), lens=lens)
            size = 8 * case["B"] * (case["ctx_max"] + n_max) * case["L"] * Hkv * d
        elif op == "evict":
            kv_max = _log_int(rng, 100, 8000)
            case = dict(op=op, B=_log_int(rng, 1, 16), kv_min=rng.randint(1, kv_max),
                        kv_max=kv_max, share=round(rng.uniform(0.05, 0.95), 2),
                        L=_log_int(rng, 1, 8), page=page, Hkv=Hkv, d=d, head_major=hm,
                        dtype=rng.choice(["bf16", "bf16", "f32"]), lens=lens)
            size = 8 * case["B"] * kv_max * case["L"] * Hkv * d
        else:
            case = dict(op=op, B=_log_int(rng, 1, 48), width=rng.randint(1, 6), len_min=1,
                        len_max=_log_int(rng, 1, 1200), grow=rng.randint(0, 60), P=4096,
                        L=_log_int(rng, 1, 4), page=rng.choice([16, 32]), Hkv=Hkv, d=d,
                        head_major=hm, dtype=rng.choice(["bf16", "bf16", "f32"]), lens=lens)
            room = case["B"] * (_cdiv(case["len_max"], case["page"]) +
                                case["width"] * (2 + _cdiv(case["grow"], case["page"])))
            size = 0 if room <= case["P"] else 1 << 62
        if size <= 1 << 31 and _seconds(case) <= limit:
            return case


def _cdiv(a, b):
    return -(-a // b)


def _nodes(case):
    """Drafted nodes and cache lengths (the nodes among them) of an attention case."""
    rng = random.Random(case["lens"])
    n = [rng.randint(case["n_min"], case["n_max"]) for _ in range(case["B"])]
    return n, [rng.randint(max(case["kv_min"], x), max(case["kv_max"], x)) for x in n]


def _contexts(case):
    """Drafted nodes and context lengths of a commit."""
    rng = random.Random(case["lens"])
    n = [rng.randint(case["n_min"], case["n_max"]) for _ in range(case["B"])]
    return n, [rng.randint(0, case["ctx_max"]) for _ in n]


def _kept(case):
    """Cached and kept tokens of an eviction."""
    rng = random.Random(case["lens"])
    kv = [rng.randint(case["kv_min"], case["kv_max"]) for _ in range(case["B"])]
    return kv, [int(case["share"] * m) for m in kv]


def _prompts(case):
    """Cached tokens of a fork's prompts."""
    rng = random.Random(case["lens"])
    return [rng.randint(case["len_min"], case["len_max"]) for _ in range(case["B"])]


def work(case):
    op = case["op"]
    if op == "attn":
        n, kv = _nodes(case)
        T, H, Hkv, d = sum(n), case["H"], case["Hkv"], case["d"]
        # a node sees the context, itself and, below the root, the root
        pairs = sum(a * (m - a) + 2 * a - 1 for a, m in zip(n, kv))
        table = sum(_cdiv(m, case["page"]) for m in kv) * 4
        return {"bytes": 4 * T * H * d + 4 * T * H + 4 * sum(kv) * Hkv * d + table +
                T * case["words"] * 8, "flops": 4 * d * H * pairs}
    if op == "sample":
        B, V = case["B"], case["V"]
        # every logit once, a running maximum and a sum of exponentials; the draw
        # needs every random number only where nothing is cut off
        every = V * 4 if case["mix"] == "plain" else 0
        return {"bytes": B * (V * _BYTES[case["dtype"]] + every + 24), "flops": 4 * B * V}
    row = 2 * case["Hkv"] * case["d"] * _BYTES[case["dtype"]] * case["L"]  # a token's k and v
    if op == "commit":
        n, _ = _contexts(case)
        # the tree's numbers, and at least a row for each accepted node but the first
        return {"bytes": 20 * sum(n) + 24 * len(n) + 2 * row * sum(x > 2 for x in n),
                "flops": 2 * sum(n)}
    if op == "evict":
        kv, kept = _kept(case)
        return {"bytes": 2 * row * sum(kept) + 4 * sum(kept) +
                4 * sum(_cdiv(m, case["page"]) for m in kv), "flops": 0}
    lens, page = _prompts(case), case["page"]
    pages = case["width"] * sum(_cdiv(m, page) for m in lens)
    new = case["width"] * sum(_cdiv(m + case["grow"], page) - _cdiv(m, page) for m in lens)
    copies = case["width"] * sum(m % page > 0 for m in lens) if case["grow"] > 0 else 0
    return {"bytes": 4 * case["P"] + 20 * pages + 16 * new + 2 * copies * row * page, "flops": 0}


# ------------------------------------------------------------------ inputs

def _pages(needed, spare, device, g):
    """Block table rows (python lists) over a shuffled pool with spare pages."""
    total = sum(needed) + spare
    perm = torch.randperm(total, generator=g, device=device).tolist()
    rows, at = [], 0
    for n in needed:
        rows.append(perm[at:at + n])
        at += n
    return rows, total


def _table(rows, width, device):
    return torch.tensor([r + [0] * (width - len(r)) for r in rows], dtype=torch.int32,
                        device=device)


def _pool(case, lead, num_pages, device, g):
    """A [*lead, num_pages, page, Hkv, d] cache, stored page- or head-major inside a page."""
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    inner = (Hkv, page, d) if case["head_major"] else (page, Hkv, d)
    c = torch.randn(*lead, num_pages, *inner, generator=g, device=device,
                    dtype=_DT[case.get("dtype", "bf16")])
    return c.transpose(-3, -2) if case["head_major"] else c


def _ints(x, device):
    return torch.tensor(x, dtype=torch.int32, device=device)


def _offsets(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


def _trees(n, rng):
    """Parents (the root's is -1) and ancestors (bit sets, the node itself among
    them) of one random tree after the other."""
    parents, ancestors = [], []
    for size in n:
        bits = []
        for i in range(size):
            # mostly a child of one of the last few nodes, as drafts are deep and narrow
            p = -1 if i == 0 else rng.randint(max(0, i - 1 - rng.randrange(8)), i - 1)
            parents.append(p)
            bits.append((bits[p] if i else 0) | 1 << i)
        ancestors += bits
    return parents, ancestors


def _words(ancestors, words, device):
    """Bit sets as int64 words [T, words]."""
    full = (1 << 64) - 1
    rows = [[(a >> (64 * w)) & full for w in range(words)] for a in ancestors]
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in rows],
                        dtype=torch.int64, device=device)


def prepare(case, seed):
    device = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=device).manual_seed(seed)
    st = dict(case=case)
    {"attn": _prepare_attn, "sample": _prepare_sample, "commit": _prepare_commit,
     "evict": _prepare_evict, "fork": _prepare_fork}[case["op"]](case, st, device, g, seed)
    return st


def _prepare_attn(case, st, device, g, seed):
    n, kv = _nodes(case)
    rows, total = _pages([_cdiv(m, case["page"]) for m in kv], 8, device, g)
    width = max(map(len, rows))
    st["table"] = _table(rows, width, device)
    st["k_cache"] = _pool(case, (), total, device, g)
    st["v_cache"] = _pool(case, (), total, device, g)
    st["q"] = torch.randn(sum(n), case["H"], case["d"], generator=g, device=device,
                          dtype=torch.bfloat16)
    st["cu_q"], st["kv_len"] = _ints(_offsets(n), device), _ints(kv, device)
    _, ancestors = _trees(n, random.Random(seed))
    st["mask"] = _words(ancestors, case["words"], device)
    st["n_max"], st["kv_max"], st["scale"] = max(n), max(kv), 1.0 / math.sqrt(case["d"])
    if own:
        from online_softmax_attention_rf_gb300 import api
        # made once a step, used by every layer
        st["plan"] = api.PagedPlan(st["cu_q"], st["kv_len"], sum(n), case["H"], case["Hkv"],
                                   case["page"], width, causal=False)
        st["ws"] = api.attn_paged_workspace(case["d"], device)


def _prepare_sample(case, st, device, g, seed):
    B, V, mix = case["B"], case["V"], case["mix"]

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=device)

    # probabilities that fall off as a power of a token's rank, as a language model's do
    slope = 0.8 + uniform(B, 1)
    x = -slope * torch.log(1 + V * uniform(B, V))
    x += 0.5 * torch.randn(B, V, generator=g, device=device)
    st["logits"] = (x + 12).to(_DT[case["dtype"]])
    st["expo"] = torch.empty(B, V, device=device).exponential_(generator=g).clamp_min_(1e-20)
    st["temperature"] = 0.6 + 0.6 * uniform(B)
    top_k = (1 + uniform(B) * 99).to(torch.int32)
    top_p, min_p = 0.8 + 0.19 * uniform(B), 0.02 + 0.08 * uniform(B)
    st["top_k"] = top_k if mix in ("all", "each", "top_k") else None
    st["top_p"] = top_p if mix in ("all", "each", "top_p") else None
    st["min_p"] = min_p if mix in ("all", "each", "min_p") else None
    if mix == "each":  # of each eight users one decodes greedily, and each limit has its users
        i = torch.arange(B, device=device)
        st["temperature"] = torch.where(i % 8 == 7, torch.zeros_like(min_p), st["temperature"])
        st["top_k"] = torch.where(i % 2 == 0, top_k, torch.zeros_like(top_k))
        st["top_p"] = torch.where(i % 4 <= 1, top_p, torch.ones_like(top_p))
        st["min_p"] = torch.where(i % 8 >= 4, min_p, torch.zeros_like(min_p))


def _prepare_commit(case, st, device, g, seed):
    n, ctx = _contexts(case)
    rng = random.Random(seed)
    parents, ancestors = _trees(n, rng)
    tokens, sampled = [], []
    at = 0
    for size in n:
        tok = [rng.randrange(1000) for _ in range(size)]
        drawn = [rng.randrange(1000, 2000) for _ in range(size)]
        for i in range(1, size):  # most draws follow a drafted child, one of the last ones
            if rng.random() < 0.6:
                drawn[parents[at + i]] = tok[i]
        tokens += tok
        sampled += drawn
        at += size
    st["parent"], st["tokens"] = _ints(parents, device), _ints(tokens, device)
    st["sampled"] = _ints(sampled, device)
    st["ancestors"] = _words(ancestors, _cdiv(max(n), 64), device)
    st["cu_q"] = _ints(_offsets(n), device)
    kv = [c + x for c, x in zip(ctx, n)]
    st["kv_len"], st["n_max"] = _ints(kv, device), max(n)
    _prepare_caches(case, st, kv, device, g)


def _prepare_caches(case, st, kv, device, g):
    rows, total = _pages([_cdiv(m, case["page"]) for m in kv], 8, device, g)
    st["table"] = _table(rows, max(map(len, rows)) + 1, device)
    st["k_cache"] = _pool(case, (case["L"],), total, device, g)
    st["v_cache"] = _pool(case, (case["L"],), total, device, g)


def _prepare_evict(case, st, device, g, seed):
    kv, kept = _kept(case)
    rng = random.Random(seed)
    keep = []
    for m, k in zip(kv, kept):
        keep += sorted(rng.sample(range(m), k))
    st["keep"], st["cu_keep"] = _ints(keep, device), _ints(_offsets(kept), device)
    _prepare_caches(case, st, kv, device, g)


def _prepare_fork(case, st, device, g, seed):
    lens, page, width = _prompts(case), case["page"], case["width"]
    grown = [m + case["grow"] for m in lens]
    used = [_cdiv(m, page) for m in lens]
    rows, _ = _pages(used, case["P"] - sum(used), device, g)
    cols = max(_cdiv(m, page) for m in grown)
    st["table"], st["kv_len"] = _table(rows, cols, device), _ints(lens, device)
    # each prompt's children next to each other; the other pages: those that the
    # call does not need are mostly some other sequence's
    st["src"] = torch.arange(case["B"], device=device, dtype=torch.int32).repeat_interleave(width)
    st["grown"] = _ints(grown, device).repeat_interleave(width)
    need = width * sum(1 + _cdiv(b, page) - a for a, b in zip(used, grown))
    refs = torch.zeros(case["P"], dtype=torch.int32, device=device)
    others = torch.randperm(case["P"], generator=g, device=device)
    refs[others[min(case["P"], need + 64 + sum(used)):]] = 1
    refs[torch.tensor(sum(rows, []), dtype=torch.int64, device=device)] = 1
    st["refs"] = refs
    st["children"] = torch.zeros(width * case["B"], cols, dtype=torch.int32, device=device)
    st["k_cache"] = _pool(case, (case["L"],), case["P"], device, g)
    st["v_cache"] = _pool(case, (case["L"],), case["P"], device, g)


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _own(op, st)
    return {"attn": _plain_attn, "sample": _plain_sample, "commit": _plain_commit,
            "evict": _plain_evict, "fork": _plain_fork}[op](st)


def _own(op, st):
    from online_softmax_attention_rf_gb300 import api
    if op == "attn":
        return api.attn_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["plan"],
                              scale=st["scale"], workspace=st["ws"], tree_mask=st["mask"])
    if op == "sample":
        return api.sample_rows(st["logits"], st["expo"], temperature=st["temperature"],
                               top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"])
    if op == "commit":
        path, out, n_path, base, new_len = api.tree_accept(st["parent"], st["tokens"],
                                                           st["sampled"], st["cu_q"], st["kv_len"])
        api.kv_compact_paged(st["k_cache"], st["v_cache"], st["table"], path, st["cu_q"],
                             n_keep=n_path, base=base)
        return path, out, n_path, base, new_len, st["k_cache"], st["v_cache"]
    if op == "evict":
        api.kv_compact_paged(st["k_cache"], st["v_cache"], st["table"], st["keep"], st["cu_keep"])
        return st["k_cache"], st["v_cache"]
    page = st["case"]["page"]
    lens = api.pages_fork(st["table"], st["kv_len"], st["src"], st["children"], st["refs"], page)
    src, dst, left = api.pages_grow(st["children"], lens, st["grown"], st["refs"], page)
    api.kv_copy_pages(st["k_cache"], st["v_cache"], src, dst)
    api.pages_release(st["children"], st["grown"], st["refs"], page)
    return st["children"], lens, src, dst, left, st["refs"], st["k_cache"], st["v_cache"]


def _plain_attn(st):
    case, q, table, dev = st["case"], st["q"], st["table"], st["q"].device
    H, Hkv, d, page, B, N, M = (case["H"], case["Hkv"], case["d"], case["page"], case["B"],
                                st["n_max"], st["kv_max"])
    G = H // Hkv
    cu, kv = st["cu_q"].long(), st["kv_len"].long()
    n = cu[1:] - cu[:-1]
    i, j = torch.arange(N, device=dev), torch.arange(M, device=dev)
    rows = torch.minimum(cu[:-1, None] + i, cu[1:, None] - 1)       # [B, N], the last one again
    slots = table.long()[:, j // page] * page + j % page            # [B, M]
    k = st["k_cache"][slots // page, slots % page].float()          # [B, M, Hkv, d]
    v = st["v_cache"][slots // page, slots % page].float()
    node = j - (kv - n)[:, None]                                    # [B, M], below 0: context
    word = st["mask"][rows]                                         # [B, N, words]
    at = (node.clamp(min=0) // 64).clamp(max=case["words"] - 1)
    bit = word.gather(2, at[:, None, :].expand(B, N, M)) >> (node.clamp(min=0) % 64)[:, None, :]
    seen = (node < 0)[:, None, :] | ((bit & 1) == 1)
    seen &= (j < kv[:, None])[:, None, :]
    qb = q[rows].float().view(B, N, Hkv, G, d).permute(0, 2, 3, 1, 4)
    s = torch.matmul(qb, k.permute(0, 2, 3, 1)[:, :, None]) * st["scale"]   # [B, Hkv, G, N, M]
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    mx = s.max(-1, keepdim=True).values
    p = s.sub_(mx).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)[:, :, None]) / l
    lse = (mx + torch.log(l))[..., 0].permute(0, 3, 1, 2).reshape(B, N, H)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, H, d).to(q.dtype)
    seq = torch.searchsorted(cu, torch.arange(q.shape[0], device=dev), right=True) - 1
    at = torch.arange(q.shape[0], device=dev) - cu[seq]
    return o[seq, at], lse[seq, at]


def _plain_sample(st):
    # 64 bits: a value next to a border decides a whole number
    x = st["logits"].double()
    B, V = x.shape
    dev = x.device
    temp = st["temperature"].double()
    greedy = temp <= 0
    z = x / torch.where(greedy, 1.0, temp)[:, None]
    z, order = torch.sort(z, dim=-1, descending=True, stable=True)
    w = torch.exp(z - z[:, :1])
    rank = torch.arange(V, device=dev)
    keep = torch.ones_like(w, dtype=torch.bool)
    if st["top_k"] is not None:
        k = st["top_k"].long()
        keep &= rank < torch.where(k <= 0, V, k)[:, None]
    if st["top_p"] is not None:
        kept = torch.where(keep, w, 0.0)
        before = kept.cumsum(-1) - kept
        p = st["top_p"].double()[:, None]
        keep &= (p >= 1) | (before < p * kept.sum(-1, keepdim=True)) | (rank == 0)
    if st["min_p"] is not None:
        keep &= (w >= st["min_p"].double()[:, None]) | (rank == 0)
    w = torch.where(keep, w, 0.0)
    score = torch.where(keep, w / st["expo"].gather(1, order).double(), -1.0)
    # equal scores: the lowest index
    best = score == score.max(-1, keepdim=True).values
    token = torch.where(best, order, V).min(-1).values
    token = torch.where(greedy, order[:, 0], token)
    chosen = torch.where(order == token[:, None], w, 0.0).sum(-1)
    logprob = torch.where(greedy, 0.0, torch.log(chosen / w.sum(-1)))
    return token.to(torch.int32), logprob.float()


def _padded(st):
    """[B, N] rows of the packed nodes (the last one again), and which are there."""
    cu = st["cu_q"].long()
    i = torch.arange(st["n_max"], device=cu.device)
    return torch.minimum(cu[:-1, None] + i, cu[1:, None] - 1), i < (cu[1:] - cu[:-1])[:, None]


def _bits(words, N):
    """Bit sets [..., words] as truth values [..., N]."""
    i = torch.arange(N, device=words.device)
    return (words[..., i // 64] >> (i % 64)) & 1 == 1


def _slots(table, page, seq, pos):
    return table[seq, pos // page].long(), pos % page


def _plain_commit(st):
    page, N = st["case"]["page"], st["n_max"]
    rows, there = _padded(st)
    cu = st["cu_q"].long()
    parent, tok, drawn = st["parent"][rows].long(), st["tokens"][rows], st["sampled"][rows]
    # an edge is taken when the draw at the parent is the child's token; of several
    # such children the first one counts
    i = torch.arange(N, device=rows.device)
    twin = (parent[:, :, None] == parent[:, None, :]) & (tok[:, :, None] == tok[:, None, :]) & \
        (i[None, :] < i[:, None])
    taken = (tok == drawn.gather(1, parent.clamp(min=0))) & ~twin.any(-1)
    taken |= i == 0
    line = _bits(st["ancestors"][rows], N)                          # [B, N, N]
    accepted = ~(line & ~taken[:, None, :]).any(-1) & there
    n_path = accepted.sum(-1)
    rank = accepted.cumsum(-1) - 1
    seq, node = accepted.nonzero(as_tuple=True)
    at = rank[seq, node]
    path = torch.full((st["parent"].shape[0],), -1, dtype=torch.int32, device=rows.device)
    out = path.clone()
    path[cu[seq] + at] = node.to(torch.int32)
    out[cu[seq] + at] = drawn[seq, node]
    base = st["kv_len"] - (cu[1:] - cu[:-1]).to(torch.int32)
    _plain_move(st, seq, base.long()[seq] + node, base.long()[seq] + at)
    n_path = n_path.to(torch.int32)
    return path, out, n_path, base, base + n_path, st["k_cache"], st["v_cache"]


def _plain_move(st, seq, old, new):
    page = st["case"]["page"]
    p, r = _slots(st["table"], page, seq, old)
    p2, r2 = _slots(st["table"], page, seq, new)
    st["k_cache"][:, p2, r2] = st["k_cache"][:, p, r]
    st["v_cache"][:, p2, r2] = st["v_cache"][:, p, r]


def _plain_evict(st):
    i = torch.arange(st["keep"].shape[0], device=st["keep"].device)
    cu = st["cu_keep"].long()
    seq = torch.searchsorted(cu, i, right=True) - 1
    _plain_move(st, seq, st["keep"].long(), i - cu[seq])
    return st["k_cache"], st["v_cache"]


def _plain_fork(st):
    page, refs, children = st["case"]["page"], st["refs"], st["children"]
    dev, P = refs.device, refs.shape[0]
    src, grown = st["src"].long(), st["grown"].long()
    lens = st["kv_len"][src]
    j = torch.arange(children.shape[1], device=dev)
    used = -(-lens.long() // page)
    mine = j < used[:, None]
    torch.where(mine, st["table"][src], children, out=children)
    one = mine.to(torch.int32)
    refs.index_add_(0, children.reshape(-1).long().clamp(0, P - 1), one.reshape(-1))
    # a partly filled last page with several owners is replaced by a copy before it is
    # written to, except for the last of its owners when all of them are here
    last = children.gather(1, (used - 1).clamp(min=0)[:, None])[:, 0].long()
    shared = (grown > lens) & (lens % page > 0) & (refs[last] > 1)
    same = (last[:, None] == last[None, :]) & shared[:, None] & shared[None, :]
    i = torch.arange(last.shape[0], device=dev)
    copied = shared & ((same & (i[None, :] < i[:, None])).sum(-1) < refs[last] - 1)
    # new pages: the free ones of the lowest numbers, sequence after sequence
    first = used - copied.long()
    count = (-(-grown // page) - first).clamp(min=0)
    free = torch.sort((refs != 0).to(torch.int8), stable=True).indices.to(torch.int32)
    rank = (count.cumsum(0) - count)[:, None] + j - first[:, None]
    fresh = (j >= first[:, None]) & (j < (first + count)[:, None])
    left = (refs == 0).sum() - count.sum()
    torch.where(fresh, free[rank.clamp(0, P - 1)], children, out=children)
    refs.index_add_(0, children.reshape(-1).long().clamp(0, P - 1),
                    fresh.to(torch.int32).reshape(-1))
    refs.index_add_(0, last, -copied.to(torch.int32))
    now = children.gather(1, (used - 1).clamp(min=0)[:, None])[:, 0]
    copy_src = torch.where(copied, last, -1).to(torch.int32)
    copy_dst = torch.where(copied, now, -1)
    pair = copied.nonzero()[:, 0]
    st["k_cache"][:, now[pair].long()] = st["k_cache"][:, last[pair]]
    st["v_cache"][:, now[pair].long()] = st["v_cache"][:, last[pair]]
    held = (j < (-(-grown // page))[:, None]).to(torch.int32)
    refs.index_add_(0, children.reshape(-1).long().clamp(0, P - 1), -held.reshape(-1))
    return (children, lens, copy_src, copy_dst, left.to(torch.int32).view(1), refs,
            st["k_cache"], st["v_cache"])


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    if case["op"] == "attn":
        return None if work(case)["flops"] > 6e12 else _exact_attn(prepare(case, seed))
    if case["op"] == "sample":
        return _exact_sample(prepare(case, seed))
    return None  # whole numbers, and values that are copied


def _exact_attn(st):
    case, q = st["case"], st["q"]
    T, H, d = q.shape
    o = torch.empty(T, H, d, dtype=torch.float64, device=q.device)
    lse = torch.empty(T, H, dtype=torch.float64, device=q.device)
    cu, kv = st["cu_q"].tolist(), st["kv_len"].tolist()
    for b, m in enumerate(kv):
        n = cu[b + 1] - cu[b]
        j = torch.arange(m, device=q.device)
        page = st["table"][b].long()[j // case["page"]]
        bits = torch.stack([(st["mask"][cu[b]:cu[b + 1], t // 64] >> (t % 64)) & 1
                            for t in range(n)], 1)
        hidden = torch.zeros(n, m, dtype=torch.bool, device=q.device)
        hidden[:, m - n:] = bits == 0
        for h in range(H):
            k = st["k_cache"][page, j % case["page"], h // (H // case["Hkv"])].double()
            v = st["v_cache"][page, j % case["page"], h // (H // case["Hkv"])].double()
            z = st["scale"] * (q[cu[b]:cu[b + 1], h].double() @ k.T)
            z.masked_fill_(hidden, float("-inf"))
            lse[cu[b]:cu[b + 1], h] = torch.logsumexp(z, 1)
            o[cu[b]:cu[b + 1], h] = torch.exp(z - lse[cu[b]:cu[b + 1], h][:, None]) @ v
    return o, lse


def _exact_sample(st):
    B, V = st["logits"].shape
    token = torch.zeros(B, dtype=torch.int32)
    logprob = torch.zeros(B, dtype=torch.float64)
    for b in range(B):
        temp = float(st["temperature"][b])
        z = st["logits"][b].double()
        if temp <= 0:
            token[b] = int((z == z.max()).nonzero()[0, 0])
            continue
        logp = torch.log_softmax(z / temp, 0)
        kept = torch.argsort(-logp, stable=True)
        if st["top_k"] is not None and int(st["top_k"][b]) > 0:
            kept = kept[:int(st["top_k"][b])]
        if st["top_p"] is not None and float(st["top_p"][b]) < 1:
            p = torch.exp(logp[kept] - torch.logsumexp(logp[kept], 0))
            enough = torch.cumsum(p, 0) >= float(st["top_p"][b])
            kept = kept[:int(enough.nonzero()[0, 0]) + 1]
        if st["min_p"] is not None and float(st["min_p"][b]) > 0:
            low = math.log(float(st["min_p"][b])) + float(logp.max())
            kept = torch.cat([kept[:1], kept[1:][logp[kept[1:]] >= low]])
        race = logp[kept] - torch.log(st["expo"][b].double()[kept])
        token[b] = int(kept[race == race.max()].min())
        logprob[b] = logp[token[b]] - torch.logsumexp(logp[kept], 0)
    return token.to(st["logits"].device), logprob.to(st["logits"].device)
