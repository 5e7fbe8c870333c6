"""Workloads of the operators for decoding with trees of drafted tokens over the paged
key/value cache: page tables that follow the requests' lengths, tokens written at
slots that are not their positions, the trees' masks, attention, and keeping the
branch that turned out right.

Each case runs in two ways on the same inputs: as the plain formulas in torch
(`own` false) and as the library's calls (`own` true). The definitions:

resize  sequences go from old to new lengths (0, or at least the shared `prefix`). The
        free pages are a ring: `free` = (head, count). In order, a growing sequence takes
        the pages that it lacks from the ring's head, up to the first that the free pages
        or the room for tokens do not suffice for; a shrinking one appends the pages that
        it no longer needs to the ring. Out: the table, the ring, the granted lengths, the
        new tokens' offsets and their (sequence, position); -1 behind the last token.
append  x_q, x_k, x_v: the 128-wide heads of a token's projection row.
        q = R(rope_pos) (x_q / rms(x_q) * g_q), k likewise, v = x_v. R turns the first r
        dims of a head: pairs (j, j + r/2) or (2j, 2j + 1) by the angle rope_pos * w_j.
        w_j = theta^(-2j/r), "linear": / f; "base": theta f^(r/(r-2)) in theta's place;
        "parts": (1 - s) w_j / f + s w_j with s = clamp((L w_j / 2 pi - lo) / (hi - lo), 0, 1).
        Cosine and sine are taken times `magnitude`. k and v go to slot pos % 16 of page
        table[seq][pos / 16], as bf16 or as e4m3 with one power of two per token and head.
plan    of trees given by their nodes' parents: which nodes are a node's ancestors or
        itself, as bits, and its rotary position len - n + depth.
attend  o = softmax(q K^T / sqrt(128)) V and its log-sum-exp. A sequence's queries are
        the n nodes of its tree, its last n cached tokens; each sees the keys before the
        tree and, in the tree, its ancestors and itself.
accept  a drafted node is right if its token is the one that the model took after its
        parent (of several such children the first), and its parent is right; node 0 is.
        Out: the path of the right nodes, how many, the sequences' new lengths, the token
        taken after the last. The path's rows move to the front of the tree, in every layer.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
D, PAGE, EPS = 128, 16, 1e-6
VOCAB = 151936


# ------------------------------------------------------------------ cases
def listed():
    return [
        # four short requests, each a drafted tree larger: once a step, latency only
        {"name": "resize 4 requests", "op": "resize", "seqs": 4, "len_hi": 700, "step": 8, "prefix": 0, "spare": 1.0},
        # a batch of documents admitted behind their instruction while others leave
        {"name": "resize 512 documents", "op": "resize", "seqs": 512, "len_hi": 2048, "step": 2048, "prefix": 512,
         "spare": 1.0},
        # the drafted tokens of four short requests, small layer
        {"name": "append 4 trees of 6", "op": "append", "seqs": 4, "new_lo": 6, "new_hi": 6, "past": 700, "tree": True,
         "hq": 8, "hkv": 2, "src": "f32", "cache": "bf16", "norm": True, "interleaved": True, "rotary": 64,
         "scaling": "none"},
        # a prefill of ragged documents at positions past the model's first context, 8-bit cache
        {"name": "append 40 documents e4m3", "op": "append", "seqs": 40, "new_lo": 128, "new_hi": 1024, "past": 0,
         "tree": False, "hq": 32, "hkv": 8, "src": "bf16", "cache": "e4m3", "norm": True, "interleaved": False,
         "rotary": 128, "scaling": "parts"},
        # the masks of four small trees: once a step
        {"name": "plan 4 trees of 8", "op": "plan", "seqs": 4, "q_lo": 8, "q_hi": 8, "own_hi": 700},
        # a label trie of hundreds of nodes for every document
        {"name": "plan 256 trees to 500", "op": "plan", "seqs": 256, "q_lo": 300, "q_hi": 500, "own_hi": 2048},
        # four short requests with eight drafted tokens each, small layer: latency
        {"name": "attend 4 trees of 8", "op": "attend", "seqs": 4, "q_lo": 8, "q_hi": 8, "own_lo": 100, "own_hi": 700,
         "hq": 8, "hkv": 2, "cache": "bf16"},
        # a batch of documents, small ragged trees
        {"name": "attend 64 trees to 12", "op": "attend", "seqs": 64, "q_lo": 1, "q_hi": 12, "own_lo": 128,
         "own_hi": 2048, "hq": 32, "hkv": 8, "cache": "bf16"},
        # long documents in the 8-bit cache
        {"name": "attend 32 x 24 long e4m3", "op": "attend", "seqs": 32, "q_lo": 24, "q_hi": 24, "own_lo": 7000,
         "own_hi": 8192, "hq": 32, "hkv": 8, "cache": "e4m3"},
        # large trees: a trie's nodes over documents of a few thousand tokens
        {"name": "attend 16 trees to 100", "op": "attend", "seqs": 16, "q_lo": 40, "q_hi": 100, "own_lo": 1024,
         "own_hi": 4096, "hq": 32, "hkv": 8, "cache": "bf16"},
        # the verdict on four small trees, one layer
        {"name": "accept 4 trees of 8", "op": "accept", "seqs": 4, "q_lo": 8, "q_hi": 8, "own_hi": 700, "hkv": 2,
         "cache": "bf16", "layers": 1},
        # and on a batch of larger ones, through a stack of layers in 8 bits
        {"name": "accept 128 trees, 12 layers", "op": "accept", "seqs": 128, "q_lo": 16, "q_hi": 64, "own_hi": 256,
         "hkv": 8, "cache": "e4m3", "layers": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["resize", "append", "plan", "attend", "attend", "attend", "accept"])
    hq, hkv = rng.choice([(8, 2), (32, 8), (32, 4), (12, 3), (16, 1), (32, 1), (5, 5)])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "resize":
        n = _log_int(rng, 16, 4000)
        return {"op": op, "seqs": _log_int(rng, 1, max(2, 500000 // n)), "len_hi": n, "step": _log_int(rng, 1, n),
                "prefix": 16 * rng.choice([0, rng.randint(0, n // 16)]), "spare": rng.choice([1.0, 1.0, 0.6])}
    if op == "append":
        new = _log_int(rng, 1, 700)
        tree = new <= 64 and rng.random() < 0.7
        return {"op": op, "seqs": _log_int(rng, 1, 14000 // new if new > 50 else 250), "new_lo": max(1, new // 3),
                "new_hi": new, "past": _log_int(rng, 1, 4000), "tree": tree, "hq": hq, "hkv": hkv,
                "src": rng.choice(["bf16", "f32"]), "cache": cache, "norm": rng.random() < 0.8,
                "interleaved": rng.random() < 0.5, "rotary": 16 * rng.randint(1, 8),
                "scaling": rng.choice(["none", "linear", "base", "parts"])}
    q_hi = _log_int(rng, 1, 1000)
    q_lo = rng.randint(1, q_hi)
    if op == "plan":
        return {"op": op, "seqs": _log_int(rng, 1, max(2, min(256, 100000 // q_hi))), "q_lo": q_lo, "q_hi": q_hi,
                "own_hi": _log_int(rng, q_hi, 4000)}
    if op == "accept":
        layers = rng.randint(1, 12)
        return {"op": op, "seqs": _log_int(rng, 1, max(2, min(128, 8000 // q_hi))), "q_lo": q_lo, "q_hi": q_hi,
                "own_hi": q_hi + _log_int(rng, 1, 200), "hkv": hkv, "cache": cache, "layers": layers}
    n = max(q_hi, _log_int(rng, 8, 8192))
    seqs = _log_int(rng, 1, max(1, min(256, 120000 // n, 200000000 // (hq * n * q_hi))))
    return {"op": op, "seqs": seqs, "q_lo": q_lo, "q_hi": q_hi, "own_lo": rng.randint(q_hi, n), "own_hi": n, "hq": hq,
            "hkv": hkv, "cache": cache}


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], the same for every seed."""
    return [lo + int((hi - lo + 1) * ((0.5 + 0.6180339887498949 * i) % 1.0)) for i in range(n)]


def _tree_lens(c):
    """Nodes, and cached tokens, of every sequence."""
    q = _spread(c["q_lo"], c["q_hi"], c["seqs"])
    n = _spread(c.get("own_lo", c["q_hi"]), c["own_hi"], c["seqs"])
    return q, [max(a, b) for a, b in zip(q, n[::-1])]


def _resize_lens(c):
    """Lengths before and after: about half the sequences grow by up to `step`, the others give as much back."""
    a = [max(n, c["prefix"]) for n in _spread(0, c["len_hi"], c["seqs"])]
    by = _spread(0, c["step"], c["seqs"])
    b = [max(c["prefix"], min(c["len_hi"], x + d)) for x, d in zip(a, by)]
    return [x if i % 2 else y for i, (x, y) in enumerate(zip(a, b))], [y if i % 2 else x for i, (x, y) in enumerate(zip(a, b))]


def _row_bytes(cache):
    return D * 2 if cache == "bf16" else D + 1


def work(case):
    c = case
    if c["op"] == "resize":
        a, b = _resize_lens(c)
        tokens = sum(max(0, y - x) for x, y in zip(a, b))
        pages = sum(abs(-(-y // PAGE) + x // -PAGE) for x, y in zip(a, b))
        return {"bytes": 16 * c["seqs"] + 8 * tokens + 8 * pages, "flops": 0}
    if c["op"] == "append":
        t = sum(_spread(c["new_lo"], c["new_hi"], c["seqs"]))
        heads = c["hq"] + 2 * c["hkv"]
        b = t * (heads * D * (2 if c["src"] == "bf16" else 4) + c["hq"] * D * 2 + 2 * c["hkv"] * _row_bytes(c["cache"]) + 12)
        if c["cache"] == "e4m3":  # and read back
            b += t * 2 * c["hkv"] * (_row_bytes("e4m3") + D * 2)
        return {"bytes": b, "flops": t * heads * D * 8}
    q, n = _tree_lens(c)
    words = (max(q) + 31) // 32
    if c["op"] == "plan":
        return {"bytes": sum(q) * (8 + 4 * words) + 12 * c["seqs"], "flops": 0}
    if c["op"] == "accept":
        moved = sum(_about_right(a) for a in q)
        b = sum(q) * (16 + 4 * words) + 20 * c["seqs"] + moved * 4 * c["hkv"] * c["layers"] * _row_bytes(c["cache"])
        if c["cache"] == "e4m3":  # and the trees' rows read
            b += sum(q) * 2 * c["hkv"] * c["layers"] * (_row_bytes("e4m3") + D * 2)
        return {"bytes": b, "flops": 0}
    b = sum(n) * 2 * c["hkv"] * _row_bytes(c["cache"]) + sum(q) * (c["hq"] * (2 * D * 2 + 4) + 4 * words)
    pairs = sum(a * (m - a) + a * a // 4 for a, m in zip(q, n))
    return {"bytes": b, "flops": pairs * c["hq"] * 4 * D}


def _about_right(nodes):
    return min(nodes, 3)  # nodes of a tree that turn out right, on the mean


# ------------------------------------------------------------------ inputs
def _normal(g, *shape, dtype=torch.bfloat16):
    out = torch.empty(shape, device=DEV, dtype=dtype)
    return out.normal_(generator=g)


def _pow2(e):
    """2^e in fp32 from its bits, for whole numbers e in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """[..., 128] -> the e4m3 codes (as bytes) and the biased exponent of each row's power of two."""
    m, e = torch.frexp(x.float().abs().amax(-1))
    e = torch.where(m <= 0.875, e - 9, e - 8)  # 448 = 0.875 * 2^9
    return (x.float() * _pow2(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=dtype))).to(DEV)


def _cache(c, lens, seed, g=None, layers=1):
    """Pools of shuffled pages with the sequences' tokens in them (g given: random ones), and the table of their pages."""
    rng = np.random.RandomState(seed % (1 << 31))
    need = [-(-n // PAGE) for n in lens]
    total = sum(need) + 3  # a pool is never quite full
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(1, max(need))), -1, dtype=np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for i, k in enumerate(need):
        table[i, :k] = perm[at[i]:at[i + 1]]
    st = {"cache": c["cache"], "hkv": c["hkv"], "table": _dev(table), "layers": []}
    shape = (total, c["hkv"], PAGE, D)
    for _ in range(layers):
        layer = {"k_scale": None, "v_scale": None}
        for name in ("k", "v"):
            x = _normal(g, *shape) if g is not None else torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
            if c["cache"] == "e4m3":
                x, layer[name + "_scale"] = _quantise(x)
            layer[name] = x
        st["layers"].append(layer)
    return st


def _parents(rng, q):
    """Random trees: a node hangs off one of the eight before it, a near one the likelier."""
    out = []
    for n in q:
        i = np.arange(n)
        back = 1 + np.floor(rng.random_sample(n) ** 2 * np.minimum(i, 8)).astype(np.int64)
        out.append(np.where(i == 0, -1, i - np.minimum(back, np.maximum(i, 1))))
    return np.concatenate(out).astype(np.int32)


def _tree_state(c, st, q, lens, seed):
    rng = np.random.RandomState((seed + 7) % (1 << 31))
    parent = _parents(rng, q)
    st.update(parent=_dev(parent), offsets=_dev(np.concatenate([[0], np.cumsum(q)])), seq_len=_dev(lens),
              max_q=max(q), words=(max(q) + 31) // 32, total=int(sum(q)))
    return rng, parent


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"op": c["op"]}
    if c["op"] == "resize":
        _prepare_resize(c, seed, st)
    elif c["op"] == "append":
        _prepare_append(c, seed, g, st)
    else:
        q, lens = _tree_lens(c)
        if c["op"] != "plan":
            st.update(_cache(c, lens, seed, g, c.get("layers", 1)))
        rng, parent = _tree_state(c, st, q, lens, seed)
        mask = torch.zeros((st["total"], st["words"]), dtype=torch.int32, device=DEV)
        st.update(mask=mask, rope_pos=torch.zeros(st["total"], dtype=torch.int32, device=DEV))
        if c["op"] != "plan":  # a program has planned the step before
            _masks(st, mask, st["rope_pos"])
        if c["op"] == "attend":
            st["q"] = _normal(g, st["total"], c["hq"], D)
            st["out"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty((st["total"], c["hq"]), dtype=torch.float32, device=DEV)
            st.update(hq=c["hq"], max_len=max(lens))
        elif c["op"] == "accept":
            offs = np.concatenate([[0], np.cumsum(q)])
            start = np.repeat(offs[:-1], q)
            taken = rng.randint(0, VOCAB, st["total"])
            draft = rng.randint(0, VOCAB, st["total"])
            hit = (rng.random_sample(st["total"]) < 0.7) & (parent >= 0)
            draft[hit] = taken[(start + parent)[hit]]
            i32 = dict(dtype=torch.int32, device=DEV)
            st.update(draft=_dev(draft), taken=_dev(taken), path=torch.empty(st["total"], **i32),
                      accepted=torch.empty(len(q), **i32), new_len=torch.empty(len(q), **i32),
                      bonus=torch.empty(len(q), **i32))
            seq = np.repeat(np.arange(len(q)), q)
            st["seq"], st["pos"] = _dev(seq), _dev(np.asarray(lens)[seq] - np.asarray(q)[seq] + np.arange(st["total"]) - start)
            st["rows"] = [torch.empty((st["total"], c["hkv"], D), dtype=torch.bfloat16, device=DEV) for _ in range(2 * c["layers"])]
    if own and "layers" in st:  # the handles on the pools and the workspace, which a program keeps over its calls
        import trie_label_scoring_gb300 as Q
        st["handles"] = [Q.KVCache(x["k"], x["v"], st["table"], x["k_scale"], x["v_scale"]) for x in st["layers"]]
        if c["op"] == "attend":
            st["ws"] = torch.empty(Q.workspace_size_attention_tree(st["handles"][0], st["hq"], st["total"], st["max_q"],
                                                                   st["max_len"]), dtype=torch.uint8, device=DEV)
        if c["op"] == "append":
            st["rope"] = Q.Rope(layout="interleaved" if c["interleaved"] else "half", rotary_dim=c["rotary"],
                                **st["rope_args"])
    return st


def _prepare_resize(c, seed, st):
    """The table of the lengths before, in shuffled pages; the pages left are free. A pool whose `spare` is below 1
    has that share of the pages that the growing sequences will ask for."""
    rng = np.random.RandomState(seed % (1 << 31))
    a, b = _resize_lens(c)
    pp = c["prefix"] // PAGE
    pages = lambda n: max(pp, -(-n // PAGE)) - pp  # noqa: E731
    need = [pages(n) for n in a]
    grow = sum(max(0, pages(y) - pages(x)) for x, y in zip(a, b))
    free = int(math.ceil(grow * c["spare"]))
    total = pp + sum(need) + free
    perm = rng.permutation(max(1, total)).astype(np.int32)
    width = max(1, -(-c["len_hi"] // PAGE), pp)
    table = np.full((c["seqs"], width), -1, dtype=np.int32)
    at = pp + np.concatenate([[0], np.cumsum(need)])
    for i, k in enumerate(need):
        table[i, :pp] = perm[:pp]
        table[i, pp:pp + k] = perm[at[i]:at[i + 1]]
    ring = np.full(max(1, total), -1, dtype=np.int32)
    head = int(rng.randint(max(1, total)))
    ring[(head + np.arange(free)) % max(1, total)] = perm[at[-1]:at[-1] + free]
    st["room"] = max(1, sum(max(0, y - x) for x, y in zip(a, b)), sum(max(0, x - y) for x, y in zip(a, b)))
    st.update(table=_dev(table), ring=_dev(ring), free=_dev([head, free, 0, 0]), old=_dev(a), targets=(_dev(b), _dev(a)),
              turn=0, prefix=c["prefix"], prefix_pages=_dev(perm[:pp]) if pp else None, granted=_dev([0] * c["seqs"]),
              offsets=_dev([0] * (c["seqs"] + 1)), seq=_dev([0] * st["room"]), pos=_dev([0] * st["room"]))
    if own:  # a handle on the pool: small ones here, the call moves no keys
        import trie_label_scoring_gb300 as Q
        pool = torch.zeros((max(1, total), 1, PAGE, D), dtype=torch.bfloat16, device=DEV)
        st["handle"] = Q.KVCache(pool, pool, st["table"])


def _prepare_append(c, seed, g, st):
    new = _spread(c["new_lo"], c["new_hi"], c["seqs"])
    past = _spread(0, c["past"], c["seqs"])
    lens = [p + n for p, n in zip(past, new)]
    st.update(_cache(c, lens, seed))
    rng = np.random.RandomState((seed + 3) % (1 << 31))
    seq = np.repeat(np.arange(c["seqs"]), new)
    at = np.concatenate([np.arange(n) for n in new])
    pos = np.asarray(past)[seq] + at
    # a tree's node turns by its depth: its parent's and one
    deep = np.sort(rng.random_sample(len(at))) if c["tree"] else at
    rope = np.asarray(past)[seq] + (np.floor(deep * (at + 1)).astype(np.int64) if c["tree"] else at)
    st["seq"], st["pos"], st["rope_pos"] = _dev(seq), _dev(pos), _dev(rope)
    t, hq, hkv = len(seq), c["hq"], c["hkv"]
    st["qkv"] = _normal(g, t, (hq + 2 * hkv) * D, dtype=torch.bfloat16 if c["src"] == "bf16" else torch.float32)
    for name in ("q_norm", "k_norm"):
        st[name] = (1 + 0.1 * _normal(g, D, dtype=torch.float32)).bfloat16() if c["norm"] else None
    st["q"] = torch.empty((t, hq, D), dtype=torch.bfloat16, device=DEV)
    st["rows"] = [torch.empty((t, hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    # contexts four times the first one's 4,096 for the scaled kinds
    st["rope_args"] = {"theta": 1e6, "scaling": c["scaling"]}
    if c["scaling"] != "none":
        st["rope_args"]["factor"] = 4.0
    if c["scaling"] == "parts":
        st["rope_args"].update(original_len=4096.0, low=1.0, high=32.0, magnitude=0.1 * math.log(4.0) + 1)
    st.update(hq=hq, interleaved=c["interleaved"], rotary=c["rotary"])


# ------------------------------------------------------------------ the passes
def run(state):
    return {"resize": _resize, "append": _append, "plan": _plan, "attend": _attend, "accept": _accept}[state["op"]](state)


def _resize(st):
    new = st["targets"][st["turn"]]
    st["turn"] = 1 - st["turn"]  # the next step gives back what this one took
    old, granted = st["old"], st["granted"]
    if own:
        import trie_label_scoring_gb300 as Q
        Q.cache_resize(st["handle"], old, new, st["ring"], st["free"], granted, st["offsets"], st["seq"], st["pos"],
                       prefix_pages=st["prefix_pages"])
    else:
        _resize_plain(st, old, new, granted)
    st["old"], st["granted"] = granted, old
    return {"table": st["table"], "ring": st["ring"], "free": st["free"][:2], "granted": granted,
            "offsets": st["offsets"], "seq": st["seq"], "pos": st["pos"]}


def _resize_plain(st, old, new, granted):
    table, ring, free, prefix, room = st["table"], st["ring"], st["free"], st["prefix"], st["room"]
    N, pp = ring.numel(), prefix // PAGE
    old, new = old.long(), new.long()
    head, count = free[0].long(), free[1].long()
    o, n = old.clamp(min=prefix), new.clamp(min=prefix)
    po, pn = (o + PAGE - 1) // PAGE, (n + PAGE - 1) // PAGE
    grow = new > old
    need, tokens = torch.where(grow, pn - po, 0), torch.where(grow, n - o, 0)
    ok = ~grow | ((need.cumsum(0) <= count) & (tokens.cumsum(0) <= room))
    need, tokens = need * ok, tokens * ok
    back = torch.where(grow, 0, po - pn)
    col = torch.arange(table.shape[1], device=DEV)
    first = (need.cumsum(0) - need + head - po)[:, None] + col
    t = torch.where((grow & ok)[:, None] & (col >= po[:, None]) & (col < pn[:, None]), ring[first % N], table)
    if pp:
        from_none = (grow & ok & (old == 0))[:, None] & (col < pp)
        t = torch.where(from_none, torch.nn.functional.pad(st["prefix_pages"], (0, table.shape[1] - pp)), t)
    give = (col >= pn[:, None]) & (col < po[:, None]) & ~grow[:, None]
    at = (back.cumsum(0) - back + head + count - pn)[:, None] + col
    ring[at[give] % N] = table[give]
    table.copy_(torch.where(give, -1, t))
    free[0], free[1] = (head + need.sum()) % N, count - need.sum() + back.sum()
    granted.copy_(torch.where(ok, new, old))
    ends = tokens.cumsum(0)
    st["offsets"][1:] = ends
    i = torch.arange(room, device=DEV)
    b = torch.searchsorted(ends, i, right=True)
    live = i < ends[-1]
    b0 = b.clamp(max=len(ends) - 1)
    st["seq"].copy_(torch.where(live, b, -1))
    st["pos"].copy_(torch.where(live, o[b0] + i - (ends - tokens)[b0], 0))


def _angles(st, pos, dtype):
    """pos * w_j, [T, r/2], and the magnitude."""
    r, a = st["rotary"], st["rope_args"]
    theta, f = a["theta"], a.get("factor", 1.0)
    if a["scaling"] == "base":
        theta = theta * f ** (r / (r - 2))
    w = theta ** (-torch.arange(0, r, 2, device=DEV, dtype=dtype) / r)
    if a["scaling"] == "linear":
        w = w / f
    elif a["scaling"] == "parts":
        s = ((a["original_len"] * w / (2 * math.pi) - a["low"]) / (a["high"] - a["low"])).clamp(0, 1)
        w = (1 - s) * w / f + s * w
    return pos.to(dtype)[:, None] * w, a.get("magnitude", 1.0)


def _append(st):
    layer = st["layers"][0]
    if own:
        import trie_label_scoring_gb300 as Q
        h = st["handles"][0]
        Q.cache_append_rope(h, st["qkv"], st["hq"], st["seq"], st["pos"], st["rope"], rope_pos=st["rope_pos"],
                            q_out=st["q"], q_norm=st["q_norm"], k_norm=st["k_norm"], rms_eps=EPS)
        if st["cache"] == "bf16":
            return {"q": st["q"], "k_pool": layer["k"], "v_pool": layer["v"]}
        Q.cache_read(h, st["seq"], st["pos"], *st["rows"])
        return {"q": st["q"], "k": st["rows"][0], "v": st["rows"][1]}
    hq, hkv = st["hq"], st["hkv"]
    x = st["qkv"].float().view(-1, hq + 2 * hkv, D)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if st["q_norm"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * st["q_norm"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * st["k_norm"].float()
    # angles in 64 bits: a far position times a frequency loses its fraction in 32
    ang, mag = _angles(st, st["rope_pos"], torch.float64)
    cos, sin = (ang.cos() * mag).float()[:, None], (ang.sin() * mag).float()[:, None]
    q, k = _rotate(st, q, cos, sin), _rotate(st, k, cos, sin)
    seq, pos = st["seq"].long(), st["pos"].long()
    page, slot = st["table"][seq, pos // PAGE].long(), pos % PAGE
    q = q.bfloat16()
    if st["cache"] == "bf16":
        layer["k"][page, :, slot], layer["v"][page, :, slot] = k.bfloat16(), v.bfloat16()
        return {"q": q, "k_pool": layer["k"], "v_pool": layer["v"]}
    codes, e = _quantise(torch.stack([k, v]))
    layer["k"][page, :, slot], layer["v"][page, :, slot] = codes[0], codes[1]
    layer["k_scale"][page, :, slot], layer["v_scale"][page, :, slot] = e[0], e[1]
    return {"q": q, "k": _values(st, layer, "k", page, slot).bfloat16(), "v": _values(st, layer, "v", page, slot).bfloat16()}


def _rotate(st, x, cos, sin):
    r = st["rotary"]
    y, rest = x[..., :r], x[..., r:]
    if st["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _plan(st):
    if own:
        import trie_label_scoring_gb300 as Q
        Q.tree_plan(st["parent"], st["offsets"], st["seq_len"], st["max_q"], st["mask"], st["rope_pos"])
    else:
        _masks(st, st["mask"], st["rope_pos"])
    return {"mask": st["mask"], "rope_pos": st["rope_pos"]}


def _padded(st):
    """Of the trees side by side, each padded to the largest: its nodes' rows, which there are, and their parents (-1: none)."""
    starts = st["offsets"][:-1].long()
    n = st["offsets"][1:].long() - starts
    at = torch.arange(st["max_q"], device=DEV)
    live = at < n[:, None]
    row = (starts[:, None] + at).clamp(max=st["total"] - 1)
    return row, live, n, torch.where(live, st["parent"].long()[row], -1)


def _closure(st):
    """[B, n, n]: whether node j is node i's ancestor or itself. The paths of up to 1, 3, 7, .. steps, doubled."""
    row, live, n, parent = _padded(st)
    eye = torch.eye(st["max_q"], dtype=torch.bool, device=DEV)
    step = (parent[..., None] == torch.arange(st["max_q"], device=DEV)).half()
    seen = step + eye
    for _ in range(max(1, math.ceil(math.log2(st["max_q"])))):
        seen = (seen @ seen > 0).half()
    return seen.bool(), row, live, n, parent


def _masks(st, mask, rope_pos):
    seen, row, live, n, _ = _closure(st)
    pad = torch.nn.functional.pad(seen, (0, 32 * st["words"] - st["max_q"])).view(*seen.shape[:2], st["words"], 32)
    bits = (pad.long() << torch.arange(32, device=DEV)).sum(-1)
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
    mask.copy_(bits[live])
    depth = seen.sum(-1) - 1
    rope_pos.copy_((st["seq_len"].long()[:, None] - n[:, None] + depth)[live])


def _values(st, layer, name, page, slot=None):
    """Cached rows in fp32: whole pages [..., hkv, 16, 128], or one slot of each [..., hkv, 128]."""
    at = (page,) if slot is None else (page, slice(None), slot)
    x = layer[name][at]
    if st["cache"] == "bf16":
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * _pow2(layer[name + "_scale"][at].int() - 127)[..., None]


def _attend(st):
    if own:
        import trie_label_scoring_gb300 as Q
        Q.attention_tree(st["handles"][0], st["q"], st["offsets"], st["seq_len"], st["mask"], st["max_q"], st["max_len"],
                         st["out"], st["ws"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    hq, hkv, max_q = st["hq"], st["hkv"], st["max_q"]
    G, B = hq // hkv, st["seq_len"].numel()
    row, live, n, _ = _padded(st)
    seq_len = st["seq_len"].long()
    # every sequence's keys, padded to the longest
    pages = st["table"].long().clamp(min=0)
    k, v = (_values(st, st["layers"][0], x, pages).permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, D) for x in ("k", "v"))
    key = torch.arange(k.shape[2], device=DEV)
    q = (st["q"].float() / math.sqrt(D))[row].view(B, max_q, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, max_q * G, D)
    s = (q @ k.transpose(2, 3)).view(B, hkv, max_q, G, -1)
    # bit j of a node's mask: whether it sees node j
    j = key - (seq_len - n)[:, None]
    word = st["mask"][row].gather(2, (j // 32).clamp(0, st["words"] - 1)[:, None].expand(-1, max_q, -1))
    seen = (j < 0)[:, None] | ((word >> (j % 32)[:, None]) & 1).bool() & (j < n[:, None])[:, None]
    s = torch.where(seen[:, None, :, None], s, float("-inf"))
    v = torch.where((key < seq_len[:, None])[:, None, :, None], v, 0)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0, m))
    l = p.sum(-1, keepdim=True)
    o = (p.reshape(B, hkv, max_q * G, -1) @ v).view(B, hkv, max_q, G, D)
    o = torch.where(l > 0, o / l, 0)
    lse = (m + torch.log(l))[..., 0]
    pick = lambda x: x.permute(0, 2, 1, 3, *range(4, x.dim())).reshape(B, max_q, hq, *x.shape[4:])[live]  # noqa: E731
    return {"out": pick(o).bfloat16(), "lse": pick(lse)}


def _accept(st):
    if own:
        import trie_label_scoring_gb300 as Q
        Q.tree_accept(st["handles"], st["parent"], st["mask"], st["draft"], st["taken"], st["offsets"], st["seq_len"],
                      st["max_q"], st["path"], st["accepted"], st["new_len"], st["bonus"])
    else:
        _accept_plain(st)
    out = {"path": st["path"], "accepted": st["accepted"], "new_len": st["new_len"], "bonus": st["bonus"]}
    if st["cache"] == "bf16":
        out["pools"] = [x[name] for x in st["layers"] for name in ("k", "v")]
        return out
    if own:
        for i, h in enumerate(st["handles"]):
            Q.cache_read(h, st["seq"], st["pos"], st["rows"][2 * i], st["rows"][2 * i + 1])
        out["rows"] = st["rows"]
        return out
    page, slot = _place(st, st["seq"].long(), st["pos"].long())
    out["rows"] = [_values(st, x, name, page, slot).bfloat16() for x in st["layers"] for name in ("k", "v")]
    return out


def _place(st, seq, pos):
    return st["table"][seq, pos // PAGE].long(), pos % PAGE


def _accept_plain(st):
    seen, row, live, n, parent = _closure(st)
    draft, taken = st["draft"].long()[row], st["taken"].long()[row]
    up = parent.clamp(min=0)
    node = torch.arange(st["max_q"], device=DEV)
    match = (parent >= 0) & live & (draft == taken.gather(1, up))
    # not the first child with that token
    twin = (parent[:, :, None] == parent[:, None]) & (draft[:, :, None] == draft[:, None]) & (node[:, None] > node)
    match = (match & ~(twin & match[:, None]).any(-1)) | ((node == 0) & live)
    right = match & ~(seen & ~match[:, None]).any(-1)
    depth = seen.sum(-1) - 1
    count = right.sum(1)
    path = torch.full((len(n), st["max_q"]), -1, dtype=torch.int64, device=DEV)
    b, i = right.nonzero(as_tuple=True)
    path[b, depth[b, i]] = i
    st["path"].copy_(path[live])
    st["accepted"].copy_(count)
    st["new_len"].copy_(st["seq_len"] - n + count)
    last = path.gather(1, (count - 1).clamp(min=0)[:, None])
    st["bonus"].copy_(torch.where(count > 0, taken.gather(1, last.clamp(min=0))[:, 0], -1))
    base = (st["seq_len"].long() - n)[b]
    (p0, s0), (p1, s1) = _place(st, b, base + i), _place(st, b, base + depth[b, i])
    for x in st["layers"]:
        for pool in x.values():
            if pool is not None:
                pool[p1, :, s1] = pool[p0, :, s0]


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _round_e4m3(x):
    """Nearest value of e4m3 (4-bit exponent, 3-bit mantissa, smallest step 2^-9), ties to even."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))), min=-6) - 3)
    return torch.round(x / step) * step


def _exact_rows(st, layer, name, page, slot):
    x = layer[name][page, :, slot]
    if st["cache"] == "bf16":
        return x.double()
    b = x.int()
    sign, ex, man = b >> 7, (b >> 3) & 15, (b & 7).double()
    v = torch.where(ex > 0, (8 + man) * torch.exp2(ex.double() - 10), man * 2.0 ** -9)
    v = torch.where(sign > 0, -v, v)
    return v * torch.exp2(layer[name + "_scale"][page, :, slot].double() - 127)[..., None]


def exact(case, seed):
    if case["op"] in ("resize", "plan"):
        return None  # whole numbers
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attend": _exact_attend, "accept": _exact_accept}[case["op"]](case, st)


def _exact_append(case, st):
    seq, pos = st["seq"].long(), st["pos"].long()
    page, slot = st["table"].long()[seq, torch.div(pos, PAGE, rounding_mode="floor")], torch.remainder(pos, PAGE)
    hq, hkv, r = case["hq"], case["hkv"], case["rotary"]
    heads = st["qkv"].double().reshape(len(seq), -1, D)
    a = st["rope_args"]
    f, base = a.get("factor", 1.0), a["theta"]
    turns = []
    for j in range(r // 2):  # frequency by frequency, as defined
        w = base ** (-2.0 * j / r)
        if a["scaling"] == "linear":
            w = w / f
        if a["scaling"] == "base":
            w = (base * f ** (r / (r - 2.0))) ** (-2.0 * j / r)
        if a["scaling"] == "parts":
            s = min(1.0, max(0.0, (a["original_len"] / (2 * math.pi / w) - a["low"]) / (a["high"] - a["low"])))
            w = (1 - s) * (w / f) + s * w
        turns.append(w)
    # pairs as complex numbers: rotation is a product with exp(i angle)
    turn = a.get("magnitude", 1.0) * torch.exp(1j * st["rope_pos"].double()[:, None] * torch.tensor(turns, dtype=torch.float64, device=DEV))[:, None]
    parts = {}
    for name, lo, hi in (("q", 0, hq), ("k", hq, hq + hkv)):
        x = heads[:, lo:hi].clone()
        if case["norm"]:
            x = x / ((x * x).sum(-1, keepdim=True) / D + EPS).sqrt() * st[name + "_norm"].double()
        first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        parts[name] = x
    parts["v"] = heads[:, hq + hkv:]
    out = {"q": parts["q"]}
    for name in ("k", "v"):
        x = parts[name]
        if case["cache"] == "bf16":
            pool = st["layers"][0][name].double()
            pool[page, :, slot] = x
            out[name + "_pool"] = pool
        else:
            m, e = torch.frexp(x.abs().amax(-1, keepdim=True) / 448)
            e = (e - (m == 0.5).int()).double()
            out[name] = _round_e4m3(x / torch.exp2(e)) * torch.exp2(e)
    return out


def _exact_attend(case, st):
    hq, hkv = case["hq"], case["hkv"]
    G = hq // hkv
    q_len, lens = _tree_lens(case)
    if work(case)["flops"] > 6e12:
        return None
    table, parent = st["table"].long(), st["parent"].cpu().numpy()
    out = torch.zeros((sum(q_len), hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((sum(q_len), hq), dtype=torch.float64, device=DEV)
    at = 0
    for b, (nq, n) in enumerate(zip(q_len, lens)):
        pos = torch.arange(n, device=DEV)
        page = table[b, torch.div(pos, PAGE, rounding_mode="floor")]
        k, v = (_exact_rows(st, st["layers"][0], x, page, torch.remainder(pos, PAGE)) for x in ("k", "v"))
        hide = np.ones((nq, nq), dtype=bool)
        for i in range(nq):  # a node sees what its parent sees, and itself
            p = parent[at + i]
            if p >= 0:
                hide[i] = hide[p]
            hide[i, i] = False
        q = st["q"][at:at + nq].double().view(nq, hkv, G, D)
        s = torch.einsum("qhgd,khd->hgqk", q, k) / D ** 0.5
        s[..., n - nq:].masked_fill_(torch.from_numpy(hide).to(DEV), float("-inf"))
        z = torch.logsumexp(s, -1)
        out[at:at + nq] = torch.einsum("hgqk,khd->qhgd", torch.exp(s - z[..., None]), v).reshape(nq, hq, D)
        lse[at:at + nq] = z.permute(2, 0, 1).reshape(nq, hq)
        at += nq
    return {"out": out, "lse": lse}


def _exact_accept(case, st):
    q_len, lens = _tree_lens(case)
    parent, draft, taken, table = (st[x].cpu().numpy() for x in ("parent", "draft", "taken", "table"))
    src, dst, at = [], [], 0
    for b, (nq, n) in enumerate(zip(q_len, lens)):
        node, depth = 0, 0
        while True:  # from the root on, the first child with the token that was taken
            for to, pos in ((src, n - nq + node), (dst, n - nq + depth)):
                to.append((table[b, pos // PAGE], pos % PAGE))
            nxt = [i for i in range(node + 1, nq) if parent[at + i] == node and draft[at + i] == taken[at + node]]
            if not nxt:
                break
            node, depth = nxt[0], depth + 1
        at += nq
    (p0, s0), (p1, s1) = ([_dev([x[i] for x in rows]).long() for i in (0, 1)] for rows in (src, dst))
    out = {"path": None, "accepted": None, "new_len": None, "bonus": None}
    for layer in st["layers"]:
        for name in [x for x in layer if layer[x] is not None]:
            layer[name][p1, :, s1] = layer[name][p0, :, s0].clone()
    pairs = [(layer, name) for layer in st["layers"] for name in ("k", "v")]
    if case["cache"] == "bf16":
        out["pools"] = [layer[name].double() for layer, name in pairs]
    else:
        seq, pos = st["seq"].long(), st["pos"].long()
        page = st["table"].long()[seq, torch.div(pos, PAGE, rounding_mode="floor")]
        out["rows"] = [_exact_rows(st, layer, name, page, torch.remainder(pos, PAGE)) for layer, name in pairs]
    return out
