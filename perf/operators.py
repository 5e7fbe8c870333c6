"""Workloads of the key/value cache operators: writing a paged cache, reading it
back, and attention for a batch whose sequences share a prefix.

Each case runs in two ways on the same inputs: as the plain formulas in torch
(`own` false) and as the library's calls (`own` true). The definitions:

append  x_q, x_k, x_v: the 128-wide heads of a token's projection row.
        q = R(pos) (x_q / rms(x_q) * g_q), k likewise with g_k, v = x_v, where
        rms(x) = sqrt(mean(x^2) + eps) and R turns the pair (j, j + 64) by the
        angle pos * theta^(-2j/128). q is rounded to bf16. k and v go to slot
        pos % 16 of page table[seq][pos / 16]: rounded to bf16, or as e4m3 with
        one power of two per token and head, the smallest 2^e for which
        max |x| <= 448 * 2^e (x / 2^e rounded to e4m3, ties to even).
read    the cached k and v of given (sequence, position) pairs, as bf16.
attend  o = softmax(q K^T / sqrt(128)) V and its log-sum-exp, for the query
        tokens of every sequence over that sequence's cached keys; query head h
        reads key head h // (hq / hkv). The first `prefix` keys are the same
        pages for every sequence. Causal: a sequence's queries are its last
        tokens, and each sees the keys up to its own position. A sequence
        without keys has o = 0 and log-sum-exp -inf.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
D, PAGE, EPS, THETA = 128, 16, 1e-6, 1e6
NAN8 = 0x7F  # e4m3 NaN


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token a sequence of the small layer, as a short answer is decoded: latency only
        {"name": "append 4 tokens", "op": "append", "seqs": 4, "new_lo": 1, "new_hi": 1, "past_lo": 100, "past_hi": 700,
         "hq": 8, "hkv": 2, "src": "f32", "cache": "bf16", "norm": True},
        # one token for each of 256 documents of the 4-billion-parameter layer
        {"name": "append 256 tokens", "op": "append", "seqs": 256, "new_lo": 1, "new_hi": 1, "past_lo": 128,
         "past_hi": 1024, "hq": 32, "hkv": 8, "src": "bf16", "cache": "bf16", "norm": True},
        # a prefill of ragged documents into an 8-bit cache, read back for the layers that want bf16
        {"name": "append+read 40 documents e4m3", "op": "append", "seqs": 40, "new_lo": 128, "new_hi": 1024,
         "past_lo": 0, "past_hi": 0, "hq": 32, "hkv": 8, "src": "bf16", "cache": "e4m3", "norm": True},
        # a few hundred tokens of odd-length documents read back from the small layer's cache
        {"name": "read 7 documents", "op": "read", "seqs": 7, "past_lo": 1, "past_hi": 129, "hkv": 2, "cache": "e4m3"},
        # 64 cached documents of 2,048 tokens taken out of the 8-bit cache
        {"name": "read 64x2048 e4m3", "op": "read", "seqs": 64, "past_lo": 2048, "past_hi": 2048, "hkv": 8,
         "cache": "e4m3"},
        # four short requests behind one instruction text, small layer: latency
        {"name": "attend 4 short", "op": "attend", "seqs": 4, "q_lo": 1, "q_hi": 1, "own_lo": 1, "own_hi": 128,
         "prefix": 512, "hq": 8, "hkv": 2, "cache": "bf16", "causal": True},
        # 256 documents behind a 2,048-token instruction, one decoded token each
        {"name": "attend 256 behind 2048", "op": "attend", "seqs": 256, "q_lo": 1, "q_hi": 1, "own_lo": 128,
         "own_hi": 1024, "prefix": 2048, "hq": 32, "hkv": 8, "cache": "bf16", "causal": True},
        # the same batch behind many worked examples, 8-bit cache
        {"name": "attend 256 behind 8192 e4m3", "op": "attend", "seqs": 256, "q_lo": 1, "q_hi": 1, "own_lo": 1,
         "own_hi": 1024, "prefix": 8192, "hq": 32, "hkv": 8, "cache": "e4m3", "causal": True},
        # long documents, 8-bit cache, short shared instruction
        {"name": "attend 32 long e4m3", "op": "attend", "seqs": 32, "q_lo": 1, "q_hi": 1, "own_lo": 7000,
         "own_hi": 8192, "prefix": 512, "hq": 32, "hkv": 8, "cache": "e4m3", "causal": True},
        # a single request far into a long context: the whole card on one sequence
        {"name": "attend 1 at 65k", "op": "attend", "seqs": 1, "q_lo": 1, "q_hi": 1, "own_lo": 257, "own_hi": 257,
         "prefix": 65520, "hq": 32, "hkv": 8, "cache": "bf16", "causal": True},
        # six answer positions a document that see the whole document, 8-bit cache, some documents empty
        {"name": "attend 64 x 6 positions e4m3", "op": "attend", "seqs": 64, "q_lo": 6, "q_hi": 6, "own_lo": 0,
         "own_hi": 2048, "prefix": 1024, "hq": 32, "hkv": 8, "cache": "e4m3", "causal": False},
        # ragged documents prefilled behind their instruction
        {"name": "attend 16 prefills", "op": "attend", "seqs": 16, "q_lo": 128, "q_hi": 1024, "own_lo": 128,
         "own_hi": 1024, "prefix": 2048, "hq": 32, "hkv": 8, "cache": "bf16", "causal": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend"])
    hq, hkv = rng.choice([(8, 2), (32, 8), (32, 4), (12, 3), (16, 1), (32, 1), (5, 5)])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "append":
        new = _log_int(rng, 1, 700)
        return {"op": op, "seqs": _log_int(rng, 1, 14000 // new if new > 50 else 300), "new_lo": max(1, new // 3),
                "new_hi": new, "past_lo": 0, "past_hi": _log_int(rng, 1, 2000), "hq": hq, "hkv": hkv,
                "src": rng.choice(["bf16", "f32"]), "cache": cache, "norm": rng.random() < 0.8}
    if op == "read":
        n = _log_int(rng, 1, 8192)
        return {"op": op, "seqs": _log_int(rng, 1, max(2, 90000 // n) if n > 400 else 256), "past_lo": n // 2,
                "past_hi": n, "hkv": hkv, "cache": cache}
    prefix = 16 * rng.choice([0, _log_int(rng, 1, 512)])
    causal = rng.random() < 0.7
    if rng.random() < 0.7:  # single tokens
        n = _log_int(rng, 1, 8192)
        seqs = _log_int(rng, 1, max(2, 90000 // n) if n > 400 else 256)
        q_lo = q_hi = 1
        own_lo = rng.randint(1 if causal else 0, n)
    else:
        q_hi = _log_int(rng, 2, 900)
        q_lo = rng.randint(1, q_hi)
        n = rng.randint(q_hi, 1024)
        seqs = _log_int(rng, 1, max(1, min(6000, 600000000 // (hq * (prefix + n))) // q_hi))
        own_lo = q_hi
    return {"op": op, "seqs": seqs, "q_lo": q_lo, "q_hi": q_hi, "own_lo": own_lo, "own_hi": n, "prefix": prefix,
            "hq": hq, "hkv": hkv, "cache": cache, "causal": causal}


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], the same for every seed."""
    return [lo + int((hi - lo + 1) * ((0.5 + 0.6180339887498949 * i) % 1.0)) for i in range(n)]


def _q_lens(c):
    q = _spread(c["q_lo"], c["q_hi"], c["seqs"])
    own_len = _spread(c["own_lo"], c["own_hi"], c["seqs"])
    return q, [max(a, b) for a, b in zip(q, own_len)] if c["causal"] else own_len


def work(case):
    c = case
    per = D * (2 if c["cache"] == "bf16" else 1) + (0 if c["cache"] == "bf16" else 1)  # bytes of a cached head row
    if c["op"] == "append":
        t = sum(_spread(c["new_lo"], c["new_hi"], c["seqs"]))
        heads = c["hq"] + 2 * c["hkv"]
        b = t * (heads * D * (2 if c["src"] == "bf16" else 4) + c["hq"] * D * 2 + 2 * c["hkv"] * per + 8)
        if c["cache"] == "e4m3":  # and read back
            b += t * 2 * c["hkv"] * (per + D * 2)
        return {"bytes": b, "flops": t * heads * D * 8}
    if c["op"] == "read":
        t = sum(_spread(c["past_lo"], c["past_hi"], c["seqs"]))
        return {"bytes": t * (2 * c["hkv"] * (per + D * 2) + 8), "flops": t * 2 * c["hkv"] * D}
    q, n = _q_lens(c)
    b = (c["prefix"] + sum(n)) * 2 * c["hkv"] * per + sum(q) * c["hq"] * (2 * D * 2 + 4)
    pairs = sum(a * (c["prefix"] + m) - (a * (a - 1) // 2 if c["causal"] else 0) for a, m in zip(q, n))
    return {"bytes": b, "flops": pairs * c["hq"] * 4 * D}


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


def _fill(g, table, lens, first, st):
    """Random k and v for the positions [first, len) of every sequence."""
    hkv = st["hkv"]
    for name in ("k", "v"):
        pool = st[name + "_pool"]
        x = _normal(g, pool.shape[0], hkv, PAGE, D)
        if st["cache"] == "e4m3":
            codes, e = _quantise(x)
            pool.copy_(codes)
            st[name + "_scale"].copy_(e)
        else:
            pool.copy_(x)
        # what lies behind a sequence's end in its last page is not a number
        for i, n in enumerate(lens):
            if n > first[i] and n % PAGE:
                pool[int(table[i, n // PAGE]), :, n % PAGE:] = NAN8 if st["cache"] == "e4m3" else float("nan")


def _cache(c, lens, prefix, seed):
    """A pool of shuffled pages, and the table of the sequences' pages; the first prefix/16 entries are shared."""
    rng = np.random.RandomState(seed % (1 << 31))
    pp = prefix // PAGE
    need = [max(0, -(-n // PAGE) - pp) for n in lens]
    total = pp + sum(need) + 3  # a pool is never quite full
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(1, pp + max(need))), -1, dtype=np.int32)
    table[:, :pp] = perm[:pp]
    at = pp
    for i, k in enumerate(need):
        table[i, pp:pp + k] = perm[at:at + k]
        at += k
    dt = torch.bfloat16 if c["cache"] == "bf16" else torch.uint8
    st = {"cache": c["cache"], "hkv": c["hkv"], "k_scale": None, "v_scale": None}
    for name in ("k", "v"):
        st[name + "_pool"] = torch.zeros((total, c["hkv"], PAGE, D), dtype=dt, device=DEV)
        if c["cache"] == "e4m3":
            st[name + "_scale"] = torch.full((total, c["hkv"], PAGE), 127, dtype=torch.uint8, device=DEV)
    st["table"] = torch.from_numpy(table).to(DEV)
    st["table_host"] = table
    st["prefix_pages"] = torch.from_numpy(perm[:pp].copy()).to(DEV)
    return st


def _tokens(lens, first):
    seq = np.concatenate([np.full(n - f, i, dtype=np.int32) for i, (n, f) in enumerate(zip(lens, first))])
    pos = np.concatenate([np.arange(f, n, dtype=np.int32) for n, f in zip(lens, first)])
    return torch.from_numpy(seq).to(DEV), torch.from_numpy(pos).to(DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["op"] == "append":
        past = _spread(c["past_lo"], c["past_hi"], c["seqs"])
        lens = [p + n for p, n in zip(past, _spread(c["new_lo"], c["new_hi"], c["seqs"]))]
        st = _cache(c, lens, 0, seed)
        st["seq"], st["pos"] = _tokens(lens, past)
        t, hq, hkv = st["seq"].numel(), c["hq"], c["hkv"]
        st["qkv"] = _normal(g, t, (hq + 2 * hkv) * D, dtype=torch.bfloat16 if c["src"] == "bf16" else torch.float32)
        st["q_norm"] = (1 + 0.1 * _normal(g, D, dtype=torch.float32)).bfloat16() if c["norm"] else None
        st["k_norm"] = (1 + 0.1 * _normal(g, D, dtype=torch.float32)).bfloat16() if c["norm"] else None
        st["q"] = torch.empty((t, hq, D), dtype=torch.bfloat16, device=DEV)
        st["hq"] = hq
    elif c["op"] == "read":
        lens = _spread(c["past_lo"], c["past_hi"], c["seqs"])
        st = _cache(c, lens, 0, seed)
        _fill(g, st["table_host"], lens, [0] * len(lens), st)
        st["seq"], st["pos"] = _tokens(lens, [0] * len(lens))
    else:
        q_len, n = _q_lens(c)
        # where nothing is causal a sequence may be without any key, the shared ones too
        lens = [m + c["prefix"] if m else 0 for m in n]
        st = _cache(c, lens, c["prefix"], seed)
        _fill(g, st["table_host"], lens, [c["prefix"]] * len(lens), st)
        offs = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        st["single"] = c["q_hi"] == 1
        st["q_offsets"] = None if st["single"] else torch.from_numpy(offs).to(DEV)
        st["q_rows"] = torch.from_numpy(offs).to(DEV)
        st["seq_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["q"] = _normal(g, int(offs[-1]), c["hq"], D)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((int(offs[-1]), c["hq"]), dtype=torch.float32, device=DEV)
        st.update(prefix=c["prefix"], causal=c["causal"], max_q=max(q_len), max_len=max(max(lens), c["prefix"], 1),
                  max_own=max(max(lens) - c["prefix"], 0), hq=c["hq"])
    if c["op"] != "attend":
        t, hkv = st["seq"].numel(), c["hkv"]
        st["k_out"] = torch.empty((t, hkv, D), dtype=torch.bfloat16, device=DEV)
        st["v_out"] = torch.empty((t, hkv, D), dtype=torch.bfloat16, device=DEV)
    st["op"] = c["op"]
    if own:  # the handle on the pools and the workspace, which a program keeps over its calls
        import trie_label_scoring_gb300 as Q
        st["handle"] = Q.KVCache(st["k_pool"], st["v_pool"], st["table"], st["k_scale"], st["v_scale"])
        if c["op"] == "attend":
            st["ws"] = torch.empty(Q.workspace_size_attention(st["handle"], st["hq"], st["q"].shape[0], st["max_q"],
                                                              st["max_len"], st["prefix"]),
                                   dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ the passes
def run(state):
    return {"append": _append, "read": _read, "attend": _attend}[state["op"]](state)


def _append(st):
    if own:
        import trie_label_scoring_gb300 as Q
        Q.cache_append(st["handle"], st["qkv"], st["hq"], st["seq"], st["pos"], q_out=st["q"], q_norm=st["q_norm"],
                       k_norm=st["k_norm"], rms_eps=EPS, rope_theta=THETA)
        if st["cache"] == "bf16":
            return {"q": st["q"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
        Q.cache_read(st["handle"], st["seq"], st["pos"], st["k_out"], st["v_out"])
        return {"q": st["q"], "k": st["k_out"], "v": st["v_out"]}
    hq, hkv = st["hq"], st["hkv"]
    x = st["qkv"].float().view(-1, hq + 2 * hkv, D)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if st["q_norm"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * st["q_norm"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * st["k_norm"].float()
    # angles in 64 bits: a far position times a frequency loses its fraction in 32
    ang = st["pos"].double()[:, None] * THETA ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    q, k = _rotate(q, cos, sin), _rotate(k, cos, sin)
    seq, pos = st["seq"].long(), st["pos"].long()
    page, slot = st["table"][seq, pos // PAGE].long(), pos % PAGE
    q = q.bfloat16()
    if st["cache"] == "bf16":
        st["k_pool"][page, :, slot] = k.bfloat16()
        st["v_pool"][page, :, slot] = v.bfloat16()
        return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    codes, e = _quantise(torch.stack([k, v]))
    st["k_pool"][page, :, slot], st["v_pool"][page, :, slot] = codes[0], codes[1]
    st["k_scale"][page, :, slot], st["v_scale"][page, :, slot] = e[0], e[1]
    return {"q": q, **_read(st)}


def _rotate(x, cos, sin):
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _values(st, name, page, slot=None):
    """Cached rows in fp32: whole pages [..., hkv, 16, 128], or one slot of each [..., hkv, 128]."""
    at = (page,) if slot is None else (page, slice(None), slot)
    x = st[name + "_pool"][at]
    if st["cache"] == "bf16":
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * _pow2(st[name + "_scale"][at].int() - 127)[..., None]


def _read(st):
    if own:
        import trie_label_scoring_gb300 as Q
        Q.cache_read(st["handle"], st["seq"], st["pos"], st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    seq, pos = st["seq"].long(), st["pos"].long()
    page, slot = st["table"][seq, pos // PAGE].long(), pos % PAGE
    return {"k": _values(st, "k", page, slot).bfloat16(), "v": _values(st, "v", page, slot).bfloat16()}


def _attend(st):
    if own:
        import trie_label_scoring_gb300 as Q
        Q.attention_shared(st["handle"], st["q"], st["q_offsets"], st["seq_len"], st["max_q"], st["max_len"],
                           st["prefix_pages"], st["out"], st["ws"], lse=st["lse"], causal=st["causal"])
        return {"out": st["out"], "lse": st["lse"]}
    hq, hkv, prefix, max_own, max_q = st["hq"], st["hkv"], st["prefix"], st["max_own"], st["max_q"]
    G, B, T = hq // hkv, st["seq_len"].numel(), st["q"].shape[0]
    starts, seq_len = st["q_rows"][:-1].long(), st["seq_len"].long()
    q_len = st["q_rows"][1:].long() - starts
    q = st["q"].float() / math.sqrt(D)
    # the shared keys: every query of the batch against one set
    kp, vp = (_values(st, n, st["prefix_pages"].long()).transpose(0, 1).reshape(hkv, prefix, D) for n in ("k", "v"))
    qf = q.view(T, hkv, G, D).permute(1, 0, 2, 3).reshape(hkv, T * G, D)
    sp = (qf @ kp.transpose(1, 2)).view(hkv, T, G, prefix)
    # the sequences' own keys, padded to the longest
    pages = st["table"][:, prefix // PAGE:prefix // PAGE + -(-max_own // PAGE)].long().clamp(min=0)
    ko, vo = (_values(st, n, pages).permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, D) for n in ("k", "v"))
    at = torch.arange(max_q, device=DEV)
    row = (starts[:, None] + at).clamp(max=T - 1)
    live = at < q_len[:, None]
    qo = q[row].view(B, max_q, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, max_q * G, D)
    last = seq_len[:, None] - (q_len[:, None] - at if st["causal"] else 1) - prefix  # last own key of a query
    key = torch.arange(ko.shape[2], device=DEV)
    seen = (key <= last[..., None]) & (key < (seq_len[:, None, None] - prefix))
    vo = torch.where((key < (seq_len - prefix)[:, None])[:, None, :, None], vo, 0)
    so = (qo @ ko.transpose(2, 3)).view(B, hkv, max_q, G, -1)
    so = torch.where(seen[:, None, :, None], so, float("-inf"))
    # one softmax over both parts, each query's rows brought to [B, hkv, max_q, G, ...]
    spo = sp[:, row].transpose(0, 1)
    spo = torch.where((seq_len > 0)[:, None, None, None, None], spo, float("-inf"))
    m = torch.cat([spo, so], -1).amax(-1, keepdim=True) if prefix + key.numel() else so.new_full(so.shape[:-1] + (1,), float("-inf"))
    m0 = torch.where(m == float("-inf"), 0, m)
    pp, po = torch.exp(spo - m0), torch.exp(so - m0)
    l = pp.sum(-1, keepdim=True) + po.sum(-1, keepdim=True)
    o = (pp.transpose(0, 1).reshape(hkv, B * max_q * G, prefix) @ vp).view(hkv, B, max_q, G, D).transpose(0, 1)
    o = o + (po.reshape(B, hkv, max_q * G, -1) @ vo).view(B, hkv, max_q, G, D)
    o = torch.where(l > 0, o / l, 0)
    lse = (m + torch.log(l))[..., 0]
    pick = lambda x: x.permute(0, 2, 1, 3, *range(4, x.dim())).reshape(B, max_q, hq, *x.shape[4:])[live]  # noqa: E731
    return {"out": pick(o).bfloat16(), "lse": pick(lse)}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _round_e4m3(x):
    """Nearest value of e4m3 (4-bit exponent, 3-bit mantissa, smallest step 2^-9), ties to even."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))), min=-6) - 3)
    return torch.round(x / step) * step


def _exact_rows(st, name, page, slot):
    x = st[name + "_pool"][page, :, slot]
    if st["cache"] == "bf16":
        return x.double()
    b = x.int()
    sign, ex, man = b >> 7, (b >> 3) & 15, (b & 7).double()
    v = torch.where(ex > 0, (8 + man) * torch.exp2(ex.double() - 10), man * 2.0 ** -9)
    v = torch.where((b & 127) == NAN8, float("nan"), torch.where(sign > 0, -v, v))
    return v * torch.exp2(st[name + "_scale"][page, :, slot].double() - 127)[..., None]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    table = st["table"].long()
    if case["op"] != "attend":
        seq, pos = st["seq"].long(), st["pos"].long()
        page, slot = table[seq, torch.div(pos, PAGE, rounding_mode="floor")], torch.remainder(pos, PAGE)
        if case["op"] == "read":
            return {n: _exact_rows(st, n, page, slot) for n in ("k", "v")}
        hq, hkv = case["hq"], case["hkv"]
        heads = st["qkv"].double().reshape(len(seq), -1, D)
        # pairs as complex numbers: rotation is a product with exp(i angle)
        turn = torch.exp(1j * pos.double()[:, None] * torch.exp(torch.arange(D // 2, device=DEV, dtype=torch.float64)
                                                                * (-2.0 * math.log(THETA) / D)))[:, None]
        parts = {}
        for name, lo, hi in (("q", 0, hq), ("k", hq, hq + hkv)):
            x = heads[:, lo:hi]
            if case["norm"]:
                x = x / ((x * x).sum(-1, keepdim=True) / D + EPS).sqrt() * st[name + "_norm"].double()
            z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * turn
            parts[name] = torch.cat([z.real, z.imag], -1)
        parts["v"] = heads[:, hq + hkv:]
        if case["cache"] == "bf16":
            out = {"q": parts["q"]}
            for name in ("k", "v"):
                pool = st[name + "_pool"].double()
                pool[page, :, slot] = parts[name]
                out[name + "_pool"] = pool
            return out
        out = {"q": parts["q"]}
        for name in ("k", "v"):
            x = parts[name]
            m, e = torch.frexp(x.abs().amax(-1, keepdim=True) / 448)
            e = (e - (m == 0.5).int()).double()
            out[name] = _round_e4m3(x / torch.exp2(e)) * torch.exp2(e)
        return out
    hq, hkv, prefix = case["hq"], case["hkv"], case["prefix"]
    G = hq // hkv
    q_len, _ = _q_lens(case)
    flops = work(case)["flops"]
    if flops > 6e12:
        return None
    out = torch.zeros((sum(q_len), hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((sum(q_len), hq), float("-inf"), dtype=torch.float64, device=DEV)
    at = 0
    for b, nq in enumerate(q_len):
        n = int(st["seq_len"][b])
        if n:
            pos = torch.arange(n, device=DEV)
            page = table[b, torch.div(pos, PAGE, rounding_mode="floor")]
            k, v = (_exact_rows(st, x, page, torch.remainder(pos, PAGE)) for x in ("k", "v"))
            q = st["q"][at:at + nq].double().view(nq, hkv, G, D)
            s = torch.einsum("qhgd,khd->hgqk", q, k) / D ** 0.5
            if case["causal"]:
                i = torch.arange(nq, device=DEV)[:, None]
                s.masked_fill_(pos > n - nq + i, float("-inf"))
            z = torch.logsumexp(s, -1)
            out[at:at + nq] = torch.einsum("hgqk,khd->qhgd", torch.exp(s - z[..., None]), v).reshape(nq, hq, D)
            lse[at:at + nq] = z.permute(2, 0, 1).reshape(nq, hq)
        at += nq
    return {"out": out, "lse": lse}
