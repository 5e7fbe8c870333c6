"""Drafted trees over the document cache on the GPU: page tables that follow the lengths,
rotary layouts, masks, attention and the verdict, against plain arithmetic (64 bits where
there is any), and a run of them together.

Tolerances. Whole numbers are equal. A rounding to bf16 is off by at most 2^-8 of the
value, to e4m3 by 2^-4 or half its smallest step (2^-10 of the row's power of two). A
rotated element mixes two normed ones with a cosine and a sine within 1e-6 of their
values: 2e-6 times the pair's sizes, times the magnitude. Attention: a score is an fp32
sum of 128 exact products, within 128 * 2^-24 * sum |q||k| of its value; over an e4m3
cache the query's elements are also off by up to 2^-18 of the row's largest, which a key
turns into 2^-18 max|q| sum |k|; a weight is within twice that relative to itself
(numerator and sum). For the product with V a weight is rounded, within 2^-8 of itself
at most; over an e4m3 cache weights times their value rows' powers of two may be off by
2^-28 of the largest weight (1 after the division) times the largest power, key by key.
The result is rounded once, 2^-8 |o|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_cache_gpu import D, GAMMA, PAGE, Pool, built, check_stored, status  # noqa: E402,F401


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).cuda()


def random_parents(rng, n, back=8, roots=0.0):
    return [-1 if i == 0 or rng.random_sample() < roots else i - 1 - rng.randint(min(i, back)) for i in range(n)]


def ancestors(parent):
    """[n, n] truth values: node j is node i's ancestor or itself."""
    n = len(parent)
    m = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(parent):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def pack(rows, words):
    """Truth values [n, m] as int32 words [n, words]."""
    bits = np.zeros((rows.shape[0], 32 * words), dtype=np.uint8)
    bits[:, :rows.shape[1]] = rows
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


# ------------------------------------------------------------------ page tables
class Tables:
    """Page tables, free pages and lengths of plain lists, beside the library's."""

    def __init__(self, seqs, pages, max_pages, prefix=0, seed=0, head=0):
        import trie_label_scoring_gb300 as Q
        rng = np.random.RandomState(seed)
        perm = rng.permutation(pages).tolist()
        self.pp, self.prefix, self.pages, self.max_pages = prefix // PAGE, prefix, pages, max_pages
        self.prefix_pages, self.free = perm[:self.pp], perm[self.pp:]
        self.table = [[-1] * max_pages for _ in range(seqs)]
        self.len = [0] * seqs
        pool = torch.zeros((pages, 1, PAGE, D), dtype=torch.bfloat16, device="cuda")
        self.d_table = i32(self.table)
        self.cache = Q.KVCache(pool, pool, self.d_table)
        ring = np.full(pages, -5)
        ring[(head + np.arange(len(self.free))) % pages] = self.free
        self.ring, self.state = i32(ring), i32([head, len(self.free), 0, 0])
        self.d_prefix = i32(self.prefix_pages) if prefix else None

    def step(self, new, room=None, bad=(), stream=None):
        """One call and its plain counterpart; returns the granted lengths."""
        import trie_label_scoring_gb300 as Q
        B = len(self.len)
        granted, offs = torch.full((B,), 99, dtype=torch.int32, device="cuda"), torch.full((B + 1,), 99, dtype=torch.int32, device="cuda")
        seq = pos = None
        if room is not None:
            seq, pos = torch.full((room,), 99, dtype=torch.int32, device="cuda"), torch.full((room,), 99, dtype=torch.int32, device="cuda")
        Q.cache_resize(self.cache, i32(self.len), i32(new), self.ring, self.state, granted, offs, seq, pos,
                       prefix_pages=self.d_prefix, stream=stream)
        pages = lambda n: -(-max(n, self.prefix) // PAGE)  # noqa: E731
        took, given, tokens, ends, full, used = 0, [], [], [0], False, 0
        free = list(self.free)
        for b, (o, n) in enumerate(zip(self.len, new)):
            first = max(o, self.prefix)
            if b in bad:
                pass
            elif n > o:
                need, more = pages(n) - pages(o), max(n, self.prefix) - first
                full = full or took + need > len(free) or (room is not None and used + more > room)
                if not full:
                    if o == 0:
                        self.table[b][:self.pp] = self.prefix_pages
                    self.table[b][pages(o):pages(n)] = free[took:took + need]
                    took += need
                    used += more
                    tokens += [(b, p) for p in range(first, max(n, self.prefix))]
                    self.len[b] = n
            else:
                given += self.table[b][pages(n):pages(o)]
                self.table[b][pages(n):pages(o)] = [-1] * (pages(o) - pages(n))
                self.len[b] = n
            ends.append(len(tokens))
        self.free = free[took:] + given
        if not bad:
            status()
        assert granted.tolist() == self.len
        assert offs.tolist() == ends
        assert self.d_table.tolist() == self.table
        head, count, ticket, _ = self.state.tolist()
        assert count == len(self.free) and ticket == 0
        assert self.ring[(head + torch.arange(count, device="cuda")) % self.pages].tolist() == self.free
        if room is not None:
            assert seq.tolist() == [b for b, _ in tokens] + [-1] * (room - len(tokens))
            assert pos.tolist() == [p for _, p in tokens] + [0] * (room - len(tokens))
        return granted


@pytest.mark.parametrize("prefix", [0, 48])
@pytest.mark.parametrize("seqs", [1, 5, 40, 300])
def test_tables_follow_the_lengths(seqs, prefix):
    rng = np.random.RandomState(seqs + prefix)
    t = Tables(seqs, 12 * seqs + 3 + prefix // PAGE, 9 + prefix // PAGE, prefix, seed=seqs, head=7)
    for k in range(8):
        new = [int(rng.choice([0, x, x + 1, max(0, x - 1), prefix, prefix + rng.randint(0, 9 * PAGE + 1)])) for x in t.len]
        new = [0 if n < prefix else min(n, t.max_pages * PAGE) for n in new]
        t.step(new, room=None if k == 3 else seqs * 9 * PAGE + 5 * k)


def test_tables_of_thousands_of_sequences():
    """More sequences than a block has threads, and more tokens than a block's pass."""
    rng = np.random.RandomState(1)
    t = Tables(3001, 13000, 6, 32, seed=2, head=12990)
    for _ in range(4):
        t.step([32 + int(x) for x in rng.randint(0, 65, 3001)], room=3001 * 64 + 3)
    t.step([0] * 3001, room=8)


def test_growth_stops_where_pages_or_room_run_out():
    import trie_label_scoring_gb300 as Q
    t = Tables(6, 10, 8, seed=3)
    t.step([20, 33, 0, 16, 0, 0], room=200)                # 2 + 3 + 1 of 10 pages
    t.step([36, 1, 80, 17, 3, 0], room=200)                # 1 more, 2 back, then 5 of 3: refused, and all after
    t.step([36, 1, 16, 48, 3, 0], room=200)
    t.step([37, 2, 17, 48, 3, 1], room=2)                  # room for two tokens
    with pytest.raises(Q.QuailError):
        t.step([37, 2, 17, 48, 4, 2], room=0)              # an empty map is refused: it has no address to tell it from none
    t.step([0, 0, 0, 0, 0, 0], room=1)
    t.step([128, 32, 0, 0, 0, 1], room=200)                # every page, and one more
    assert t.len == [128, 32, 0, 0, 0, 0]


@pytest.mark.parametrize("new", [-1, 129, 16, 2 ** 31 - 1])
def test_bad_lengths_leave_their_sequence(new):
    import trie_label_scoring_gb300 as Q
    t = Tables(4, 40, 8, 32, seed=4)
    t.step([40, 50, 0, 33], room=200)
    t.step([56, new, 100, 32], room=200, bad=(1,))
    with pytest.raises(Q.QuailError) as e:
        Q.device_status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    status()


@pytest.mark.parametrize("state", [[-1, 3, 0, 0], [10, 3, 0, 0], [0, 11, 0, 0], [0, -1, 0, 0]])
def test_a_bad_ring_is_reported(state):
    import trie_label_scoring_gb300 as Q
    t = Tables(2, 10, 8, seed=4)
    t.step([40, 50], room=100)
    t.state.copy_(i32(state))
    granted, offs = i32([0, 0]), i32([0, 0, 0])
    before = t.d_table.clone()
    Q.cache_resize(t.cache, i32(t.len), i32([60, 10]), t.ring, t.state, granted, offs)
    with pytest.raises(Q.QuailError) as e:
        Q.device_status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    assert granted.tolist() == t.len and torch.equal(before, t.d_table) and t.state.tolist() == state


def test_more_pages_back_than_the_ring_holds_are_refused():
    """Pages that were never taken cannot be given back: the ring would overrun."""
    import trie_label_scoring_gb300 as Q
    t = Tables(2, 10, 8, seed=4)
    granted, offs = i32([0, 0]), i32([0, 0, 0])
    Q.cache_resize(t.cache, i32([32, 0]), i32([0, 16]), t.ring, t.state, granted, offs)
    with pytest.raises(Q.QuailError):
        Q.device_status()
    assert granted.tolist() == [32, 16]
    assert t.state.tolist() == [1, 9, 0, 0]


# ------------------------------------------------------------------ rotary append
def frequencies(r, theta, scaling, factor=1.0, original_len=0.0, low=1.0, high=32.0, **_):
    w = [theta ** (-2.0 * j / r) for j in range(r // 2)]
    if scaling == "linear":
        return [x / factor for x in w]
    if scaling == "base":
        return [(theta * factor ** (r / (r - 2))) ** (-2.0 * j / r) for j in range(r // 2)]
    if scaling == "parts":
        s = [min(1.0, max(0.0, (original_len * x / (2 * np.pi) - low) / (high - low))) for x in w]
        return [(1 - y) * x / factor + y * x for x, y in zip(w, s)]
    return w


def expected(qkv, pos, hq, hkv, gq, gk, eps, layout, r, theta, magnitude=1.0, **kw):
    x = qkv[:, :(hq + 2 * hkv) * D].double().reshape(qkv.shape[0], -1, D)
    ang = pos.double()[:, None] * torch.tensor(frequencies(r, theta, **kw), dtype=torch.float64, device="cuda")
    c, s = magnitude * torch.cos(ang)[:, None], magnitude * torch.sin(ang)[:, None]
    first, second = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    out = []
    for part, g in ((x[:, :hq], gq), (x[:, hq:hq + hkv], gk)):
        if g is not None:
            part = part / torch.sqrt((part ** 2).mean(-1, keepdim=True) + eps) * g.double()
        a, b = part[..., first], part[..., second]
        turned, slack = part.clone(), 2e-6 * part.abs()
        turned[..., first], turned[..., second] = a * c - b * s, b * c + a * s
        for to in (first, second):
            slack[..., to] = 2e-6 * magnitude * (a.abs() + b.abs())
        out.append((turned, slack))
    v = x[:, hq + hkv:]
    return out + [(v, torch.zeros_like(v))]


SCALED = [dict(scaling="none"), dict(scaling="linear", factor=8.0), dict(scaling="base", factor=2.5, magnitude=0.5),
          dict(scaling="parts", factor=4.0, original_len=4096.0, low=1.0, high=32.0, magnitude=1.14),
          dict(scaling="parts", factor=8.0, original_len=512.0, low=1.0, high=4.0)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("r", [16, 48, 64, 112, 128])
@pytest.mark.parametrize("scaled", range(len(SCALED)))
def test_append_rope(kind, layout, r, scaled):
    import trie_label_scoring_gb300 as Q
    kw = SCALED[scaled]
    hq, hkv, norm, src = [(8, 2, True, torch.bfloat16), (5, 5, True, torch.float32), (0, 2, False, torch.float32),
                          (16, 1, False, torch.bfloat16), (12, 3, True, torch.float32)][(scaled + r // 16) % 5]
    theta = [1e6, 1e4][r % 32 // 16]
    # slots of five sequences, a tree's positions: depths, and a few far ones
    lens, first = [1, 18, 117, 3, 4033], [0, 15, 100, 3, 4000]
    seq = np.concatenate([np.full(n - f, i) for i, (n, f) in enumerate(zip(lens, first))])
    pos = np.concatenate([np.arange(f, n) for n, f in zip(lens, first)])
    rng = np.random.RandomState(r + scaled)
    rope_pos = pos // 2
    rope_pos[-5:] = [0, 1, 100_000, 5_000_011, (1 << 24) - 1]
    order = rng.permutation(len(seq))
    seq, pos, rope_pos = i32(seq[order]), i32(pos[order]), i32(rope_pos[order])
    T = len(seq)
    pool = Pool(kind, hkv, lens, extra_pages=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn((T, (hq + 2 * hkv) * D + 8 * (r % 3)), generator=g, device="cuda").to(src)
    qkv[1] *= 1e-3
    qkv[2] *= 300
    qkv[3] = 0
    gq, gk = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() if norm else None for _ in range(2))
    q = torch.full((T, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda") if hq else None
    own = r % 32 == 0 or scaled % 2 == 0  # positions of their own, or the slots
    Q.cache_append_rope(pool.cache, qkv, hq, seq, pos, Q.Rope(theta, layout, r, **kw), rope_pos=rope_pos if own else None,
                        q_out=q, q_norm=gq, k_norm=gk, rms_eps=1e-6)
    status()
    (wq, sq), (wk, sk), (wv, sv) = expected(qkv, rope_pos if own else pos, hq, hkv, gq, gk, 1e-6, layout, r, theta, **kw)
    if hq:
        check_stored(q.double(), wq, sq)
    page, slot = pool.table[seq.long(), pos.long() // PAGE].long(), pos.long() % PAGE
    for name, want, slack, sc in (("k", wk, sk, pool.ks), ("v", wv, sv, pool.vs)):
        check_stored(pool.rows(seq, pos, name), want, slack, None if sc is None else sc[page, :, slot])
    untouched = torch.ones(pool.k.shape[:3], dtype=torch.bool, device="cuda")
    untouched[page, :, slot] = False
    fresh = Pool(kind, hkv, lens, extra_pages=2)
    raw = torch.uint8 if kind == "e4m3" else torch.int16
    assert torch.equal(pool.k.view(raw)[untouched], fresh.k.view(raw)[untouched])
    assert torch.equal(pool.v.view(raw)[untouched], fresh.v.view(raw)[untouched])


@pytest.mark.parametrize("tokens", [7, 700])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_rope_of_whole_heads_is_append(kind, tokens):
    import trie_label_scoring_gb300 as Q
    pools = [Pool(kind, 2, [tokens]) for _ in range(2)]
    seq, pos = i32([0] * tokens), i32(range(tokens))
    qkv = torch.randn((tokens, 8 * D), device="cuda").bfloat16()
    g = (1 + 0.2 * torch.randn(D, device="cuda")).bfloat16()
    q = [torch.zeros((tokens, 4, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    Q.cache_append(pools[0].cache, qkv, 4, seq, pos, q_out=q[0], q_norm=g, k_norm=g, rope_theta=1e6)
    Q.cache_append_rope(pools[1].cache, qkv, 4, seq, pos, Q.Rope(1e6), q_out=q[1], q_norm=g, k_norm=g)
    status()
    assert torch.equal(q[0], q[1])
    raw = torch.uint8 if kind == "e4m3" else torch.int16
    assert torch.equal(pools[0].k.view(raw), pools[1].k.view(raw)) and torch.equal(pools[0].v.view(raw), pools[1].v.view(raw))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_dims_that_pass_keep_infinities_to_themselves(layout):
    """Without a norm an infinity among the dims past rotary_dim reaches no other element."""
    import trie_label_scoring_gb300 as Q
    pool = Pool("bf16", 1, [4])
    qkv = torch.randn((4, 3 * D), device="cuda")
    qkv[:, 70] = float("inf")
    qkv[:, D + 127] = float("-inf")
    q = torch.zeros((4, 1, D), dtype=torch.bfloat16, device="cuda")
    seq, pos = i32([0] * 4), i32(range(4))
    Q.cache_append_rope(pool.cache, qkv, 1, seq, pos, Q.Rope(1e4, layout, 64), q_out=q)
    status()
    assert torch.isinf(q).sum().item() == 4 and bool(torch.isinf(q[:, 0, 70]).all()) and not bool(q.isnan().any())
    k = pool.rows(seq, pos, "k")
    assert torch.isinf(k).sum().item() == 4 and bool(torch.isinf(k[:, 0, 127]).all()) and not bool(k.isnan().any())


@pytest.mark.parametrize("far", [-1, 1 << 24, -2 ** 31])
def test_rope_positions_out_of_range_are_reported(far):
    import trie_label_scoring_gb300 as Q
    pool = Pool("bf16", 1, [4])
    qkv = torch.randn((4, 3 * D), device="cuda")
    q = torch.full((4, 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    Q.cache_append_rope(pool.cache, qkv, 1, i32([0, 0, -1, 0]), i32([0, 1, 2, 3]), Q.Rope(1e4), rope_pos=i32([0, far, far, 1]),
                        q_out=q)
    with pytest.raises(Q.QuailError) as e:
        Q.device_status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    assert bool((q[1:3] == 3).all()) and not bool((q[0] == 3).all())
    k = pool.rows(i32([0] * 4), i32(range(4)), "k")
    assert k.isnan().all(-1)[:, 0].tolist() == [False, True, True, False]


# ------------------------------------------------------------------ masks
TREES = {
    "one": [[-1]],
    "chain": [list(range(-1, 63))],
    "long chain": [list(range(-1, 1023))],
    "star": [[-1] + [0] * 99],
    "forest": [[-1] * 33],
    "mixed": [[-1, 0, 0, 1], [], list(range(-1, 31)), list(range(-1, 32)), [-1], [-1, -1, 1, 0, 2]],
}


@pytest.mark.parametrize("name", list(TREES) + ["random"])
@pytest.mark.parametrize("slack", [0, 1, 40])
def test_plan(name, slack):
    import trie_label_scoring_gb300 as Q
    rng = np.random.RandomState(3)
    trees = TREES.get(name) or [random_parents(rng, n, roots=0.1) for n in rng.randint(0, 300, 40)]
    n = [len(t) for t in trees]
    max_q = min(1024, max(n) + slack)
    words = (max_q + 31) // 32
    lens = [k + int(rng.randint(0, 5000)) for k in n]
    T = sum(n)
    mask = torch.full((T + 2, words), 0x55555555, dtype=torch.int32, device="cuda")
    rope = torch.full((T + 2,), -9, dtype=torch.int32, device="cuda")
    parent = i32(sum(trees, []) + [7, 7])  # rows behind the last tree
    Q.tree_plan(parent, i32(np.concatenate([[0], np.cumsum(n)])), i32(lens), max_q, mask, rope)
    status()
    want = np.concatenate([pack(ancestors(t), words) for t in trees if t])
    depth = np.concatenate([ancestors(t).sum(1) - 1 + l - len(t) for t, l in zip(trees, lens) if t])
    assert np.array_equal(mask[:T].cpu().numpy(), want)
    assert np.array_equal(rope[:T].cpu().numpy(), depth)
    assert bool((mask[T:] == 0x55555555).all()) and bool((rope[T:] == -9).all())


@pytest.mark.parametrize("what", ["self", "later", "below", "offsets", "length", "many"])
def test_plan_reports_bad_trees(what):
    import trie_label_scoring_gb300 as Q
    parent, offs, lens, max_q = [-1, 0, 1, -1, 0, 0, -1], [0, 3, 6, 7], [5, 9, 1], 3
    if what == "self":
        parent[4] = 1
    if what == "later":
        parent[4] = 2
    if what == "below":
        parent[4] = -2
    if what == "offsets":
        offs[2] = 8
    if what == "length":
        lens[1] = 2
    if what == "many":
        max_q, offs = 2, [0, 2, 6, 7]
    mask = torch.full((7, 1), 77, dtype=torch.int32, device="cuda")
    rope = torch.full((7,), 77, dtype=torch.int32, device="cuda")
    Q.tree_plan(i32(parent), i32(offs), i32(lens), max_q, mask, rope)
    with pytest.raises(Q.QuailError) as e:
        Q.device_status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    got = mask[:, 0].tolist()
    assert got[:2] == [1, 3] and rope.tolist()[:2] == [lens[0] - (offs[1]) , lens[0] - offs[1] + 1]
    if what in ("self", "later", "below"):
        assert got[3:6] == [1, 2, 5]  # alone
    elif what == "offsets":
        assert got[3:] == [77] * 4    # the third begins at 8 as well
    else:
        assert got[3:6] == [77] * 3 and got[6] == 1


# ------------------------------------------------------------------ attention
def attention_64(pool, q, offs, lens, seen, scale):
    """o, lse in 64 bits and how far each may be off; seen: per sequence truth values [n, n]."""
    T, hq, _ = q.shape
    G = hq // pool.hkv
    o, tol_o = torch.zeros((2, T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), float("-inf"), dtype=torch.float64, device="cuda")
    tol_l = torch.zeros((T, hq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        lo, hi = offs[b], offs[b + 1]
        if n == 0 or hi == lo:
            continue
        pos = torch.arange(n, device="cuda", dtype=torch.int32)
        k, v = (pool.rows(torch.full_like(pos, b), pos, x) for x in ("k", "v"))
        x = q[lo:hi].double().reshape(hi - lo, pool.hkv, G, D)
        hide = torch.zeros((hi - lo, n), dtype=torch.bool, device="cuda")
        hide[:, n - (hi - lo):] = ~torch.from_numpy(seen[b]).cuda()
        hide = hide[:, None, None]
        s = (torch.einsum("qhgd,khd->qhgk", x, k) * scale).masked_fill(hide, float("-inf"))
        mag = (torch.einsum("qhgd,khd->qhgk", x.abs(), k.abs()) * scale).masked_fill(hide, 0)
        drift = GAMMA * mag.amax(-1) + 2.0 ** -20
        if pool.kind == "e4m3":
            drift = drift + 2.0 ** -18 * scale * x.abs().amax(-1) * k.abs().sum(-1).amax(0)[:, None]
        z = torch.logsumexp(s, -1)
        none = z == float("-inf")
        p = torch.exp(s - torch.where(none, 0, z)[..., None])
        w = torch.einsum("qhgk,khd->qhgd", p, v)
        wa = torch.einsum("qhgk,khd->qhgd", p, v.abs())
        lost = 0
        if pool.kind == "e4m3":  # |v| <= 448 of its row's power of two
            page = pool.table[b, pos.long() // PAGE].long()
            power = torch.exp2(pool.vs[page, :, pos.long() % PAGE].double() - 127).amax(0)  # [hkv]
            lost = (n * 2.0 ** -28 * 448 * power)[None, :, None, None] * p.amax(-1)[..., None]
        o[lo:hi] = w.reshape(hi - lo, hq, D)
        lse[lo:hi] = z.reshape(hi - lo, hq)
        tol_o[lo:hi] = ((2.0 ** -8 * 1.01 + 2 * drift[..., None]) * wa + 2.0 ** -8 * w.abs() + lost).reshape(hi - lo, hq, D)
        tol_l[lo:hi] = (drift + 2.0 ** -22 * z.abs().nan_to_num(0, 0, 0)).reshape(hi - lo, hq)
    return o, lse, tol_o, tol_l


def attend(pool, q, offs, lens, seen, scale=None, slack=0, more=0, rows_after=2, lse=True, workspace=None, stream=None,
           bounds=None):
    """One call with rows behind the last sequence; returns out, lse of the real rows."""
    import trie_label_scoring_gb300 as Q
    T, hq, _ = q.shape
    max_q = min(1024, max([1] + [len(s) for s in seen]) + more)
    words = (max_q + 31) // 32
    rows = [pack(s, words) for s in seen if len(s)]
    # bits from n on may be anything
    for r, s in zip(rows, [s for s in seen if len(s)]):
        r.view(np.uint32)[:] |= pack(~np.pad(np.ones_like(s), ((0, 0), (0, 32 * words - len(s)))), words).view(np.uint32)
    mask = i32(np.concatenate(rows + [np.full((rows_after, words), -1)]))
    q = torch.cat([q, torch.full((rows_after, hq, D), float("nan"), dtype=q.dtype, device="cuda")])
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full(q.shape[:2], 5.0, device="cuda") if lse else None
    max_len = max(max(lens), 1) + slack
    n = Q.workspace_size_attention_tree(pool.cache, hq, q.shape[0], max_q, max_len)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    Q.attention_tree(pool.cache, q, i32(offs), i32(lens), mask, max_q, max_len, out, ws, lse=ls, scale=scale, stream=stream)
    status()
    assert bool((out[T:] == 5).all()) and (ls is None or bool((ls[T:] == 5).all()))
    return out[:T], None if ls is None else ls[:T]


def check_attention(pool, q, offs, lens, seen, scale=None, **kw):
    o, z, tol_o, tol_l = attention_64(pool, q, offs, lens, seen, scale or D ** -0.5)
    out, lse = attend(pool, q, offs, lens, seen, scale, **kw)
    live = z > float("-inf")
    err = (out.double() - o).abs()
    assert bool((err <= tol_o).all()), f"o off by {float((err - tol_o).max()):.3g} more than allowed"
    if lse is not None:
        assert torch.equal(~live, lse == float("-inf"))
        err = (lse.double() - z)[live].abs()
        assert bool((err <= tol_l[live]).all()), f"lse off by {float((err - tol_l[live]).max()):.3g} too much"
    return out, lse


HEADS = [(8, 2), (32, 8), (5, 5), (16, 1), (32, 1), (12, 3), (128, 4), (28, 4), (128, 1), (64, 64)]
ATTEND = [  # nodes, keys (the tree's included)
    ([1], [1]), ([1], [16]), ([1, 1, 1, 1], [17, 1, 15, 33]), ([3, 1, 2], [3, 5, 700]), ([8, 0, 8], [8, 40, 640]),
    ([8] * 5, [127, 128, 129, 135, 136]), ([33, 64], [33, 1000]), ([12, 1, 5, 7, 3, 11] * 7, [300, 20, 17, 128, 900, 11] * 7),
    ([100], [2300]), ([130, 257], [513, 257]), ([1000], [1100]), ([2, 40], [9000, 41]),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention_of_trees(kind, hq, hkv, case):
    n, lens = ATTEND[case]
    rng = np.random.RandomState(case)
    seen = [ancestors(random_parents(rng, k, roots=0.05)) if k else np.zeros((0, 0), dtype=bool) for k in n]
    pool = Pool(kind, hkv, lens, seed=case, extra_pages=case % 3)
    pool.fill(lens)
    offs = [0] + list(np.cumsum(n))
    q = torch.randn((offs[-1], hq, D), generator=torch.Generator(device="cuda").manual_seed(case), device="cuda").bfloat16()
    check_attention(pool, q, offs, lens, seen, slack=(0, 0, 30)[case % 3], more=(0, 1, 40)[(case + hkv) % 3], lse=case % 4 != 1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 3, 6, 7, 11, 17, 31, 33, 48, 63, 65, 96, 97, 100, 127])
@pytest.mark.parametrize("slack", [0, 1 << 20])
def test_groups_of_all_sizes(kind, group, slack):
    """Heads to a KV head that divide no tile; bounds a thousand times the lengths."""
    rng = np.random.RandomState(group)
    n, lens = [1, 2, 0, 9, 14, 1], [130, 2, 0, 300, 14, 1]
    seen = [ancestors(random_parents(rng, k, roots=0.2)) if k else np.zeros((0, 0), dtype=bool) for k in n]
    pool = Pool(kind, 1, lens, extra_pages=slack // 16)
    pool.fill(lens)
    offs = [0] + list(np.cumsum(n))
    q = torch.randn((offs[-1], group, D), device="cuda").bfloat16()
    check_attention(pool, q, offs, lens, seen, slack=slack, more=group % 3 * 100)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_the_most_heads_and_nodes(kind):
    """128 KV heads; a tree of 1,024 nodes; 3,000 sequences of a node."""
    rng = np.random.RandomState(1)
    for n, lens, hq, hkv in (([1024, 3], [1200, 3], 4, 1), ([5, 40], [200, 50], 128, 128), ([1] * 3000, [1 + i % 40 for i in range(3000)], 8, 2)):
        seen = [ancestors(random_parents(rng, k)) for k in n]
        pool = Pool(kind, hkv, lens)
        pool.fill(lens[:40])
        if len(lens) > 40:  # the same rows in every fortieth sequence
            for i in range(40, len(lens)):
                pool.table[i] = pool.table[i % 40]
        offs = [0] + list(np.cumsum(n))
        q = torch.randn((offs[-1], hq, D), device="cuda").bfloat16()
        if len(lens) <= 40:
            check_attention(pool, q, offs, lens, seen)
        else:
            out, lse = attend(pool, q, offs, lens, seen)
            o, z, tol_o, tol_l = attention_64(pool, q[:400], offs[:401], lens[:400], seen[:400], D ** -0.5)
            assert bool(((out[:400].double() - o).abs() <= tol_o).all())
            q[2000:2040] = q[:40]
            again, _ = attend(pool, q, offs, lens, seen)
            assert torch.equal(again[2000:2040], again[:40]) and torch.equal(again[:40], out[:40])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 1), (5, 5)])
def test_any_mask_and_rows_that_see_nothing(kind, hq, hkv):
    """Masks that are no tree's; nodes that see no key: o = 0, lse = -inf, also beside others that do; no keys at all."""
    rng = np.random.RandomState(7)
    n, lens = [20, 40, 3, 5, 70], [20, 300, 3, 0, 70]
    seen = [rng.random_sample((k, k)) < 0.3 for k in n]
    seen[0][::3] = False
    seen[1][5] = False
    seen[2][:] = False
    seen[4][:, 5:] = False  # far fewer keys than nodes
    seen[4][60:] = False
    pool = Pool(kind, hkv, lens)
    pool.fill(lens)
    offs = [0] + list(np.cumsum(n))
    q = torch.randn((offs[-1], hq, D), device="cuda").bfloat16()
    o, lse = check_attention(pool, q, offs, lens, seen)
    assert bool((o[offs[2]:offs[4]] == 0).all()) and bool((lse[offs[2]:offs[4]] == float("-inf")).all())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,slack", [(8, 2, 0), (16, 1, 0), (5, 5, 0), (8, 2, 200000), (32, 8, 200000)])
def test_masks_of_large_trees_that_end_early(kind, hq, hkv, slack):
    """Row tiles whose nodes see nothing behind some key, or nothing at all, or only the last; whole items and runs."""
    rng = np.random.RandomState(11)
    n, lens = [300, 300, 129, 700, 257], [300, 1500, 129, 701, 600]
    seen = [np.tril(rng.random_sample((k, k)) < 0.2) for k in n]
    seen[0][:, 40:] = False
    seen[0][::7] = False
    seen[1][:200] = False            # the keys before the tree only
    seen[2][:] = False               # nothing
    seen[3][5:9, 699] = True
    seen[3][:, 650:] &= rng.random_sample((700, 50)) < 0.02
    seen[4][:, 128:] = False
    pool = Pool(kind, hkv, lens, extra_pages=slack // 16)
    pool.fill(lens)
    offs = [0] + list(np.cumsum(n))
    q = torch.randn((offs[-1], hq, D), device="cuda").bfloat16()
    check_attention(pool, q, offs, lens, seen, slack=slack)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 6, 20, 60])
@pytest.mark.parametrize("q_scale,scale", [(60.0, None), (1e-4, None), (1.0, 1.5), (3e4, 1e-6)])
def test_attention_score_ranges(kind, n, q_scale, scale):
    """Sharp softmaxes (one key takes all), flat ones, other score factors, queries outside fp16's range."""
    lens = [n + 90, n + 333]
    pool = Pool(kind, 2, lens)
    pool.fill(lens)
    q = (torch.randn((2 * n, 8, D), device="cuda") * q_scale).bfloat16()
    if q_scale == 3e4:
        q[0, 0, 3] = 3e5
        q[1, 5] = 0
    rng = np.random.RandomState(1)
    check_attention(pool, q, [0, n, 2 * n], lens, [ancestors(random_parents(rng, n)) for _ in lens], scale)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rising", [True, False])
def test_attention_scores_that_rise_or_fall_along_the_keys(kind, rising):
    """Every block of keys moves the maximum, or none but the first."""
    n, lens = [7, 30], [2500, 1300]
    pool = Pool(kind, 2, lens)
    pool.fill(lens, k_scale=0.05)
    q = torch.randn((37, 8, D), device="cuda").abs().bfloat16() + 1
    for b, m in enumerate(lens):
        pos = torch.arange(m, device="cuda")
        page, slot = pool.table[b, pos // PAGE].long(), pos % PAGE
        lift = (pos if rising else m - pos).float()[:, None, None] / m * 2
        if kind == "bf16":
            pool.k[page, :, slot] = (pool.k[page, :, slot].float() + lift).bfloat16()
        else:
            pool.ks[page, :, slot] = 122
            pool.k[page, :, slot] = (lift.expand(-1, 2, D) * 32).to(torch.float8_e4m3fn).view(torch.uint8)
    rng = np.random.RandomState(1)
    check_attention(pool, q, [0, 7, 37], lens, [ancestors(random_parents(rng, k)) for k in n])


@pytest.mark.parametrize("n", [1, 20])
def test_attention_e4m3_scales_of_all_sizes(n):
    """Value rows whose powers of two differ by 2^100; key rows by 2^20."""
    lens = [n + 90, n + 333]
    pool = Pool("e4m3", 2, lens)
    pool.fill(lens)
    g = torch.Generator(device="cuda").manual_seed(2)
    pool.vs.copy_(torch.randint(40, 140, pool.vs.shape, generator=g, device="cuda").to(torch.uint8))
    pool.ks.copy_(torch.randint(100, 121, pool.ks.shape, generator=g, device="cuda").to(torch.uint8))
    q = torch.randn((2 * n, 8, D), device="cuda").bfloat16()
    rng = np.random.RandomState(1)
    check_attention(pool, q, [0, n, 2 * n], lens, [ancestors(random_parents(rng, n)) for _ in lens])


@pytest.mark.parametrize("n", [1, 24, 100])
def test_attention_takes_every_e4m3_code(n):
    """Keys and values of every finite code, subnormals included."""
    lens = [n + 256]
    pool = Pool("e4m3", 1, lens)
    pool.fill(lens)
    finite = [c for c in range(256) if c & 127 != 127]
    codes = torch.tensor(finite, dtype=torch.uint8, device="cuda")
    pos = torch.arange(lens[0], device="cuda")
    page, slot = pool.table[0, pos // PAGE].long(), pos % PAGE
    pool.v[page, 0, slot] = codes[(pos[:, None] * 7 + torch.arange(D, device="cuda")) % 254]
    pool.k[page, 0, slot] = codes[(pos[:, None] * 5 + 3 * torch.arange(D, device="cuda")) % 254]
    pool.vs[:], pool.ks[:] = 121, 118
    q = (torch.randn((n, 4, D), device="cuda") * 0.05).bfloat16()
    rng = np.random.RandomState(1)
    check_attention(pool, q, [0, n], lens, [ancestors(random_parents(rng, n))])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [5, 40])
def test_nan_and_infinity_stay_in_their_rows(kind, n):
    """A query row that is not a number, or not finite, makes its own row NaN and no other."""
    lens = [n + 40, n + 300]
    pool = Pool(kind, 2, lens)
    pool.fill(lens)
    q = torch.randn((2 * n, 8, D), device="cuda").bfloat16()
    q[1, 3, 5] = float("nan")
    q[n + 2, 0, 0] = float("inf")
    q[n + 3, 7, 127] = float("-inf")
    rng = np.random.RandomState(1)
    seen = [ancestors(random_parents(rng, n)) for _ in lens]
    out, lse = attend(pool, q, [0, n, 2 * n], lens, seen)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    bad[1, 3] = bad[n + 2, 0] = bad[n + 3, 7] = True
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    q[bad] = 0
    o, z, tol_o, tol_l = attention_64(pool, q, [0, n, 2 * n], lens, seen, D ** -0.5)
    assert bool(((out.double() - o).abs() <= tol_o)[~bad].all())
    assert bool(((lse.double() - z).abs() <= tol_l)[~bad].all())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [5, 40])
def test_nan_keys_and_values_in_the_cache(kind, n):
    """A key that is not a number makes NaN of the rows that see it and of no other sequence's or head's; a value that
    is not one, of its dim."""
    lens = [n + 130, n + 300]
    pool = Pool(kind, 2, lens)
    pool.fill(lens)
    rng = np.random.RandomState(1)
    seen = [ancestors(random_parents(rng, n)) for _ in lens]
    nan = 0x7F if kind == "e4m3" else float("nan")
    at = lambda b, p: (int(pool.table[b, p // PAGE]), p % PAGE)  # noqa: E731
    page, slot = at(0, 17)
    pool.v[page, 1, slot, 9] = nan
    page, slot = at(1, n + 299)  # the last node's key
    pool.k[page, 0, slot, 3] = nan
    q = torch.randn((2 * n, 8, D), device="cuda").bfloat16()
    out, lse = attend(pool, q, [0, n, 2 * n], lens, seen)
    want = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    want[:n, 4:, 9] = True
    sees = torch.from_numpy(seen[1][:, n - 1]).cuda()
    want[n:, :4][sees] = True
    assert torch.equal(out.isnan(), want)
    assert torch.equal(lse.isnan(), want.all(-1))


def test_large_pool_offsets():
    """Pages whose element offsets pass 2^31."""
    import trie_label_scoring_gb300 as Q
    first = (1 << 32) // (16 * 128 * 8) + 5  # elements
    pool = Pool("bf16", 8, [200, 33], first_page=first)
    pool.fill([200, 33])
    q = torch.randn((9, 32, D), device="cuda").bfloat16()
    rng = np.random.RandomState(1)
    check_attention(pool, q, [0, 6, 9], [200, 33], [ancestors(random_parents(rng, k)) for k in (6, 3)])
    del pool
    torch.cuda.empty_cache()
    assert Q.launch_count() > 0


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("what", ["page", "length", "short", "offsets", "many"])
def test_attention_reports_bad_indices(n, what):
    """A bad sequence is reported and void; the others' rows are right."""
    import trie_label_scoring_gb300 as Q
    lens = [n + 30, n + 200, n + 64]
    pool = Pool("bf16", 2, lens)
    pool.fill(lens)
    rng = np.random.RandomState(1)
    seen = [ancestors(random_parents(rng, n)) for _ in lens]
    offs, given = [0, n, 2 * n, 3 * n], list(lens)
    q = torch.randn((3 * n, 8, D), device="cuda").bfloat16()
    words, max_q = (n + 31) // 32, n
    o, z, tol_o, tol_l = attention_64(pool, q, offs, lens, seen, D ** -0.5)
    if what == "page":
        pool.table[1, 2] = pool.pages
    if what == "length":
        given[1] = max(lens) + 1
    if what == "short":
        given[1] = n - 1
    if what == "offsets":
        offs[1] = -3
    if what == "many":
        offs[2], offs[1] = 2 * n, n - 1
    mask = i32(np.concatenate([pack(s, words) for s in seen]))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    ws = torch.empty(Q.workspace_size_attention_tree(pool.cache, 8, 3 * n, max_q, max(lens)), dtype=torch.uint8, device="cuda")
    Q.attention_tree(pool.cache, q, i32(offs), i32(given), mask, max_q, max(lens), out, ws, lse=lse)
    with pytest.raises(Q.QuailError) as e:
        Q.device_status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    good = slice(2 * n, 3 * n)
    assert bool(((out.double() - o).abs() <= tol_o)[good].all())
    if what != "offsets" and what != "many":
        assert bool(((out.double() - o).abs() <= tol_o)[:n].all())
    status()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("limit", [-1, 200])
@pytest.mark.parametrize("n,hq,hkv,lens", [(3, 8, 2, [40, 300]), (8, 8, 2, [700] * 3), (16, 32, 8, [3000] * 24),
                                           (24, 32, 8, [2000] * 9), (3, 128, 1, [5000] * 2), (100, 16, 4, [2500] * 5)])
def test_waits_that_run_out_are_reported(kind, limit, n, hq, hkv, lens):
    """Every width of tile, whole items and runs: a wait that gives up is reported and ends the call; the next one is right."""
    import trie_label_scoring_gb300 as Q
    pool = Pool(kind, hkv, lens)
    pool.fill(lens)
    rng = np.random.RandomState(1)
    seen = [ancestors(random_parents(rng, n)) for _ in lens]
    offs = [n * b for b in range(len(lens) + 1)]
    q = torch.randn((offs[-1], hq, D), device="cuda").bfloat16()
    attend(pool, q, offs, lens, seen)
    Q._test_set_pipeline_wait_limit(limit)
    try:
        # 200 cycles are not sure to run out, below 0 is
        try:
            attend(pool, q, offs, lens, seen)
            gave_up = False
        except Q.QuailError as e:
            assert e.name == "QUAIL_ERR_DEVICE_TIMEOUT"
            gave_up = True
    finally:
        Q._test_set_pipeline_wait_limit(0)
    assert gave_up or limit > 0
    check_attention(pool, q, offs, lens, seen)


def test_two_ways_of_carrying_out_a_call_agree():
    """Bounds far above the lengths take a call from whole items to runs of the work list: the same results."""
    rng = np.random.RandomState(5)
    n, lens = [9, 0, 30, 1], [500, 0, 260, 0]
    seen = [ancestors(random_parents(rng, k)) if k else np.zeros((0, 0), dtype=bool) for k in n]
    for kind in ("bf16", "e4m3"):
        pool = Pool(kind, 2, lens, extra_pages=4000)
        pool.fill(lens)
        offs = [0] + list(np.cumsum(n))
        q = torch.randn((offs[-1], 8, D), device="cuda").bfloat16()
        check_attention(pool, q, offs, lens, seen)
        check_attention(pool, q, offs, lens, seen, slack=60000)
        check_attention(pool, q, offs, lens, seen, slack=60000, more=500)


# ------------------------------------------------------------------ the verdict
def verdict(parent, draft, taken):
    node, path = 0, [0] if parent else []
    while path:
        nxt = [i for i in range(node + 1, len(parent)) if parent[i] == node and draft[i] == taken[node]]
        if not nxt:
            break
        node = nxt[0]
        path.append(node)
    return path


def drafted(rng, n, hit=0.7, vocab=50):
    """A random tree and tokens, of which about `hit` continue their parent as taken; siblings of the same token among them."""
    parent = random_parents(rng, n, back=5, roots=0.03)
    taken = rng.randint(0, vocab, n)
    draft = [int(taken[p]) if p >= 0 and rng.random_sample() < hit else int(rng.randint(vocab)) for p in parent]
    return parent, draft, taken.tolist()


@pytest.mark.parametrize("kind,hkv,layers", [("bf16", 2, 1), ("e4m3", 2, 1), ("bf16", 8, 3), ("e4m3", 8, 5), ("bf16", 1, 130),
                                             ("e4m3", 5, 129), ("bf16", 2, 0)])
@pytest.mark.parametrize("sizes", [[1], [8, 0, 8, 5], [40, 64, 33, 1], [1000, 3]])
def test_accept(kind, hkv, layers, sizes):
    import trie_label_scoring_gb300 as Q
    rng = np.random.RandomState(sum(sizes) + layers)
    trees = [drafted(rng, n) for n in sizes]
    trees[0] = (list(range(-1, sizes[0] - 1)), [3] * sizes[0], [3] * sizes[0])  # all of a chain
    past = [int(x) for x in rng.randint(0, 40, len(sizes))]
    lens = [p + n for p, n in zip(past, sizes)]
    offs = [0] + list(np.cumsum(sizes))
    T, max_q = offs[-1], max(sizes) + (sum(sizes) % 2)
    words = (max_q + 31) // 32
    pools = []
    for i in range(layers):
        p = Pool(kind, hkv, lens, seed=1)
        p.fill(lens, seed=i)
        pools.append(p)
    caches = [Q.KVCache(p.k, p.v, pools[0].table, p.ks, p.vs) for p in pools]
    mask, rope = torch.zeros((T, words), dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    parent, draft, taken = (i32(sum((list(t[k]) for t in trees), [])) for k in range(3))
    d_offs, d_lens = i32(offs), i32(lens)
    Q.tree_plan(parent, d_offs, d_lens, max_q, mask, rope)
    path = torch.full((T,), 99, dtype=torch.int32, device="cuda")
    accepted, new_len, bonus = (torch.full((len(sizes),), 99, dtype=torch.int32, device="cuda") for _ in range(3))
    want = [[x.clone() for x in (p.k, p.v, p.ks, p.vs) if x is not None] for p in pools]
    paths = [verdict(*t) for t in trees]
    for b, way in enumerate(paths):
        for d, i in enumerate(way):
            src, dst = past[b] + i, past[b] + d
            ps, pd = (int(pools[0].table[b, x // PAGE]) if pools else 0 for x in (src, dst))
            for xs in want:
                for x in xs:
                    x[pd, :, dst % PAGE] = x[ps, :, src % PAGE]
    Q.tree_accept(caches, parent, mask, draft, taken, d_offs, d_lens, max_q, path, accepted, new_len, bonus)
    status()
    assert accepted.tolist() == [len(w) for w in paths]
    assert new_len.tolist() == [p + len(w) for p, w in zip(past, paths)]
    assert path.tolist() == sum((w + [-1] * (n - len(w)) for w, n in zip(paths, sizes)), [])
    assert bonus.tolist() == [t[2][w[-1]] if w else -1 for t, w in zip(trees, paths)]
    raw = torch.uint8 if kind == "e4m3" else torch.int16
    for p, xs in zip(pools, want):
        for x, y in zip([x for x in (p.k, p.v, p.ks, p.vs) if x is not None], xs):
            assert torch.equal(x.view(raw), y.view(raw))


@pytest.mark.parametrize("what", ["page", "offsets", "length"])
def test_accept_reports_bad_indices(what):
    import trie_label_scoring_gb300 as Q
    n, past = 6, 20
    lens, offs = [past + n] * 3, [0, n, 2 * n, 3 * n]
    pool = Pool("bf16", 2, lens)
    pool.fill(lens)
    before = pool.k.clone()
    parent, draft, taken = [-1, 0, 0, 2, 3, 3], [0, 9, 1, 2, 9, 3], [1, 0, 2, 3, 0, 7]
    d = [i32(x * 3) for x in (parent, draft, taken)]
    mask = i32(np.concatenate([pack(ancestors(parent), 1)] * 3))
    given = list(lens)
    if what == "page":
        pool.table[1, past // PAGE] = -1
    if what == "offsets":
        offs[1] = 2 * n + 1
    if what == "length":
        given[1] = n - 1
    path = torch.full((3 * n,), 99, dtype=torch.int32, device="cuda")
    accepted, new_len, bonus = (torch.full((3,), 99, dtype=torch.int32, device="cuda") for _ in range(3))
    Q.tree_accept([pool.cache], d[0], mask, d[1], d[2], i32(offs), i32(given), n, path, accepted, new_len, bonus)
    with pytest.raises(Q.QuailError) as e:
        Q.device_status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    assert accepted.tolist()[2] == 4 and path.tolist()[2 * n:] == [0, 2, 3, 5, -1, -1]
    if what != "page":
        assert accepted.tolist()[1] == 99
    seq = i32([1] * n)
    if what != "page":  # the second sequence's rows are where they were
        pos = i32(range(past, past + n))
        page, slot = pool.table[seq.long(), pos.long() // PAGE].long(), pos.long() % PAGE
        assert torch.equal(pool.k[page, :, slot], before[page, :, slot])
    seq, pos = i32([2] * 4), i32(range(past, past + 4))
    page, slot = pool.table[seq.long(), pos.long() // PAGE].long(), pos.long() % PAGE
    src = i32([past + i for i in (0, 2, 3, 5)]).long()
    assert torch.equal(pool.k[page, :, slot], before[pool.table[2, src // PAGE].long(), :, src % PAGE])


# ------------------------------------------------------------------ together
class Toy:
    """One attention layer over random tables of a token's q, k, v; the next token is the likeliest of o W."""

    def __init__(self, vocab=61, hq=8, hkv=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.vocab = hq, hkv, vocab
        self.qkv = torch.randn((vocab, (hq + 2 * hkv) * D), generator=g, device="cuda").bfloat16()
        self.w = torch.randn((hq * D, vocab), generator=g, device="cuda", dtype=torch.float64)

    def next64(self, tokens):
        """The next token after each, token by token in 64 bits, and how clearly it leads."""
        x = self.qkv[tokens].double().reshape(len(tokens), -1, D)
        ang = torch.arange(len(tokens), device="cuda").double()[:, None] * 1e4 ** (-torch.arange(0, 64, 2, device="cuda").double() / 64)
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        y = x[:, :self.hq + self.hkv].clone()
        a, b = y[..., 0:64:2].clone(), y[..., 1:64:2].clone()
        y[..., 0:64:2], y[..., 1:64:2] = a * c - b * s, b * c + a * s
        G = self.hq // self.hkv
        q, k, v = y[-1, :self.hq].reshape(self.hkv, G, D), y[:, self.hq:], x[:, self.hq + self.hkv:]
        p = torch.softmax(torch.einsum("hgd,khd->hgk", q, k) / D ** 0.5, -1)
        top = torch.topk(torch.einsum("hgk,khd->hgd", p, v).reshape(-1) @ self.w, 2)
        return int(top.indices[0]), float(top.values[0] - top.values[1])


def test_decoding_with_trees_is_decoding_token_by_token():
    """Documents are admitted, trees drafted, cached, attended to, judged and cut back, pages and all, in captured
    steps; what comes out is what one token after the other gives."""
    import trie_label_scoring_gb300 as Q
    toy, B, n, hq, hkv = Toy(), 5, 9, 8, 2
    rng = np.random.RandomState(0)
    rope = Q.Rope(1e4, "interleaved", 64)
    # o is within 2^-7 of itself, element by element, so a logit, a sum of 1,024 of them of size 1 and less with
    # random signs, is within about 32 * 2^-7 = 0.25: texts are drawn until every step leads by more
    for seed in range(100):
        draw = np.random.RandomState(seed)
        texts = [draw.randint(0, toy.vocab, k).tolist() for k in (30, 1, 17, 64, 47)]
        truth, lead = [list(x) for x in texts], []
        for seq in truth:
            for _ in range(14):
                nxt, by = toy.next64(seq)
                lead.append(by)
                seq.append(nxt)
        if min(lead) > 0.25:
            break
    assert min(lead) > 0.25
    t = Tables(B, 40, 12, seed=1)
    pool = torch.full((40, hkv, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vpool = torch.full_like(pool, float("nan"))
    cache = Q.KVCache(pool, vpool, t.d_table)
    old, new, granted = (i32([0] * B) for _ in range(3))
    offs, qoffs = i32([0] * (B + 1)), i32([n * b for b in range(B + 1)])

    def rows(token, seq, pos, rope_pos, q):
        Q.cache_append_rope(cache, toy.qkv[token.long()], hq, seq, pos, rope, rope_pos=rope_pos, q_out=q)

    # all but a text's last token is prefilled; that one is the first tree's root
    lens = [len(x) - 1 for x in texts]
    seq, pos = i32([0] * sum(lens)), i32([0] * sum(lens))
    new.copy_(i32(lens))
    Q.cache_resize(cache, old, new, t.ring, t.state, granted, offs, seq, pos)
    rows(i32(sum((x[:-1] for x in texts), [])), seq, pos, None, None)
    status()
    old.copy_(granted)

    T = B * n
    parent, draft = i32([-1] * T), i32([0] * T)
    mask, rope_pos, taken, path = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(4))
    mask = mask[:, None].contiguous()
    tseq, tpos = i32([0] * T), i32([0] * T)
    accepted, new_len, bonus = (i32([0] * B) for _ in range(3))
    q = torch.zeros((T, hq, D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.zeros(Q.workspace_size_attention_tree(cache, hq, T, n, 12 * PAGE), dtype=torch.uint8, device="cuda")
    cut = i32([0] * (B + 1))

    def step():
        torch.add(old, n, out=new)
        Q.cache_resize(cache, old, new, t.ring, t.state, granted, offs, tseq, tpos)
        Q.tree_plan(parent, qoffs, granted, n, mask, rope_pos)
        rows(draft, tseq, tpos, rope_pos, q)
        Q.attention_tree(cache, q, qoffs, granted, mask, n, 12 * PAGE, out, ws)
        taken.copy_((out.double().reshape(T, -1) @ toy.w).argmax(-1))
        Q.tree_accept([cache], parent, mask, draft, taken, qoffs, granted, n, path, accepted, new_len, bonus)
        Q.cache_resize(cache, granted, new_len, t.ring, t.state, old, cut)

    got = [list(x) for x in texts]
    graph, steps = None, 0
    while min(len(g) - len(x) for g, x in zip(got, texts)) < 10:
        trees = []
        for g, full in zip(got, truth):
            # a tree whose nodes often, not always, are what comes next
            par, tok, deep = [-1], [g[-1]], [0]
            for i in range(1, n):
                p = int(rng.randint(max(0, i - 3), i))
                at = len(g) + deep[p]
                tok.append(full[at] if at < len(full) and rng.random_sample() < 0.6 else int(rng.randint(toy.vocab)))
                par.append(p)
                deep.append(deep[p] + 1)
            trees.append((par, tok))
        parent.copy_(i32(sum((x[0] for x in trees), [])))
        draft.copy_(i32(sum((x[1] for x in trees), [])))
        if steps == 0:
            step()
        elif steps == 1:
            saved = [x.clone() for x in (old, t.ring, t.state, t.d_table)]
            graph = torch.cuda.CUDAGraph()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
                step()
            for x, y in zip(saved, (old, t.ring, t.state, t.d_table)):
                assert torch.equal(x, y)  # a capture runs nothing
            graph.replay()
        else:
            graph.replay()
        status()
        for b in range(B):
            k = int(accepted[b])
            ways = path[b * n:b * n + k].tolist()
            got[b] += [trees[b][1][i] for i in ways[1:]] + [int(bonus[b])]
        assert old.tolist() == [len(g) - 1 for g in got]
        steps += 1
        assert steps < 40
    for g, full in zip(got, truth):
        m = min(len(g), len(full))
        assert g[:m] == full[:m]
    # nothing leaked: the free pages and the tables' are all there are, each once
    head, count, _, _ = t.state.tolist()
    free = t.ring[(head + torch.arange(count, device="cuda")) % 40].tolist()
    used = [p for r, x in zip(t.d_table.tolist(), old.tolist()) for p in r[:-(-x // PAGE)]]
    assert sorted(free + used) == list(range(40))


def test_a_label_trie_is_a_tree():
    """The trie of a label set as every document's tree: its nodes' masks and positions."""
    import trie_label_scoring_gb300 as Q
    rng = np.random.RandomState(0)
    labels = {tuple(rng.randint(0, 9, rng.randint(1, 6))) for _ in range(120)}
    trie = Q.Trie([list(map(int, x)) for x in labels], 3, 300)
    view = trie.view()
    n = trie.n_nodes
    assert 32 < n < 1024
    mask, rope = torch.zeros((2 * n, (n + 31) // 32), dtype=torch.int32, device="cuda"), torch.zeros(2 * n, dtype=torch.int32, device="cuda")
    Q.tree_plan(i32(np.tile(view["parent"], 2)), i32([0, n, 2 * n]), i32([n + 100, n + 7]), n, mask, rope)
    status()
    assert np.array_equal(mask.cpu().numpy(), np.tile(pack(ancestors(view["parent"].tolist()), (n + 31) // 32), (2, 1)))
    assert rope.tolist() == (view["depth"] + 100).tolist() + (view["depth"] + 7).tolist()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_two_streams_and_a_shared_workspace_in_turn(kind):
    """Calls on two streams with a workspace each, and two captured graphs that use one after the other."""
    import trie_label_scoring_gb300 as Q
    rng = np.random.RandomState(2)
    jobs = []
    for i, (n, lens, hq, hkv) in enumerate([([9, 3], [2000, 700], 32, 8), ([40], [5000], 16, 1)]):
        pool = Pool(kind, hkv, lens, seed=i)
        pool.fill(lens)
        offs = [0] + list(np.cumsum(n))
        seen = [ancestors(random_parents(rng, k)) for k in n]
        q = torch.randn((offs[-1], hq, D), device="cuda").bfloat16()
        want = attention_64(pool, q, offs, lens, seen, D ** -0.5)
        words = (max(n) + 31) // 32
        size = Q.workspace_size_attention_tree(pool.cache, hq, offs[-1], max(n), max(lens))
        jobs.append((pool, q, i32(offs), i32(lens), i32(np.concatenate([pack(s, words) for s in seen])), max(n), max(lens),
                     torch.zeros_like(q), size, torch.zeros(q.shape[:2], device="cuda"), want))

    def call(j, ws, stream=None):
        pool, q, offs, lens, mask, max_q, max_len, out, _, lse, _ = j
        Q.attention_tree(pool.cache, q, offs, lens, mask, max_q, max_len, out, ws, lse=lse, stream=stream)

    def right():
        torch.cuda.synchronize()
        status()
        for j in jobs:
            out, lse, (o, z, tol_o, tol_l) = j[7], j[9], j[10]
            assert bool(((out.double() - o).abs() <= tol_o).all()) and bool(((lse.double() - z).abs() <= tol_l).all())
            out.zero_()
            lse.zero_()
        torch.cuda.synchronize()

    own_ws = [torch.full((j[8],), 0xFF, dtype=torch.uint8, device="cuda") for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        for j, ws, s in zip(jobs, own_ws, streams):
            call(j, ws, s)
    right()
    shared = torch.full((max(j[8] for j in jobs),), 0xFF, dtype=torch.uint8, device="cuda")
    graphs = []
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(j, shared)
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    right()


def test_python_checks_of_tensors():
    import trie_label_scoring_gb300 as Q
    pool = Pool("bf16", 2, [40])
    q = torch.zeros((4, 8, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(Q.workspace_size_attention_tree(pool.cache, 8, 4, 4, 40), dtype=torch.uint8, device="cuda")
    good = dict(q=q, q_offsets=i32([0, 4]), seq_len=i32([40]), mask=i32([[1]] * 4), out=torch.zeros_like(q), workspace=ws)
    bad = [dict(q=q.float()), dict(q=torch.zeros((4, 8, 64), dtype=torch.bfloat16, device="cuda")), dict(q_offsets=i32([0])),
           dict(q_offsets=torch.tensor([0, 4], device="cuda")), dict(seq_len=i32([40, 1])), dict(mask=i32([[1]] * 3)),
           dict(mask=i32([[1]] * 4).cpu()), dict(out=torch.zeros_like(q).transpose(0, 1)), dict(workspace=ws[:128].clone()),
           dict(workspace=ws.view(torch.int32))]
    for b in bad:
        kw = {**good, **b}
        with pytest.raises(Q.QuailError):
            Q.attention_tree(pool.cache, kw["q"], kw["q_offsets"], kw["seq_len"], kw["mask"], 4, 40, kw["out"], kw["workspace"])
    Q.attention_tree(pool.cache, *[good[k] for k in ("q", "q_offsets", "seq_len", "mask")], 4, 40, good["out"], ws)
    torch.cuda.synchronize()
    with pytest.raises(Q.QuailError):
        Q.tree_plan(i32([-1]).cpu(), i32([0, 1]), i32([1]), 1, i32([[0]]), i32([0]))
    with pytest.raises(Q.QuailError):
        Q.tree_plan(i32([-1]), i32([0, 1]), i32([1]), 33, i32([[0]]), i32([0]))  # two words a row
    with pytest.raises(Q.QuailError):
        Q.cache_resize(pool.cache, i32([0]), i32([1]), i32([0]), i32([0] * 4), i32([0]), i32([0, 0]))  # the ring is the pool's size
