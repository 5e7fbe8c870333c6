"""The document cache on the GPU against plain 64-bit arithmetic: writing it
(per-head norm, rotation, bf16 or e4m3), reading it back, and attention for
sequences that share a prefix.

Tolerances. A rounding to bf16 is off by at most 2^-8 of the value. The fp32
work before it: a rotated element mixes two normed ones with a cosine and a
sine that are within 1e-6 of their values, so 2e-6 times the pair's sizes.
e4m3 rounds within 2^-4 of the value, or half its smallest step, 2^-10 of the
row's power of two. Attention rounds every weight to bf16 before the product
with V (2^-8 of sum p|v|) and the result to bf16 (2^-8 |o|); a score is an
fp32 sum of 128 exact products, so it is within 128 * 2^-24 * sum |q||k| of its
value, and a weight within twice that relative to itself (numerator and sum).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

D, PAGE = 128, 16
GAMMA = 128 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    import trie_label_scoring_gb300 as Q
    Q.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)


class Pool:
    """A pool of shuffled pages whose every slot starts as NaN, and a table of the sequences' pages."""

    def __init__(self, kind, hkv, lens, prefix=0, seed=0, spare=3, extra_pages=0, first_page=0):
        import trie_label_scoring_gb300 as Q
        rng = np.random.RandomState(seed)
        pp = prefix // PAGE
        need = [max(0, -(-n // PAGE) - pp) for n in lens]
        total = pp + sum(need) + spare
        perm = first_page + rng.permutation(total)
        table = np.full((len(lens), max(1, pp + max(need, default=0)) + extra_pages), -7, dtype=np.int32)
        at = pp
        for i, k in enumerate(need):
            table[i, :pp] = perm[:pp]
            table[i, pp:pp + k] = perm[at:at + k]
            at += k
        self.pages = first_page + total
        self.kind, self.hkv = kind, hkv
        self.table = torch.from_numpy(table).cuda()
        self.prefix_pages = torch.from_numpy(perm[:pp].astype(np.int32)).cuda()
        shape = (self.pages, hkv, PAGE, D)
        if kind == "bf16":
            self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            self.v = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            self.ks = self.vs = None
        else:
            self.k = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
            self.v = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
            self.ks = torch.full(shape[:3], 200, dtype=torch.uint8, device="cuda")
            self.vs = torch.full(shape[:3], 200, dtype=torch.uint8, device="cuda")
        self.cache = Q.KVCache(self.k, self.v, self.table, self.ks, self.vs)

    def rows(self, seq, pos, name):
        """The cached rows of (seq, pos) in 64 bits, [n, hkv, 128]."""
        page = self.table[seq.long(), pos.long() // PAGE].long()
        return self._rows(name, page, pos.long() % PAGE)

    def _rows(self, name, page, slot):
        x = (self.k if name == "k" else self.v)[page, :, slot]
        if self.kind == "bf16":
            return x.double()
        e = (self.ks if name == "k" else self.vs)[page, :, slot].double()
        return x.view(torch.float8_e4m3fn).double() * torch.exp2(e - 127)[..., None]

    def fill(self, lens, seed=1, k_scale=1.0, v_scale=1.0):
        """Random rows at every position of every sequence (shared pages once), in the pool's own format."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pos = torch.arange(n, device="cuda")
            page, slot = self.table[b, pos // PAGE].long(), pos % PAGE
            for pool, sc, f in ((self.k, self.ks, k_scale), (self.v, self.vs, v_scale)):
                x = torch.randn((n, self.hkv, D), generator=g, device="cuda") * f
                if self.kind == "bf16":
                    pool[page, :, slot] = x.bfloat16()
                else:
                    e = torch.randint(118, 122, (n, self.hkv), generator=g, device="cuda")
                    pool[page, :, slot] = (x * torch.exp2(127.0 - e)[..., None]).clamp(-448, 448).to(
                        torch.float8_e4m3fn).view(torch.uint8)
                    sc[page, :, slot] = e.to(torch.uint8)


def tokens(lens, first=None):
    first = first or [0] * len(lens)
    seq = np.concatenate([np.full(n - f, i) for i, (n, f) in enumerate(zip(lens, first))]).astype(np.int32)
    pos = np.concatenate([np.arange(f, n) for n, f in zip(lens, first)]).astype(np.int32)
    return torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()


def status():
    import trie_label_scoring_gb300 as Q
    Q.device_status()


# ------------------------------------------------------------------ append
def expected_rows(qkv, pos, hq, hkv, gq, gk, eps, theta):
    """q, k, v in 64 bits and how far the fp32 work may take each element."""
    x = qkv[:, :(hq + 2 * hkv) * D].double().reshape(qkv.shape[0], -1, D)
    out = []
    for part, g, turn in ((x[:, :hq], gq, True), (x[:, hq:hq + hkv], gk, True), (x[:, hq + hkv:], None, False)):
        if g is not None:
            part = part / torch.sqrt((part ** 2).mean(-1, keepdim=True) + eps) * g.double()
        a, b = part[..., :64], part[..., 64:]
        slack = 2e-6 * torch.cat([a.abs() + b.abs()] * 2, -1)
        if turn and theta:
            ang = pos.double()[:, None] * theta ** (-torch.arange(64, device="cuda").double() / 64)
            c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
            part = torch.cat([a * c - b * s, b * c + a * s], -1)
        out.append((part, slack if turn else torch.zeros_like(slack)))
    return out


def check_stored(got, want, slack, scale_exp=None):
    err = (got - want).abs()
    if scale_exp is None:
        tol = 2.0 ** -8 * want.abs() + slack * 1.01
    else:
        unit = torch.exp2(scale_exp.double() - 127)[..., None]
        tol = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * unit) + slack * 1.1
        amax = want.abs().amax(-1)
        m, e = torch.frexp(amax / 448)
        e = torch.clamp(e - (m == 0.5).int(), min=-100) + 127
        at_border = (m - 0.5).abs() < 1e-5  # the fp32 maximum may fall on the other side
        at_border |= (m - 1.0).abs() < 1e-5
        assert bool((((scale_exp - e) == 0) | at_border | (amax == 0)).all())
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv,norm,theta,pad", [(8, 2, True, 1e6, 0), (32, 8, True, 1e6, 8), (5, 5, True, 1e4, 136),
                                                   (16, 1, False, 1e6, 0), (12, 3, True, 0.0, 0), (0, 2, False, 0.0, 0)])
def test_append(kind, src, hq, hkv, norm, theta, pad):
    import trie_label_scoring_gb300 as Q
    first, lens = [0, 15, 100, 3, 4000], [1, 18, 117, 3, 4033]
    seq, pos = tokens(lens, first)
    order = torch.randperm(seq.numel(), generator=torch.Generator().manual_seed(3)).cuda()
    seq, pos = seq[order].contiguous(), pos[order].contiguous()  # tokens in any order
    T = seq.numel()
    pool = Pool(kind, hkv, lens, extra_pages=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn((T, (hq + 2 * hkv) * D + pad), generator=g, device="cuda").to(src)
    wide[1] *= 1e-3
    wide[2] *= 300
    wide[3] = 0
    gq = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() if norm else None
    gk = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() if norm else None
    q = torch.full((T, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    before = [t.clone() for t in (pool.k, pool.v)]
    Q.cache_append(pool.cache, wide, hq, seq, pos, q_out=q, q_norm=gq, k_norm=gk, rms_eps=1e-6, rope_theta=theta)
    status()
    (wq, sq), (wk, sk), (wv, sv) = expected_rows(wide, pos, hq, hkv, gq, gk, 1e-6, theta)
    check_stored(q.double(), wq, sq)
    page, slot = pool.table[seq.long(), pos.long() // PAGE].long(), pos.long() % PAGE
    for name, want, slack, sc in (("k", wk, sk, pool.ks), ("v", wv, sv, pool.vs)):
        check_stored(pool.rows(seq, pos, name), want, slack, None if sc is None else sc[page, :, slot])
    touched = torch.zeros(pool.k.shape[:3], dtype=torch.bool, device="cuda")
    touched[page, :, slot] = True
    for old, new in zip(before, (pool.k, pool.v)):  # everything else as it was
        a, b = old.view(torch.uint8 if kind == "e4m3" else torch.int16), new.view(torch.uint8 if kind == "e4m3" else torch.int16)
        assert torch.equal(a[~touched], b[~touched])


def test_append_skips_padding_and_leaves_its_rows():
    import trie_label_scoring_gb300 as Q
    pool = Pool("bf16", 2, [20, 20])
    seq = torch.tensor([0, -1, 1, -1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([19, 5, 0, -3], dtype=torch.int32, device="cuda")
    qkv = torch.randn((4, 8 * D), device="cuda")
    q = torch.full((4, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    Q.cache_append(pool.cache, qkv, 4, seq, pos, q_out=q)
    status()
    assert bool((q[1] == 7).all()) and bool((q[3] == 7).all())
    assert torch.equal(q[0], qkv[0, :4 * D].view(4, D).bfloat16())
    assert int((~pool.k.isnan()).all(-1).sum()) == 4  # two tokens x two heads


def test_append_e4m3_rounds_each_code_as_the_format_does():
    """Every finite code times every power of two in reach comes back bit for bit, and midpoints go to even."""
    import trie_label_scoring_gb300 as Q
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    vals = codes.view(torch.float8_e4m3fn).float()
    vals = vals[vals.isfinite()]  # 254 values
    pos_vals = torch.unique(vals.abs())  # ascending
    mids = (pos_vals[1:] + pos_vals[:-1]) / 2
    rows = []
    for e in (-90, -20, 0, 30, 100):
        for block in (vals[:126], vals[126:252], mids):
            r = torch.zeros(D, device="cuda")
            r[:block.numel()] = block
            r[127] = 448  # fixes the row's power of two
            rows.append(r * 2.0 ** e)
    x = torch.stack(rows)
    T = x.shape[0]
    pool = Pool("e4m3", 1, [T])
    seq, pos = tokens([T])
    out = torch.empty((T, 1, D), dtype=torch.bfloat16, device="cuda")
    Q.cache_append(pool.cache, torch.cat([x, -x], 1), 0, seq, pos)
    Q.cache_read(pool.cache, seq, pos, out, None)
    status()
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(mids.double())), min=-6) - 3)
    even = (torch.round(mids.double() / step) * step)  # torch.round: halves to even
    for i, r in enumerate(rows):
        e = (-90, -20, 0, 30, 100)[i // 3]
        want = r.double()
        if i % 3 == 2:
            want = torch.zeros(D, device="cuda", dtype=torch.float64)
            want[:mids.numel()] = even * 2.0 ** e
            want[127] = 448 * 2.0 ** e
        assert torch.equal(out[i, 0].double(), want), i


def test_append_e4m3_extremes():
    """Infinities saturate at the finite elements' scale, NaN stays, tiny rows keep the smallest scale."""
    import trie_label_scoring_gb300 as Q
    x = torch.zeros((4, D), device="cuda")
    x[0, :3] = torch.tensor([float("inf"), -float("inf"), 1.75])
    x[1, :2] = torch.tensor([float("nan"), 2.0])
    x[2, :2] = torch.tensor([1e-38, 2.0 ** -108])
    x[3, :2] = torch.tensor([3.0e38, -1.0])
    pool = Pool("e4m3", 1, [4])
    seq, pos = tokens([4])
    out = torch.empty((4, 1, D), dtype=torch.bfloat16, device="cuda")
    Q.cache_append(pool.cache, torch.cat([x, x], 1), 0, seq, pos)
    Q.cache_read(pool.cache, seq, pos, None, out)
    status()
    o = out[:, 0].double().cpu()
    assert o[0, 0] == 1.75 and o[0, 1] == -1.75 and o[0, 2] == 1.75
    assert torch.isnan(o[1, 0]) and o[1, 1] == 2.0
    assert o[2, 0] == 0 and o[2, 1] == 2.0 ** -108
    assert abs(o[3, 0] - 3.0e38) <= 2.0 ** -4 * 3.0e38 and o[3, 1] == 0


@pytest.mark.parametrize("seq,pos", [(9, 0), (0, -1), (0, 1 << 20), (1, 40)])
def test_append_reports_bad_indices_and_writes_the_rest(seq, pos):
    """A sequence, position or page id (the table's -7) out of range drops that token only."""
    import trie_label_scoring_gb300 as Q
    pool = Pool("bf16", 2, [64, 20])
    s = torch.tensor([0, seq], dtype=torch.int32, device="cuda")
    p = torch.tensor([7, pos], dtype=torch.int32, device="cuda")
    Q.cache_append(pool.cache, torch.ones((2, 4 * D), device="cuda"), 0, s, p)
    with pytest.raises(Q.QuailError) as e:
        Q.device_status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    assert int((pool.k == 1).sum()) == 2 * D
    out = torch.zeros((2, 2, D), dtype=torch.bfloat16, device="cuda")
    Q.cache_read(pool.cache, s, p, out, None)
    with pytest.raises(Q.QuailError):
        Q.device_status()
    assert bool((out[0] == 1).all()) and bool((out[1] == 0).all())
    status()


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hkv,lens", [(1, [1]), (2, [17, 1, 130]), (8, [300, 16]), (5, [33])])
def test_read_returns_what_the_cache_stands_for(kind, hkv, lens):
    import trie_label_scoring_gb300 as Q
    pool = Pool(kind, hkv, lens)
    pool.fill(lens)
    seq, pos = tokens(lens)
    pick = torch.randint(0, seq.numel(), (seq.numel() + 5,), device="cuda")  # any order, some twice
    seq, pos = seq[pick].contiguous(), pos[pick].contiguous()
    seq[3 % seq.numel()] = -1
    k = torch.full((seq.numel(), hkv, D), 9.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 9.0)
    Q.cache_read(pool.cache, seq, pos, k, v)
    status()
    live = seq >= 0
    for got, name in ((k, "k"), (v, "v")):
        assert torch.equal(got[live].double(), pool.rows(seq[live], pos[live], name))
        assert bool((got[~live] == 9).all())
    k2 = torch.full_like(k, 9.0)
    Q.cache_read(pool.cache, seq, pos, k2, None)
    status()
    assert torch.equal(k2, k)


# ------------------------------------------------------------------ attention
def attention_64(pool, q, offs, lens, prefix, causal, scale):
    """o, lse and the tolerances of both, in 64 bits, a sequence at a time."""
    T, hq, _ = q.shape
    G = hq // pool.hkv
    o = torch.zeros((T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), float("-inf"), dtype=torch.float64, device="cuda")
    tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        lo, hi = offs[b], offs[b + 1]
        if n == 0 or hi == lo:
            continue
        pos = torch.arange(n, device="cuda", dtype=torch.int32)
        seq = torch.full_like(pos, b)
        k, v = pool.rows(seq, pos, "k"), pool.rows(seq, pos, "v")
        x = q[lo:hi].double().reshape(hi - lo, pool.hkv, G, D)
        s = torch.einsum("qhgd,khd->qhgk", x, k) * scale
        mag = torch.einsum("qhgd,khd->qhgk", x.abs(), k.abs()) * scale
        if causal:
            i = torch.arange(hi - lo, device="cuda")[:, None]
            hide = (pos[None, :] > n - (hi - lo) + i)[:, None, None, :]
            s = s.masked_fill(hide, float("-inf"))
            mag = mag.masked_fill(hide, 0)
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[..., None])
        w = torch.einsum("qhgk,khd->qhgd", p, v)
        wa = torch.einsum("qhgk,khd->qhgd", p, v.abs())
        drift = GAMMA * mag.amax(-1) + 2.0 ** -20  # scores; and exp2, the sums and the joins
        o[lo:hi] = w.reshape(hi - lo, hq, D)
        lse[lo:hi] = z.reshape(hi - lo, hq)
        tol_o[lo:hi] = ((2.0 ** -8 * 1.01 + 2 * drift[..., None]) * wa + 2.0 ** -8 * w.abs()).reshape(hi - lo, hq, D)
        tol_l[lo:hi] = (drift + 2.0 ** -22 * z.abs()).reshape(hi - lo, hq)
    return o, lse, tol_o, tol_l


def attend(pool, q, offs, lens, prefix, causal, scale=None, slack=0, max_q=None, rows_after=2, lse=True, workspace=None,
           stream=None):
    """One call with rows behind the last sequence; returns out, lse of the real rows."""
    import trie_label_scoring_gb300 as Q
    T, hq, _ = q.shape
    single = offs is None
    if not single:
        q = torch.cat([q, torch.full((rows_after, hq, D), float("nan"), dtype=q.dtype, device="cuda")])
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full(q.shape[:2], 5.0, device="cuda") if lse else None
    max_q = max_q or (1 if single else max([1] + [int(b - a) for a, b in zip(offs, offs[1:])]))
    max_len = max(max(lens), prefix, 1) + slack
    n = Q.workspace_size_attention(pool.cache, hq, q.shape[0], max_q, max_len, prefix)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    Q.attention_shared(pool.cache, q, None if single else torch.tensor(offs, dtype=torch.int32, device="cuda"),
                       torch.tensor(lens, dtype=torch.int32, device="cuda"), max_q, max_len, pool.prefix_pages, out, ws,
                       lse=ls, causal=causal, scale=scale, stream=stream)
    status()
    if not single:
        assert bool((out[T:] == 5).all()) and (ls is None or bool((ls[T:] == 5).all()))
    return out[:T], None if ls is None else ls[:T]


@pytest.fixture(params=[0, 1, 2, 3])
def way(request):
    """Every way that an attention call can be carried out."""
    import trie_label_scoring_gb300 as Q
    Q._test_set_attention_way(request.param)
    yield request.param
    Q._test_set_attention_way(-1)


def check_attention(pool, q, offs, lens, prefix, causal, scale=None, **kw):
    """Every way, and the one that the call takes by itself, against 64 bits."""
    import trie_label_scoring_gb300 as Q
    at = list(range(len(lens) + 1)) if offs is None else offs
    o, z, tol_o, tol_l = attention_64(pool, q, at, lens, prefix, causal, scale or D ** -0.5)
    live = z > float("-inf")
    for way in [0, 1, 2, 3, -1] if prefix else [0, 3, -1]:
        Q._test_set_attention_way(way)
        try:
            out, lse = attend(pool, q, offs, lens, prefix, causal, scale, **kw)
        finally:
            Q._test_set_attention_way(-1)
        err = (out.double() - o).abs()
        assert bool((err <= tol_o).all()), f"way {way}: o off by {float((err - tol_o).max()):.3g} more than allowed"
        if lse is not None:
            assert torch.equal(z == float("-inf"), lse == float("-inf")), f"way {way}"
            err = (lse.double() - z)[live].abs()
            assert bool((err <= tol_l[live]).all()), f"way {way}: lse off by {float((err - tol_l[live]).max()):.3g} too much"
    return out, lse


HEADS = [(8, 2), (32, 8), (5, 5), (16, 1), (32, 1), (12, 3), (128, 4)]
SINGLE = [  # own lengths, prefix
    ([1], 0), ([16], 0), ([17, 1, 15, 33], 0), ([1, 2, 3], 16), ([127, 128, 129, 1000, 64], 48), ([5] * 40, 272),
    ([700, 3], 4096), ([9000], 0), ([1] * 300, 32),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("case", range(len(SINGLE)))
def test_attention_single_tokens(kind, hq, hkv, case):
    own, prefix = SINGLE[case]
    lens = [n + prefix for n in own]
    pool = Pool(kind, hkv, lens, prefix, seed=case, extra_pages=case % 3)
    pool.fill(lens)
    q = torch.randn((len(lens), hq, D), generator=torch.Generator(device="cuda").manual_seed(case), device="cuda").bfloat16()
    check_attention(pool, q, None, lens, prefix, causal=bool(case % 2), slack=0 if case % 3 == 0 else 16)


MANY = [  # queries, own lengths, prefix, causal
    ([1, 3, 2], [5, 3, 16], 0, True),
    ([4, 1, 0, 4], [20, 33, 0, 4], 64, True),
    ([6, 6, 6], [0, 40, 700], 128, False),
    ([17, 100, 33], [17, 100, 257], 0, True),
    ([130, 1, 64], [130, 300, 64], 160, True),
    ([257, 5], [513, 1030], 32, True),
    ([31, 32, 33], [300, 10, 128], 512, False),
    ([700], [700], 0, True),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 8), (5, 5), (16, 1), (32, 1)])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_attention_many_tokens(kind, hq, hkv, case):
    nq, own, prefix, causal = MANY[case]
    lens = [n + prefix for n in own]
    pool = Pool(kind, hkv, lens, prefix, seed=case)
    pool.fill(lens)
    offs = [0] + list(np.cumsum(nq))
    q = torch.randn((offs[-1], hq, D), generator=torch.Generator(device="cuda").manual_seed(case), device="cuda").bfloat16()
    check_attention(pool, q, offs, lens, prefix, causal, max_q=max(nq) + case % 2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq", [1, 5, 40])
def test_attention_without_keys(kind, nq):
    """Sequences of length zero, alone and among others: o = 0, lse = -inf; also a prefix that is all there is."""
    for lens, prefix in (([0, 0, 0], 0), ([0, 32, 50, 0], 32), ([0], 64)):
        pool = Pool(kind, 2, lens, prefix)
        pool.fill(lens)
        offs = [nq * i for i in range(len(lens) + 1)]
        q = torch.randn((offs[-1], 8, D), device="cuda").bfloat16()
        check_attention(pool, q, None if nq == 1 else offs, lens, prefix, causal=False)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq", [1, 20])
@pytest.mark.parametrize("q_scale,scale", [(60.0, None), (1e-4, None), (1.0, 1.5), (3e4, 1e-6)])
def test_attention_score_ranges(kind, nq, q_scale, scale):
    """Sharp softmaxes (one key takes all), flat ones, other score factors, queries outside fp16's range."""
    lens = [90, 333]
    pool = Pool(kind, 2, lens, 64)
    pool.fill(lens)
    q = (torch.randn((2 * nq, 8, D), device="cuda") * q_scale).bfloat16()
    if q_scale == 3e4:
        q[0, 0, 3] = 3e5
        q[1, 5] = 0
    check_attention(pool, q, None if nq == 1 else [0, nq, 2 * nq], lens, 64, True, scale)


@pytest.mark.parametrize("nq", [1, 20])
def test_attention_e4m3_value_scales_far_apart(nq, way):
    """V rows whose powers of two differ by 2^100: the sums keep what counts."""
    lens = [90, 333]
    pool = Pool("e4m3", 2, lens, 64)
    pool.fill(lens)
    g = torch.Generator(device="cuda").manual_seed(2)
    pool.vs.copy_(torch.randint(40, 220, pool.vs.shape, generator=g, device="cuda").to(torch.uint8))
    q = torch.randn((2 * nq, 8, D), device="cuda").bfloat16()
    offs = [0, nq, 2 * nq]
    out, lse = attend(pool, q, None if nq == 1 else offs, lens, 64, True)
    o, z, tol_o, tol_l = attention_64(pool, q, offs, lens, 64, True, D ** -0.5)
    err = (out.double() - o).abs()
    fits = tol_o < 3e38  # bf16's range
    assert bool((err <= tol_o)[fits & (o.abs() < 3e38)].all())
    assert bool(((lse.double() - z).abs() <= tol_l).all())


def test_attention_nan_and_infinity_stay_in_their_rows(way):
    """A NaN query row gives NaN in its own rows only; an infinite score takes the whole weight or gives NaN, as the formula."""
    lens = [40, 70, 33]
    pool = Pool("bf16", 2, lens, 16)
    pool.fill(lens)
    q = torch.randn((3, 8, D), device="cuda").bfloat16()
    ref, _ = attend(pool, q, None, lens, 16, True)
    q[1, 2, 7] = float("nan")
    out, lse = attend(pool, q, None, lens, 16, True)
    bad = torch.zeros((3, 8), dtype=torch.bool, device="cuda")
    bad[1, 2] = True
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    assert torch.equal(out[~bad], ref[~bad])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("prefix", [0, 64])
def test_attention_nan_in_the_cache_stays_in_its_rows(kind, nq, prefix, way):
    """A NaN value reaches its own dimension of its sequence's rows, a NaN key all of them; nothing else changes."""
    lens = [prefix + 90, prefix + 300, prefix + 49]
    pool = Pool(kind, 2, lens, prefix)
    pool.fill(lens)
    q = torch.randn((3 * nq, 8, D), device="cuda").bfloat16()
    offs = None if nq == 1 else [0, nq, 2 * nq, 3 * nq]
    good, lse = attend(pool, q, offs, lens, prefix, False)
    at = prefix + 137
    nan = float("nan") if kind == "bf16" else 0xFF
    page = int(pool.table[1, at // PAGE])
    mine = torch.zeros(good.shape, dtype=torch.bool, device="cuda")
    keep = pool.v[page, 1, at % PAGE, 71].clone()
    pool.v[page, 1, at % PAGE, 71] = nan
    out, z = attend(pool, q, offs, lens, prefix, False)
    mine[nq:2 * nq, 4:, 71] = True
    assert bool(out[mine].isnan().all()) and torch.equal(out[~mine], good[~mine]) and torch.equal(z, lse)
    pool.v[page, 1, at % PAGE, 71] = keep
    pool.k[page, 1, at % PAGE, 3] = nan
    out, z = attend(pool, q, offs, lens, prefix, False)
    mine[nq:2 * nq, 4:] = True
    assert bool(out[mine].isnan().all()) and torch.equal(out[~mine], good[~mine])
    assert bool(z[mine[..., 0]].isnan().all()) and torch.equal(z[~mine[..., 0]], lse[~mine[..., 0]])


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_takes_every_e4m3_code(nq, way):
    """All 254 finite codes among keys and values, keys' scales from 2^-30 to 2^-9, values' from 2^-60 to 2^60. Streamed
    weights times the values' scales are fp16: below 2^-14 they round by at most 2^-25 of the largest one's step to 1."""
    lens = [254, 254]
    pool = Pool("e4m3", 2, lens)
    pool.fill(lens)
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8, device="cuda")
    for i in range(2):
        for j in range(254):
            page = int(pool.table[i, j // PAGE])
            pool.v[page, :, j % PAGE] = codes[(torch.arange(D, device="cuda") + j) % 254]
            pool.k[page, :, j % PAGE] = codes[(torch.arange(D, device="cuda") * 3 + j) % 254]
    pool.ks.copy_(torch.randint(97, 119, pool.ks.shape, generator=g, device="cuda").to(torch.uint8))
    pool.vs.copy_(torch.randint(67, 188, pool.vs.shape, generator=g, device="cuda").to(torch.uint8))
    q = torch.randn((2 * nq, 8, D), generator=g, device="cuda").bfloat16()
    offs = [0, nq, 2 * nq]
    out, lse = attend(pool, q, None if nq == 1 else offs, lens, 0, True)
    o, z, tol_o, tol_l = attention_64(pool, q, offs, lens, 0, True, D ** -0.5)
    pos = torch.arange(254, device="cuda", dtype=torch.int32)
    for b in range(2):
        seq = torch.full_like(pos, b)
        k, v = pool.rows(seq, pos, "k"), pool.rows(seq, pos, "v")
        ve = torch.exp2(pool.vs[pool.table[b, pos.long() // PAGE].long(), :, pos.long() % PAGE].double() - 127)  # [n, hkv]
        x = q[b * nq:(b + 1) * nq].double().reshape(nq, 2, 4, D)
        sc = torch.einsum("qhgd,khd->qhgk", x, k) * D ** -0.5
        i = torch.arange(nq, device="cuda")[:, None]
        sc = sc.masked_fill((pos[None, :] > 254 - nq + i)[:, None, None, :], float("-inf"))
        top = (torch.softmax(sc, -1) * ve.T[None, :, None, :]).amax(-1)  # [q, hkv, G]
        size = (v.abs() / ve[..., None]).sum(0)  # sum of |code| [hkv, D]
        tol_o[b * nq:(b + 1) * nq] += (2.0 ** -25 * top[..., None] * size[None, :, None, :]).reshape(nq, 8, D)
    assert bool(((out.double() - o).abs() <= tol_o).all())
    assert bool(((lse.double() - z).abs() <= tol_l).all())


def test_attention_large_pool_offsets():
    """Page ids whose byte and element offsets pass 32 bits."""
    for kind in ("bf16", "e4m3"):
        first = 140000 if kind == "bf16" else 270000
        pool = Pool(kind, 8, [300, 40], 32, first_page=first)
        pool.fill([300, 40])
        q = torch.randn((2, 32, D), device="cuda").bfloat16()
        check_attention(pool, q, None, [300, 40], 32, True)
        q = torch.randn((60, 32, D), device="cuda").bfloat16()
        check_attention(pool, q, [0, 52, 60], [300, 40], 32, True)  # 8 own keys, 8 queries
        del pool
        torch.cuda.empty_cache()


@pytest.mark.parametrize("nq", [1, 20])
@pytest.mark.parametrize("what", ["page", "prefix page", "length", "short", "offsets"])
def test_attention_reports_bad_indices(nq, what, way):
    """Out-of-range ids and lengths set the error word; the other sequences' rows stay right."""
    import trie_label_scoring_gb300 as Q
    lens, prefix = [90, 64, 333], 32
    pool = Pool("bf16", 2, lens, prefix)
    pool.fill(lens)
    q = torch.randn((3 * nq, 8, D), device="cuda").bfloat16()
    offs = [0, nq, 2 * nq, 3 * nq]
    good, _ = attend(pool, q, None if nq == 1 else offs, lens, prefix, True)
    table, pp, L, of = pool.table, pool.prefix_pages, torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor(
        offs, dtype=torch.int32, device="cuda")
    if what == "page":
        table[1, 3] = pool.pages
    elif what == "prefix page":
        pp[1] = -1
    elif what == "length":
        L[1] = 334
    elif what == "short":
        L[1] = 32
    else:
        if nq == 1:
            return
        of[2] = 3 * nq + 1000
    out = torch.zeros_like(q)
    n = Q.workspace_size_attention(pool.cache, 8, q.shape[0], nq, 333, prefix)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    Q.attention_shared(pool.cache, q, None if nq == 1 else of, L, nq, 333, pp, out, ws)
    with pytest.raises(Q.QuailError) as e:
        Q.device_status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    if what != "prefix page":
        assert torch.equal(out[:nq], good[:nq])
        if what != "offsets":
            assert torch.equal(out[2 * nq:], good[2 * nq:])
    status()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_wait_timeout_is_reported(kind, way):
    """With the limit of every pipeline wait cut to a few hundred cycles (a test hook) the waits run out before their
    copies arrive: the kernels drain what is in flight, free their tensor memory and return, the error word says so,
    and the next call is right."""
    import trie_label_scoring_gb300 as Q
    lens, prefix = [3000, 2222] * 40, 1024  # enough pages under way for some to wait in line
    pool = Pool(kind, 8, lens, prefix)
    pool.fill(lens)
    q = torch.randn((80, 32, D), device="cuda").bfloat16()
    good, _ = attend(pool, q, None, lens, prefix, True)
    Q._test_set_pipeline_wait_limit(200)
    try:
        short, _ = attend(pool, q, None, lens, prefix, True)
    except Q.QuailError as e:
        assert e.name == "QUAIL_ERR_DEVICE_TIMEOUT"
    else:  # streamed pages: a wait may be over within its first try, which has no limit of its own
        assert way == 0 and torch.equal(good, short)
    finally:
        Q._test_set_pipeline_wait_limit(0)
    again, _ = attend(pool, q, None, lens, prefix, True)
    assert torch.equal(good, again)


def test_python_checks_of_tensors():
    import trie_label_scoring_gb300 as Q
    pool = Pool("bf16", 2, [64, 64])
    q = torch.zeros((2, 8, D), dtype=torch.bfloat16, device="cuda")
    L = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    ws = torch.empty(Q.workspace_size_attention(pool.cache, 8, 2, 1, 64), dtype=torch.uint8, device="cuda")
    good = dict(cache=pool.cache, q=q, q_offsets=None, seq_len=L, max_q_len=1, max_seq_len=64, prefix_pages=None,
                out=torch.empty_like(q), workspace=ws)
    Q.attention_shared(**good)
    status()
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(seq_len=L.long()), dict(seq_len=L[:1]), dict(out=q[:1]),
                dict(q=q.transpose(0, 1)), dict(lse=torch.zeros((2, 4), device="cuda")), dict(workspace=ws[:100])):
        with pytest.raises(Q.QuailError):
            Q.attention_shared(**{**good, **bad})
    with pytest.raises(Q.QuailError):
        Q.KVCache(pool.k, pool.v, pool.table, pool.k, pool.v)
    with pytest.raises(Q.QuailError):
        Q.KVCache(pool.k.view(torch.uint8)[..., :D].contiguous(), pool.v.view(torch.uint8)[..., :D].contiguous(), pool.table)
    host = torch.zeros((2, 6 * D))
    with pytest.raises(Q.QuailError):
        Q.cache_append(pool.cache, host, 2, L, L)


# ------------------------------------------------------------------ streams, graphs, the operators together
@pytest.mark.parametrize("nq", [1, 24])
def test_capture_and_replay_on_a_side_stream(nq, way):
    """append + attention captured into two graphs with a workspace each, replayed with new inputs, against eager calls."""
    import trie_label_scoring_gb300 as Q
    lens, prefix, hq, hkv = [100, 77, 200], 48, 8, 2
    offs = [nq * i for i in range(4)]
    T = offs[-1]
    seq = torch.tensor(np.repeat(np.arange(3), nq), dtype=torch.int32, device="cuda")
    pos = torch.tensor(np.concatenate([np.arange(n - nq, n) for n in lens]), dtype=torch.int32, device="cuda")
    pools = [Pool("e4m3", hkv, lens, prefix, seed=i) for i in range(2)]
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    of = None if nq == 1 else torch.tensor(offs, dtype=torch.int32, device="cuda")
    qkv = [torch.randn((T, (hq + 2 * hkv) * D), device="cuda") for _ in range(2)]
    q = [torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = [torch.zeros_like(q[0]) for _ in range(2)]
    size = Q.workspace_size_attention(pools[0].cache, hq, T, nq, 200, prefix)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(i):
        Q.cache_append(pools[i].cache, qkv[i], hq, seq, pos, q_out=q[i], rope_theta=1e6)
        Q.attention_shared(pools[i].cache, q[i], of, L, nq, 200, pools[i].prefix_pages, out[i], ws[i])

    for p in pools:
        p.fill(lens)
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            step(i)
        graphs.append(g)
    for trial in range(3):
        for x in qkv:
            x.normal_()
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for i in range(2):
            step(i)
            torch.cuda.synchronize()
            assert torch.equal(out[i], got[i])
            check = attention_64(pools[i], q[i], offs, lens, prefix, True, D ** -0.5)
            assert bool(((out[i].double() - check[0]).abs() <= check[2]).all())
    status()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prefill_then_tokens(kind, way):
    """The operators as a document engine uses them: the instructions written once, documents prefilled behind them in
    two chunks, then single tokens; every step's attention against 64 bits on what the cache holds."""
    import trie_label_scoring_gb300 as Q
    hq, hkv, prefix = 8, 2, 64
    final = [prefix + n for n in (75, 130, 33)]
    pool = Pool(kind, hkv, final, prefix)
    gain = (1 + 0.1 * torch.randn(D, device="cuda")).bfloat16()

    def append(seq, pos):
        qkv = torch.randn((seq.numel(), (hq + 2 * hkv) * D), device="cuda").bfloat16()
        q = torch.empty((seq.numel(), hq, D), dtype=torch.bfloat16, device="cuda")
        Q.cache_append(pool.cache, qkv, hq, seq, pos, q_out=q, q_norm=gain, k_norm=gain, rope_theta=1e6)
        return q

    q = append(*tokens([prefix]))  # the shared pages, through sequence 0
    one = Q.KVCache(pool.k, pool.v, pool.table[:1].contiguous(), pool.ks, pool.vs)
    out = torch.empty_like(q)
    ws = torch.empty(Q.workspace_size_attention(one, hq, prefix, prefix, prefix, 0), dtype=torch.uint8, device="cuda")
    Q.attention_shared(one, q, torch.tensor([0, prefix], dtype=torch.int32, device="cuda"),
                       torch.tensor([prefix], dtype=torch.int32, device="cuda"), prefix, prefix, None, out, ws)
    status()
    o, _, tol, _ = attention_64(pool, q, [0, prefix], [prefix], 0, True, D ** -0.5)
    assert bool(((out.double() - o).abs() <= tol).all())
    lens = [prefix] * 3
    for new in ([40, 64, 1], [33, 65, 31], [1, 1, 1], [1, 0, 0]):
        first, lens = lens, [a + b for a, b in zip(lens, new)]
        seq, pos = tokens(lens, first)
        q = append(seq, pos)
        offs = [0] + list(np.cumsum(new))
        check_attention(pool, q, None if new == [1, 1, 1] else offs, lens, prefix, True)
    assert lens == final


def test_appended_cache_feeds_classification():
    """A bf16 cache written by cache_append is the paged KV of classify_trie_tree: against the oracle on the same rows."""
    import synthetic as S
    import trie_label_scoring_gb300 as Q
    from oracle import scoring as OS
    from oracle.trie import build_trie
    from tests import gpu_cases as C
    w = S.WORKLOADS["tiny-support10-4x128"]
    sh = w.shape
    model = C.device_model(sh)
    ls = S.make_labels(w, 0)
    lens = [128, 45, 1, 97]
    pool = Pool("bf16", sh.n_kv_heads, lens)
    seq, pos = tokens(lens)
    rows = 0.02 * torch.randn((seq.numel(), 2 * sh.n_kv_heads * D), device="cuda")
    Q.cache_append(pool.cache, rows, 0, seq, pos, k_norm=model.weights["k_norm"], rope_theta=sh.rope_theta)
    kv = Q.KV(pool.k, pool.v, pool.table, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens))
    trie = Q.Trie(ls.labels, ls.root_token, sh.vocab, ls.continuation)
    N, M = len(lens), len(ls.labels)
    ws = torch.empty(Q.workspace_size(model, trie, 0, N, max(lens), Q.MODE_TRIE_TREE), dtype=torch.uint8, device="cuda")
    lsc, prob = torch.empty((N, M), device="cuda"), torch.empty((N, M), device="cuda")
    am = torch.empty((N,), dtype=torch.int32, device="cuda")
    Q.classify_trie_tree(model, kv, trie, N, ws, lsc, prob, am)
    status()
    t = build_trie(ls.labels, ls.root_token, sh.vocab, ls.continuation)
    layer = C.oracle_layer(sh)
    for i, n in enumerate(lens):
        at = torch.arange(n, device="cuda", dtype=torch.int32)
        which = torch.full_like(at, i)
        dk, dv = (pool.rows(which, at, x).cpu().numpy() for x in ("k", "v"))
        r = OS.trie_tree(layer, dk, dv, t)
        C.check_scores(lsc[i].cpu().numpy(), prob[i].cpu().numpy(), int(am[i]), r["logscore"], r["prob"], r["argmax"],
                       f"doc {i}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("prefix", [0, 64])
def test_letters_over_a_cache(kind, prefix, way):
    """classify_letters_cached against the oracle on the rows that the cache holds, which it leaves as they are; over a
    bf16 cache classify_letters gives the same."""
    import synthetic as S
    import trie_label_scoring_gb300 as Q
    from oracle import scoring as OS
    from tests import gpu_cases as C
    sh = S.TINY
    model, layer = C.device_model(sh), C.oracle_layer(sh)
    letters, root = [7, 4000, 12, 900, 55, 8191, 0], 321
    lens = [prefix + n for n in (128, 15, 16, 300, 97)]
    N, M = len(lens), len(letters)
    pool = Pool(kind, sh.n_kv_heads, [n + 1 for n in lens], prefix)
    pool.fill(lens, k_scale=0.02, v_scale=0.02)
    if kind == "e4m3":  # codes of unit size times 2^-6 or so: rows like the bf16 ones
        pool.ks.copy_((pool.ks.int() - 6).to(torch.uint8))
        pool.vs.copy_((pool.vs.int() - 6).to(torch.uint8))
    keep = (pool.k.clone(), pool.v.clone())
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(Q.workspace_size_letters_cached(model, pool.cache, M, max(lens), prefix), dtype=torch.uint8,
                     device="cuda")
    lp, pr = torch.empty((N, M), device="cuda"), torch.empty((N, M), device="cuda")
    am = torch.empty((N,), dtype=torch.int32, device="cuda")
    Q.classify_letters_cached(model, pool.cache, pool.prefix_pages, L, max(lens), letters, root, ws, lp, pr, am)
    status()
    for i, n in enumerate(lens):
        at = torch.arange(n, device="cuda", dtype=torch.int32)
        which = torch.full_like(at, i)
        dk, dv = (pool.rows(which, at, x).cpu().numpy() for x in ("k", "v"))
        r = OS.letters(layer, dk, dv, letters, root)
        C.check_scores(lp[i].cpu().numpy(), pr[i].cpu().numpy(), int(am[i]), r["logprob"], r["prob"], r["argmax"], f"doc {i}")
    assert torch.equal(keep[0].view(torch.uint8), pool.k.view(torch.uint8))
    assert torch.equal(keep[1].view(torch.uint8), pool.v.view(torch.uint8))
    if kind == "bf16":
        kv = Q.KV(pool.k, pool.v, pool.table, L, max(lens))
        ws2 = torch.empty(Q.workspace_size(model, None, M, N, max(lens), Q.MODE_LETTERS), dtype=torch.uint8, device="cuda")
        lp2, pr2, am2 = torch.empty_like(lp), torch.empty_like(pr), torch.empty_like(am)
        Q.classify_letters(model, kv, letters, root, N, ws2, lp2, pr2, am2)
        status()
        assert float((lp - lp2).abs().max()) <= C.TOL_LOGSCORE


def test_letters_over_a_cache_refusals():
    import synthetic as S
    import trie_label_scoring_gb300 as Q
    from tests import gpu_cases as C
    sh = S.TINY
    model = C.device_model(sh)
    pool = Pool("bf16", sh.n_kv_heads, [32, 20])
    pool.fill([31, 19])
    L = torch.tensor([31, 19], dtype=torch.int32, device="cuda")
    ws = torch.empty(Q.workspace_size_letters_cached(model, pool.cache, 2, 31), dtype=torch.uint8, device="cuda")
    lp, pr = torch.empty((2, 2), device="cuda"), torch.empty((2, 2), device="cuda")
    am = torch.empty((2,), dtype=torch.int32, device="cuda")

    def call(cache=pool.cache, lens=L, max_len=31, letters=(1, 2), root=3, w=ws):
        Q.classify_letters_cached(model, cache, None, lens, max_len, letters, root, w, lp, pr, am)

    call()
    status()
    for kw, name in ((dict(letters=(1, 1)), "QUAIL_ERR_DUPLICATE_LABEL"), (dict(letters=(1, 9000)), "QUAIL_ERR_TOKEN_RANGE"),
                     (dict(root=-1), "QUAIL_ERR_TOKEN_RANGE"), (dict(w=ws[:256]), "QUAIL_ERR_WORKSPACE"),
                     (dict(max_len=33), "QUAIL_ERR_INVALID_ARG")):  # no page for position 32
        with pytest.raises(Q.QuailError) as e:
            call(**kw)
        assert e.value.name == name, (kw, e.value)
    other = Pool("bf16", 3, [32, 20])
    with pytest.raises(Q.QuailError):
        call(cache=other.cache)
    call(lens=torch.tensor([31, 32], dtype=torch.int32, device="cuda"))  # past max_doc_len
    with pytest.raises(Q.QuailError) as e:
        status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    call()
    status()


def test_letters_over_a_cache_of_empty_documents():
    """No document token at all: the answer token attends to itself alone, o = v."""
    import synthetic as S
    import trie_label_scoring_gb300 as Q
    from oracle import scoring as OS
    from tests import gpu_cases as C
    sh = S.TINY
    model, layer = C.device_model(sh), C.oracle_layer(sh)
    pool = Pool("bf16", sh.n_kv_heads, [16, 16, 16])
    pool.fill([16, 16, 16])
    lens = [0, 5, 0]
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(Q.workspace_size_letters_cached(model, pool.cache, 3, 16), dtype=torch.uint8, device="cuda")
    lp, pr = torch.empty((3, 3), device="cuda"), torch.empty((3, 3), device="cuda")
    am = torch.empty((3,), dtype=torch.int32, device="cuda")
    Q.classify_letters_cached(model, pool.cache, None, L, 16, [3, 5, 8000], 9, ws, lp, pr, am)
    status()
    for i, n in enumerate(lens):
        at = torch.arange(n, device="cuda", dtype=torch.int32)
        dk, dv = (pool.rows(torch.full_like(at, i), at, x).cpu().numpy().reshape(n, sh.n_kv_heads, 128) for x in ("k", "v"))
        r = OS.letters(layer, dk, dv, [3, 5, 8000], 9)
        C.check_scores(lp[i].cpu().numpy(), pr[i].cpu().numpy(), int(am[i]), r["logprob"], r["prob"], r["argmax"], f"doc {i}")
