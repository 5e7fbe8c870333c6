"""The document cache on the GPU at the edges that the larger comparisons do not
reach: waits that give up, infinite scores, appends of many tokens, positions up
to 2^24, hundreds of sequences."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_cache_gpu import (D, PAGE, Pool, attend, attention_64, built, check_attention, check_stored,  # noqa: E402,F401
                                  expected_rows, status, tokens, way)


# ------------------------------------------------------------------ waits that give up
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,nq", [([3000, 2222] * 40, 1), ([1000, 900], 1), ([1500, 150, 700], 40)])
def test_every_wait_that_gives_up_is_reported(kind, lens, nq, way):
    """With every pipeline wait giving up at once (a test hook) each kernel, those of a cluster of key ranges too, waits
    for its own copies, frees its tensor memory and returns: the error word says timeout, and the next call is right."""
    import trie_label_scoring_gb300 as Q
    for prefix in (0, 64):
        pool = Pool(kind, 2, lens, prefix)
        pool.fill(lens)
        q = torch.randn((len(lens) * nq, 8, D), device="cuda").bfloat16()
        offs = None if nq == 1 else [nq * i for i in range(len(lens) + 1)]
        good, lse = attend(pool, q, offs, lens, prefix, True)
        for _ in range(2):
            Q._test_set_pipeline_wait_limit(-1)
            try:
                with pytest.raises(Q.QuailError) as e:
                    attend(pool, q, offs, lens, prefix, True)
            finally:
                Q._test_set_pipeline_wait_limit(0)
            assert e.value.name == "QUAIL_ERR_DEVICE_TIMEOUT"
            again, z = attend(pool, q, offs, lens, prefix, True)
            assert torch.equal(good, again) and torch.equal(lse, z)


# ------------------------------------------------------------------ infinities
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq", [1, 20])
@pytest.mark.parametrize("prefix", [0, 64])
def test_attention_infinite_queries(kind, nq, prefix, way):
    """Query rows with an infinite element: scores of both infinities give NaN, o and lse; scores that are all -inf NaN and
    -inf, as the formula has them. Every other row as without them."""
    lens = [prefix + 90, prefix + 600]
    pool = Pool(kind, 2, lens, prefix)
    pool.fill(lens)
    code = torch.tensor(0xB8, dtype=torch.uint8, device="cuda") if kind == "e4m3" else -1.0  # -1
    pool.k[..., 9] = code
    q = torch.randn((2 * nq, 8, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    offs = [nq * i for i in range(3)]
    at = None if nq == 1 else offs
    good, lse = attend(pool, q, at, lens, prefix, True)
    inf = float("inf")
    q[nq - 1, 1, 9], q[2 * nq - 1, 6, 9], q[nq, 3, 50], q[0, 5, 50] = inf, inf, inf, -inf
    out, z = attend(pool, q, at, lens, prefix, True)
    o64, z64, _, _ = attention_64(pool, q, offs, lens, prefix, True, D ** -0.5)
    all_minus = z64 == -inf
    assert int(all_minus.sum()) == 2 and int((z64 == inf).sum()) == 2
    bad = o64.isnan().all(-1)
    assert int(bad.sum()) == 4 and torch.equal(bad, all_minus | (z64 == inf))
    assert bool(out[bad].isnan().all()) and bool((z[all_minus] == -inf).all()) and bool(z[bad & ~all_minus].isnan().all())
    assert torch.equal(out[~bad], good[~bad]) and torch.equal(z[~bad], lse[~bad])


@pytest.mark.parametrize("nq", [1, 20])
@pytest.mark.parametrize("prefix", [0, 64])
def test_attention_infinities_in_a_bf16_cache(nq, prefix, way):
    """An infinite value gives its dimension of every row that sees it; an infinite key makes NaN of the rows whose score
    it makes +inf and has weight 0 in those whose score is -inf."""
    lens = [prefix + 90, prefix + 600]
    pool = Pool("bf16", 2, lens, prefix)
    pool.fill(lens)
    q = torch.randn((2 * nq, 8, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    offs = [nq * i for i in range(3)]
    at = None if nq == 1 else offs
    inf = float("inf")
    page = int(pool.table[1, (prefix + 137) // PAGE])
    slot = (prefix + 137) % PAGE
    pool.v[page, 1, slot, 71] = -inf
    pool.k[page, 0, slot, 3] = inf
    out, z = attend(pool, q, at, lens, prefix, False)
    o64, z64, _, _ = attention_64(pool, q, offs, lens, prefix, False, D ** -0.5)
    assert bool((out[nq:, 4:, 71] == -inf).all()) and bool((o64[nq:, 4:, 71] == -inf).all())
    up = torch.zeros(z.shape, dtype=torch.bool, device="cuda")
    up[nq:, :4] = q[nq:, :4, 3] > 0
    assert 0 < int(up.sum()) < 4 * nq or nq == 1
    assert torch.equal(o64.isnan().all(-1), up)
    assert torch.equal(out.isnan().all(-1), up) and torch.equal(z.isnan(), up)
    _, _, t_o, t_l = _without_key(pool, page, slot, q, offs, lens, prefix)
    fin = o64.isfinite() & ~up[..., None]
    assert bool(((out.double() - o64).abs() <= t_o)[fin].all())
    assert bool(((z.double() - z64).abs() <= t_l)[~up].all())


def _without_key(pool, page, slot, q, offs, lens, prefix):
    """The tolerances with the infinite key and value at their finite size."""
    keep = pool.k[page, 0, slot, 3].clone(), pool.v[page, 1, slot, 71].clone()
    pool.k[page, 0, slot, 3], pool.v[page, 1, slot, 71] = 1.0, 1.0
    r = attention_64(pool, q, offs, lens, prefix, False, D ** -0.5)
    pool.k[page, 0, slot, 3], pool.v[page, 1, slot, 71] = keep
    return r


# ------------------------------------------------------------------ appends of many tokens
def _append_case(kind, src, hq, hkv, extra, norm=True, seed=0):
    """Tokens of ragged sequences in any order: 4 an SM and `extra` more, past which a block takes four of them."""
    n = 4 * torch.cuda.get_device_properties(0).multi_processor_count + extra
    rng = np.random.RandomState(seed)
    lens = [int(x) for x in rng.randint(1, 200, size=n // 60)]
    while sum(lens) < n:
        lens.append(97)
    pool = Pool(kind, hkv, lens)
    seq, pos = tokens(lens)
    pick = torch.from_numpy(rng.permutation(seq.numel())[:n]).cuda()
    seq, pos = seq[pick].contiguous(), pos[pick].contiguous()
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((n, (hq + 2 * hkv) * D), generator=g, device="cuda").to(src)
    gq = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() if norm else None
    gk = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() if norm else None
    return pool, seq, pos, qkv, gq, gk


def _check_append(pool, seq, pos, live, qkv, hq, gq, gk, q, before, theta):
    hkv = pool.hkv
    s, p = seq[live], pos[live]
    (wq, sq), (wk, sk), (wv, sv) = expected_rows(qkv[live], p, hq, hkv, gq, gk, 1e-6, theta)
    check_stored(q[live].double(), wq, sq)
    assert bool((q[~live] == 7).all())
    page, slot = pool.table[s.long(), p.long() // PAGE].long(), p.long() % PAGE
    for name, want, slack, sc in (("k", wk, sk, pool.ks), ("v", wv, sv, pool.vs)):
        check_stored(pool.rows(s, p, name), want, slack, None if sc is None else sc[page, :, slot])
    touched = torch.zeros(pool.k.shape[:3], dtype=torch.bool, device="cuda")
    touched[page, :, slot] = True
    for old, new in zip(before, (pool.k, pool.v)):
        as_int = torch.uint8 if pool.kind == "e4m3" else torch.int16
        assert torch.equal(old.view(as_int)[~touched], new.view(as_int)[~touched])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hq,hkv,extra,norm,theta", [(5, 3, 0, True, 1e6), (5, 3, 1, True, 1e6), (8, 2, 2, False, 1e4),
                                                     (1, 1, 3, True, 0.0), (32, 8, 2401, True, 1e6), (0, 1, 4, False, 0.0)])
def test_append_of_many_tokens(kind, src, hq, hkv, extra, norm, theta):
    """Both block forms at their border, with padding tokens at the ends and between the others."""
    import trie_label_scoring_gb300 as Q
    pool, seq, pos, qkv, gq, gk = _append_case(kind, src, hq, hkv, extra, norm, seed=extra)
    n = seq.numel()
    pad = torch.tensor([0, 5, 6, 7, 8, 17, n // 2, n - 3, n - 1], device="cuda")
    seq[pad] = -1
    pos[pad[::2]] = -9
    q = torch.full((n, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    before = (pool.k.clone(), pool.v.clone())
    Q.cache_append(pool.cache, qkv, hq, seq, pos, q_out=q, q_norm=gq, k_norm=gk, rms_eps=1e-6, rope_theta=theta)
    status()
    _check_append(pool, seq, pos, seq >= 0, qkv, hq, gq, gk, q, before, theta)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("extra", [0, 3])
def test_append_of_many_tokens_drops_bad_indices_only(kind, extra):
    """Bad sequences, positions and pages inside and at the end of a block: reported, and their tokens alone dropped."""
    import trie_label_scoring_gb300 as Q
    pool, seq, pos, qkv, gq, gk = _append_case(kind, torch.float32, 5, 3, extra, seed=7)
    n = seq.numel()
    bad = torch.tensor([2, 4, 7, 9, n - 2, n - 1], device="cuda")
    seq[2], seq[7] = pool.table.shape[0], 1 << 30
    pos[4], pos[9], pos[n - 2] = -1, (1 << 24) - 1, pool.table.shape[1] * PAGE
    pool.table[seq[n - 1].long(), pos[n - 1].long() // PAGE] = pool.pages  # and of whoever shares that page
    live = torch.ones(n, dtype=torch.bool, device="cuda")
    live[bad] = False
    live &= ~((seq == seq[n - 1]) & (pos // PAGE == pos[n - 1] // PAGE))
    q = torch.full((n, 5, D), 7.0, dtype=torch.bfloat16, device="cuda")
    before = (pool.k.clone(), pool.v.clone())
    Q.cache_append(pool.cache, qkv, 5, seq, pos, q_out=q, q_norm=gq, k_norm=gk, rms_eps=1e-6, rope_theta=1e6)
    with pytest.raises(Q.QuailError) as e:
        Q.device_status()
    assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    _check_append(pool, seq, pos, live, qkv, 5, gq, gk, q, before, 1e6)
    status()


# ------------------------------------------------------------------ far positions
def _round_bf16(x):
    """Nearest bf16 of 64-bit values in its normal range, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -120))) - 7)
    return torch.round(x / step) * step


@pytest.mark.parametrize("theta", [1e6, 1e4, 1.5])
def test_append_rotates_to_the_last_position(theta):
    """Unit rows at positions up to 2^24 - 1 come out as cosines and sines. The kernel's are within 1.7e-7 of the exact ones
    (emulated over every position: 1.6e-7), so what it rounds to bf16 lies between the roundings of exact -+ 1.7e-7."""
    import trie_label_scoring_gb300 as Q
    rng = np.random.RandomState(int(theta))
    pos = np.unique(np.concatenate([
        np.array([0, 1, 2, 4095, 65535, 65536, (1 << 20) + 1, (1 << 24) - 2, (1 << 24) - 1]),
        rng.randint(0, 1 << 24, size=12000), rng.randint((1 << 24) - 4096, 1 << 24, size=3000)])).astype(np.int32)
    pages = np.unique(pos // PAGE)
    table = np.full((1, 1 << 20), -1, dtype=np.int32)
    table[0, pages] = rng.permutation(pages.size)
    k, v = (torch.zeros((pages.size, 1, PAGE, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = Q.KVCache(k, v, torch.from_numpy(table).cuda())
    n = pos.size
    qkv = torch.zeros((n, 3 * D), device="cuda")
    qkv[:, :64] = 1            # q: (cos, sin)
    qkv[:, D + 64:2 * D] = 1   # k: (-sin, cos)
    p = torch.from_numpy(pos).cuda()
    q = torch.empty((n, 1, D), dtype=torch.bfloat16, device="cuda")
    Q.cache_append(cache, qkv, 1, torch.zeros_like(p), p, q_out=q, rope_theta=theta)
    status()
    ang = p.double()[:, None] * theta ** (-torch.arange(64, device="cuda").double() / 64)
    c, s = torch.cos(ang), torch.sin(ang)
    at = torch.from_numpy(table).cuda()[0, p.long() // PAGE].long()
    for got, want in ((q[:, 0], torch.cat([c, s], -1)), (k[at, 0, p.long() % PAGE], torch.cat([-s, c], -1))):
        got = got.double()
        assert bool((got >= _round_bf16(want - 1.7e-7)).all()) and bool((got <= _round_bf16(want + 1.7e-7)).all())


@pytest.mark.parametrize("n", [65537, (1 << 20) + 1, (1 << 24) - 1])
def test_letters_over_a_cache_of_far_documents(n):
    """The answer token at positions up to 2^24 - 1: classify_letters_cached beside classify_letters, whose own rotation is
    another one, on a document whose pages repeat."""
    import synthetic as S
    import trie_label_scoring_gb300 as Q
    from tests import gpu_cases as C
    sh = S.TINY
    model = C.device_model(sh)
    pages = 64
    g = torch.Generator(device="cuda").manual_seed(n % 1000)
    k, v = (0.02 * torch.randn((pages, sh.n_kv_heads, PAGE, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = (torch.arange(-(-n // PAGE), device="cuda", dtype=torch.int32) * 37 % pages).view(1, -1).contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    letters = [7, 4000, 12, 900, 55]
    cache = Q.KVCache(k, v, table)
    kv = Q.KV(k, v, table, lens, n)
    got = []
    for cached in (True, False):
        outs = [torch.empty((1, 5), device="cuda"), torch.empty((1, 5), device="cuda"),
                torch.empty((1,), dtype=torch.int32, device="cuda")]
        size = (Q.workspace_size_letters_cached(model, cache, 5, n) if cached else
                Q.workspace_size(model, None, 5, 1, n, Q.MODE_LETTERS))
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        if cached:
            Q.classify_letters_cached(model, cache, None, lens, n, letters, 321, ws, *outs)
        else:
            Q.classify_letters(model, kv, letters, 321, 1, ws, *outs)
        status()
        got.append(outs)
    assert float((got[0][0] - got[1][0]).abs().max()) <= C.TOL_LOGSCORE
    assert int(got[0][2]) == int(got[1][2])


# ------------------------------------------------------------------ hundreds of sequences
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("seqs,max_q", [(385, 1), (770, 3), (1537, 1), (1200, 2)])
def test_attention_of_hundreds_of_sequences(kind, seqs, max_q):
    """More sequences than the streaming kernel has threads, so that one of them plans several: ragged lengths, some of them
    0, some sequences without queries."""
    rng = np.random.RandomState(seqs)
    own = rng.randint(0, 70, size=seqs)
    own[rng.rand(seqs) < 0.1] = 0
    own[seqs // 2] = 3000
    nq = np.ones(seqs, dtype=int) if max_q == 1 else rng.randint(0, max_q + 1, size=seqs)
    for prefix in (0, 32):
        lens = [int(x) + prefix if x else 0 for x in own]
        pool = Pool(kind, 2, lens, prefix, seed=seqs)
        pool.fill(lens)
        offs = [0] + [int(x) for x in np.cumsum(nq)]
        q = torch.randn((offs[-1], 8, D), generator=torch.Generator(device="cuda").manual_seed(seqs), device="cuda").bfloat16()
        check_attention(pool, q, None if max_q == 1 else offs, lens, prefix, False, max_q=max_q)


@pytest.mark.parametrize("seqs", [60, 5000])
@pytest.mark.parametrize("prefix", [0, 16])
@pytest.mark.parametrize("bad,value", [(None, 0), (5, 1 << 20), (0.6, -5), (0.6, 10), (0.59, 1 << 30), (0.3, 0)])
def test_attention_bad_offsets_void_their_own_rows(seqs, prefix, bad, value, way):
    """Sequences of 0 to 2 queries, rows before the first and behind the last; an offset that makes nonsense of the two
    sequences it bounds leaves the others' rows right, and rows of no sequence as they were."""
    import trie_label_scoring_gb300 as Q
    hq, hkv, n, skip = 4, 2, 20 + prefix, 3
    rng = np.random.RandomState(1)
    nq = rng.randint(0, 3, size=seqs)
    offs = skip + np.concatenate([[0], np.cumsum(nq)])
    pool = Pool("bf16", hkv, [n] * 8, prefix)
    pool.fill([n] * 8)
    which = torch.from_numpy(rng.randint(0, 8, size=seqs)).cuda()
    cache = Q.KVCache(pool.k, pool.v, pool.table[which].contiguous())
    total = int(offs[-1]) + 4
    q = torch.randn((total, hq, D), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    of = torch.from_numpy(offs.astype(np.int32)).cuda()
    row_seq = torch.from_numpy(np.repeat(np.arange(seqs), nq)).cuda()
    o = torch.zeros((total, hq, D), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(o)
    for doc in range(8):  # all rows on one document at once
        rows = skip + torch.nonzero(which[row_seq] == doc)[:, 0]
        at = [0 if d <= doc else rows.numel() for d in range(9)]
        r = attention_64(pool, q[rows], at, [n if d == doc else 0 for d in range(8)], prefix, False, D ** -0.5)
        o[rows], tol[rows] = r[0], r[2]
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    live[skip:int(offs[-1])] = True
    if bad is not None:
        bad = int(bad if bad > 1 else bad * seqs)
        of[bad] = value
        live[skip:int(offs[-1])] = (row_seq != bad) & (row_seq != bad - 1)
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(Q.workspace_size_attention(cache, hq, total, 2, n, prefix), dtype=torch.uint8, device="cuda")
    L = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    Q.attention_shared(cache, q, of, L, 2, n, pool.prefix_pages, out, ws, causal=False)
    if bad is None:
        status()
    else:
        with pytest.raises(Q.QuailError) as e:
            status()
        assert e.value.name == "QUAIL_ERR_DEVICE_BOUNDS"
    err = ((out.double() - o).abs() <= tol).all(-1).all(-1)
    assert bool(err[live].all()), f"{int((~err[live]).sum())} rows wrong"
    assert bool((out[:skip] == 5).all()) and bool((out[int(offs[-1]):] == 5).all())


# ------------------------------------------------------------------ bits of the streamed weights
@pytest.fixture
def streamed():
    import trie_label_scoring_gb300 as Q
    Q._test_set_attention_way(0)
    yield
    Q._test_set_attention_way(-1)


@pytest.mark.parametrize("lens,prefix,nq", [([17] * 200, 0, 1), ([90, 400, 333], 64, 1), ([300] * 40, 0, 3), ([700], 0, 1)])
def test_streamed_bf16_weights_are_two_terms(lens, prefix, nq, streamed):
    """Queries and keys of -1, 0 and 1, so that the scores' sums are exact. A weight's two bf16 terms leave 2^-15 of it (a
    step of the first, 2^-7, times half a step of the second); its exponent, up to 16, is rounded three times in fp32, 2^-18 of the weight at most, twice (numerator
    and sum) with exp2 2^-17; fewer than 512 additions and joins in fp32 2^-15; the result is rounded once, 2^-8."""
    pool = Pool("bf16", 2, lens, prefix)
    pool.fill(lens)
    g = torch.Generator(device="cuda").manual_seed(4)
    pool.k.copy_(torch.randint(-1, 2, pool.k.shape, generator=g, device="cuda"))
    offs = [nq * i for i in range(len(lens) + 1)]
    q = torch.randint(-1, 2, (offs[-1], 8, D), generator=g, device="cuda").bfloat16()
    out, _ = attend(pool, q, None if nq == 1 else offs, lens, prefix, True)
    o = attention_64(pool, q, offs, lens, prefix, True, D ** -0.5)[0]
    pool.v.abs_()
    size = attention_64(pool, q, offs, lens, prefix, True, D ** -0.5)[0]  # sum p|v|
    allowed = (2.0 ** -15 + 2.0 ** -17 + 2.0 ** -15) * size + 2.0 ** -8 * o.abs()
    err = (out.double() - o).abs()
    assert bool((err <= allowed).all()), f"{int((err > allowed).sum())} of {err.numel()}"


def test_streamed_e4m3_weights_keep_small_ones(streamed):
    """One key takes nearly all the weight but has no value; 511 others have weights of 2^-26 and values of 1. So many
    sequences that a worker streams all keys of one: o is the others' sum, not 0."""
    n, seqs = 512, 2000
    pool = Pool("e4m3", 1, [n] * seqs)
    pool.k.zero_()
    pool.k[..., 0] = torch.tensor(-26.0).to(torch.float8_e4m3fn).view(torch.uint8)
    pool.v.fill_(torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8))
    pool.ks.fill_(127)
    pool.vs.fill_(127)
    first = pool.table[:, 0].long()
    pool.k[first, 0, 0] = 0
    pool.v[first, 0, 0] = 0
    q = torch.zeros((seqs, 4, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    out, lse = attend(pool, q, None, [n] * seqs, 0, True, scale=float(np.log(2)))
    rest = (n - 1) * 2.0 ** -26
    want = rest / (1 + rest)
    # the weights are powers of two but for the score factor's rounding, 2^-24 * 26; the result is rounded to bf16
    assert bool(((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -15) * want).all()), float(out.float().min())
    # a lane adds the weights of 64 keys of the 512 in fp32; beside the first key's 1, whose half step is 2^-24, each of
    # the other 63 adds nothing: 63 2^-26 at most are missing from the sum
    assert bool(((lse.double() - np.log1p(rest)).abs() <= 63 * 2.0 ** -26 + 2.0 ** -23).all())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("nq,prefix", [(1, 0), (1, 1024), (5, 640)])
def test_attention_of_a_padded_batch(kind, nq, prefix, way):
    """A batch padded far past its queries: thousands of rows of no sequence, which the bounds count, stay as they are."""
    lens = [3000 + prefix, 20 + prefix]
    pool = Pool(kind, 2, lens, prefix)
    pool.fill(lens)
    offs = [0, nq, 2 * nq]
    q = torch.randn((2 * nq, 8, D), generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").bfloat16()
    o, z, tol_o, tol_l = attention_64(pool, q, offs, lens, prefix, True, D ** -0.5)
    for rows_after in (0, 5000):
        out, lse = attend(pool, q, offs, lens, prefix, True, rows_after=rows_after)
        assert bool(((out.double() - o).abs() <= tol_o).all()) and bool(((lse.double() - z).abs() <= tol_l).all())
