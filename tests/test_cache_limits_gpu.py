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
