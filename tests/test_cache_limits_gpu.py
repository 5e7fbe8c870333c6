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
