"""Refusals of the document cache calls that are made on the host, before any
device work: no GPU needed."""
import ctypes

import pytest

import trie_label_scoring_gb300 as Q

try:
    import torch
    HAS_GPU = torch.cuda.is_available()
except ImportError:
    HAS_GPU = False


@pytest.fixture(scope="module", autouse=True)
def built():
    Q.build()


def desc(**kw):
    d = dict(k_pool=0x1000, v_pool=0x2000, k_scale=None, v_scale=None, dtype=Q.DTYPE_BF16, n_kv_heads=2, head_dim=128,
             num_pages=8, page_size=16, page_table=0x3000, num_seqs=3, max_pages=4)
    d.update(kw)
    return Q.CacheDesc(*[d[k] for k, _ in Q.CacheDesc._fields_])


def refused(call, status):
    with pytest.raises(Q.QuailError) as e:
        Q._check(call)
    assert e.value.name == status, e.value
    assert str(e.value)


SHAPES = [
    (dict(head_dim=64), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(page_size=32), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(dtype=Q.DTYPE_F32), "QUAIL_ERR_INVALID_ARG"),
    (dict(n_kv_heads=0), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(num_pages=0), "QUAIL_ERR_INVALID_ARG"),
    (dict(num_seqs=-1), "QUAIL_ERR_INVALID_ARG"),
    (dict(num_seqs=65536), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(max_pages=0), "QUAIL_ERR_INVALID_ARG"),
    (dict(num_pages=1 << 27), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(k_pool=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(page_table=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(k_pool=0x1008), "QUAIL_ERR_INVALID_ARG"),
    (dict(dtype=Q.DTYPE_E4M3), "QUAIL_ERR_INVALID_ARG"),
    (dict(k_scale=0x4000), "QUAIL_ERR_INVALID_ARG"),
]


def append(d, qkv=0x5000, dtype=0, ld=1024, n=4, hq=4, seq=0x6000, pos=0x7000, gq=None, gk=None, eps=1e-6, theta=1e6,
           q_out=0x8000):
    return Q.lib().quail_cache_append(None if d is None else ctypes.byref(d), qkv, dtype, ld, n, hq, seq, pos, gq, gk,
                                      eps, theta, q_out, None)


def read(d, seq=0x6000, pos=0x7000, n=4, k=0x8000, v=0x9000):
    return Q.lib().quail_cache_read(None if d is None else ctypes.byref(d), seq, pos, n, k, v, None)


def attend(d, pp=0x5000, prefix=16, seq_len=0x6000, max_len=64, q=0x7000, offs=None, total=3, max_q=1, hq=4, causal=1,
           scale=0.0, ws=0x10000, ws_bytes=1 << 40, out=0x9000, lse=None):
    return Q.lib().quail_attention_shared(None if d is None else ctypes.byref(d), pp, prefix, seq_len, max_len, q,
                                          offs, total, max_q, hq, causal, scale, ws, ws_bytes, out, lse, None)


@pytest.mark.parametrize("call", [append, read, attend])
@pytest.mark.parametrize("kw,status", SHAPES)
def test_bad_caches_are_refused(call, kw, status):
    refused(call(desc(**kw)), status)


@pytest.mark.parametrize("call", [append, read, attend])
def test_null_cache_is_refused(call):
    refused(call(None), "QUAIL_ERR_INVALID_ARG")


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=Q.DTYPE_E4M3), "QUAIL_ERR_INVALID_ARG"),
    (dict(ld=1020), "QUAIL_ERR_INVALID_ARG"),      # not a multiple of 8
    (dict(ld=1016), "QUAIL_ERR_INVALID_ARG"),      # shorter than the 8 heads
    (dict(n=-1), "QUAIL_ERR_INVALID_ARG"),
    (dict(hq=-1), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(hq=129, ld=1 << 20), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(gq=0x100, eps=0.0), "QUAIL_ERR_INVALID_ARG"),
    (dict(theta=0.5), "QUAIL_ERR_INVALID_ARG"),
    (dict(theta=float("inf")), "QUAIL_ERR_INVALID_ARG"),
    (dict(theta=float("nan")), "QUAIL_ERR_INVALID_ARG"),
    (dict(qkv=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(seq=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(pos=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(qkv=0x5004), "QUAIL_ERR_INVALID_ARG"),
    (dict(q_out=0x8004), "QUAIL_ERR_INVALID_ARG"),
])
def test_append_refusals(kw, status):
    refused(append(desc(), **kw), status)


def test_append_refuses_positions_past_the_exact_angles():
    refused(append(desc(max_pages=(1 << 20) + 1)), "QUAIL_ERR_UNSUPPORTED_SHAPE")


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), "QUAIL_ERR_INVALID_ARG"),
    (dict(seq=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(k=None, v=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(k=0x8008), "QUAIL_ERR_INVALID_ARG"),
])
def test_read_refusals(kw, status):
    refused(read(desc(), **kw), status)


@pytest.mark.parametrize("kw,status", [
    (dict(hq=3), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(hq=0), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(hq=130), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(total=-1), "QUAIL_ERR_INVALID_ARG"),
    (dict(total=4), "QUAIL_ERR_INVALID_ARG"),       # one query a sequence without q_offsets
    (dict(max_q=2), "QUAIL_ERR_INVALID_ARG"),
    (dict(max_q=0), "QUAIL_ERR_INVALID_ARG"),
    (dict(prefix=8), "QUAIL_ERR_INVALID_ARG"),
    (dict(prefix=-16), "QUAIL_ERR_INVALID_ARG"),
    (dict(max_len=8), "QUAIL_ERR_INVALID_ARG"),     # below the prefix
    (dict(max_len=65), "QUAIL_ERR_INVALID_ARG"),    # past the page table
    (dict(causal=2), "QUAIL_ERR_INVALID_ARG"),
    (dict(scale=-1.0), "QUAIL_ERR_INVALID_ARG"),
    (dict(scale=float("nan")), "QUAIL_ERR_INVALID_ARG"),
    (dict(q=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(out=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(seq_len=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(pp=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(q=0x7002), "QUAIL_ERR_INVALID_ARG"),
    (dict(offs=0x100, total=1 << 29), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(ws=None), "QUAIL_ERR_WORKSPACE"),
    (dict(ws=0x10010), "QUAIL_ERR_WORKSPACE"),
    (dict(ws_bytes=16), "QUAIL_ERR_WORKSPACE"),
])
def test_attention_refusals(kw, status):
    refused(attend(desc(), **kw), status)


def test_nothing_to_do_is_fine():
    assert append(desc(), n=0) == 0
    assert read(desc(), n=0) == 0
    assert attend(desc(num_seqs=0), total=0) == 0


def test_attention_workspace_size():
    def size(**kw):
        a = dict(hq=32, total=256, max_q=1, max_len=4096, prefix=2048)
        a.update(kw)
        d = desc(n_kv_heads=8, num_pages=4096, num_seqs=256, max_pages=256)
        return Q.lib().quail_workspace_size_attention(ctypes.byref(d), a["hq"], a["total"], a["max_q"], a["max_len"],
                                                      a["prefix"])
    assert size() >= 256
    assert size(max_len=4097) == 0 and size(prefix=8) == 0 and size(hq=12) == 0


@pytest.mark.parametrize("max_len", [(1 << 30) + 1, (1 << 31) - 128, (1 << 31) - 127, (1 << 31) - 1])
def test_attention_refuses_lengths_whose_sums_pass_32_bits(max_len):
    """The page table may hold 2^31 positions; a call's longest sequence may not."""
    d = desc(n_kv_heads=1, num_seqs=1, max_pages=1 << 27)
    refused(attend(d, total=1, max_len=max_len), "QUAIL_ERR_UNSUPPORTED_SHAPE")
    assert Q.lib().quail_workspace_size_attention(ctypes.byref(d), 4, 1, 1, max_len, 16) == 0


def test_attention_workspace_of_the_longest_sequence():
    d = desc(n_kv_heads=1, num_seqs=1, max_pages=1 << 27)
    short = Q.lib().quail_workspace_size_attention(ctypes.byref(d), 4, 1, 1, 1 << 20, 16)
    assert 256 < short <= Q.lib().quail_workspace_size_attention(ctypes.byref(d), 4, 1, 1, 1 << 30, 16) < 1 << 30


def _attention_bounds(rng):
    """Random bounds of an attention call, log-uniform: (kv heads, q heads, sequences, total_q, max_q, max_len, prefix)."""
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8, 16])
    seqs, max_q = log(1, 512), log(1, 2048)
    total = rng.choice([seqs * max_q, max(1, seqs * max_q // 3), log(1, 1 << 20)])  # batches may carry spare rows
    total = min(total, (1 << 30) // (hkv * group))
    max_len = log(1, 1 << 18)
    return [hkv, hkv * group, seqs, total, max_q, max_len, rng.choice([0, log(1, max_len) // 16 * 16])]


def _need(dtype, b, ws_bytes):
    """The status of an attention call with that much workspace (other refusals come before or after it)."""
    d = desc(dtype=dtype, n_kv_heads=b[0], num_seqs=b[2], max_pages=1 << 18, num_pages=4096, k_scale=0x4000 if dtype else None,
             v_scale=0x5000 if dtype else None)
    code = attend(d, prefix=b[6], max_len=b[5], offs=0x100, total=b[3], max_q=b[4], hq=b[1], ws_bytes=ws_bytes)
    with pytest.raises(Q.QuailError) as e:
        Q._check(code)
    return e.value.name


def _size(dtype, b):
    d = desc(dtype=dtype, n_kv_heads=b[0], num_seqs=b[2], max_pages=1 << 18, num_pages=4096)
    return Q.lib().quail_workspace_size_attention(ctypes.byref(d), b[1], b[3], b[4], b[5], b[6])


@pytest.mark.skipif(HAS_GPU, reason="the calls would go past the workspace check with addresses that are none")
@pytest.mark.parametrize("dtype", [Q.DTYPE_BF16, Q.DTYPE_E4M3])
def test_attention_workspace_serves_all_smaller_bounds(dtype):
    """One allocation for the largest bounds: smaller ones ask for no more, and no call within them is refused it,
    whatever the way it takes."""
    import random
    rng = random.Random(dtype)
    for _ in range(400):
        big = _attention_bounds(rng)
        small = list(big)
        for i in rng.sample([2, 3, 4, 5, 6], rng.randint(0, 5)):
            small[i] = rng.randint(1, big[i]) if i != 6 else rng.randint(0, big[6] // 16) * 16
        small[6] = min(small[6], small[5] // 16 * 16)
        size = _size(dtype, big)
        assert 0 < _size(dtype, small) <= size, (big, small)
        for way in (-1, 0, 1, 2, 3):
            Q._test_set_attention_way(way)
            try:
                assert _need(dtype, small, size) != "QUAIL_ERR_WORKSPACE", (big, small, way)
            finally:
                Q._test_set_attention_way(-1)


def test_attention_workspace_grows_with_the_length():
    """64 sequences of one query behind 512 shared keys, 32 heads on 8; and 16 sequences of one."""
    for seqs, prefix in ((64, 512), (16, 0)):
        sizes = [_size(Q.DTYPE_BF16, [8, 32, seqs, seqs, 1, n, prefix]) for n in (512, 1024, 2048, 4096, 8192, 16384)]
        assert sizes == sorted(sizes)


@pytest.mark.parametrize("seqs", [1, 16, 64, 256])
def test_letters_workspace_grows_with_its_bounds(seqs):
    """Letters over a cache: more letters, longer documents or more shared tokens ask for no less."""
    m = Q.ModelDesc(2560, 32, 8, 128, 151936, 1e-6, 1e6)
    d = desc(n_kv_heads=8, num_seqs=seqs, max_pages=1 << 16, num_pages=4096)

    def size(letters, n, prefix):
        return Q.lib().quail_workspace_size_letters_cached(ctypes.byref(m), ctypes.byref(d), letters, n, prefix)

    for sizes in ([size(26, n, 512) for n in (512, 1024, 4096, 8192, 16384, 100000)],
                  [size(26, 8192, p) for p in (0, 16, 512, 2048, 8192)], [size(k, 8192, 0) for k in (2, 26, 300, 8192)]):
        assert sizes[0] > 0 and sizes == sorted(sizes)
