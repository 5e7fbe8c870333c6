"""Refusals of the document cache calls that are made on the host, before any
device work: no GPU needed."""
import ctypes

import pytest

import trie_label_scoring_gb300 as Q


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
