"""Refusals of the calls for drafted trees that are made on the host, before any
device work: no GPU needed."""
import ctypes

import pytest

import trie_label_scoring_gb300 as Q
from tests.test_cache_host import SHAPES, desc, refused


@pytest.fixture(scope="module", autouse=True)
def built():
    Q.build()


def resize(d, pp=0x5000, prefix=16, old=0x6000, new=0x6100, ring=0x7000, state=0x7100, granted=0x7200, offs=0x7300,
           seq=0x8000, pos=0x9000, room=64):
    return Q.lib().quail_cache_resize(None if d is None else ctypes.byref(d), pp, prefix, old, new, ring, state, granted,
                                      offs, seq, pos, room, None)


ROPE = dict(layout=0, rotary_dim=128, theta=1e6, scaling=0, factor=1.0, original_len=0.0, low=1.0, high=32.0, magnitude=0.0)


def append(d, qkv=0x5000, dtype=0, ld=1024, n=4, hq=4, seq=0x6000, pos=0x7000, rope_pos=0x7100, gq=None, gk=None, eps=1e-6,
           q_out=0x8000, rope=None, no_rope=False):
    r = Q.RopeDesc(*[{**ROPE, **(rope or {})}[k] for k, _ in Q.RopeDesc._fields_])
    return Q.lib().quail_cache_append_rope(None if d is None else ctypes.byref(d), qkv, dtype, ld, n, hq, seq, pos,
                                           rope_pos, gq, gk, eps, None if no_rope else ctypes.byref(r), q_out, None)


def attend(d, q=0x7000, offs=0x100, seq_len=0x6000, mask=0xa000, total=6, max_q=4, max_len=64, hq=4, scale=0.0, ws=0x10000,
           ws_bytes=1 << 40, out=0x9000, lse=None):
    return Q.lib().quail_attention_tree(None if d is None else ctypes.byref(d), q, offs, seq_len, mask, total, max_q,
                                        max_len, hq, scale, ws, ws_bytes, out, lse, None)


def plan(parent=0x1000, offs=0x1100, seq_len=0x1200, seqs=3, total=6, max_q=4, mask=0x2000, rope_pos=0x3000):
    return Q.lib().quail_tree_plan(parent, offs, seq_len, seqs, total, max_q, mask, rope_pos, None)


def accept(descs, n=None, parent=0x1000, mask=0x2000, draft=0x2100, taken=0x2200, offs=0x1100, seq_len=0x1200, seqs=3,
           total=6, max_q=4, path=0x3000, accepted=0x3100, new_len=0x3200, bonus=0x3300):
    arr = (Q.CacheDesc * max(1, len(descs)))(*descs)
    return Q.lib().quail_tree_accept(arr, len(descs) if n is None else n, parent, mask, draft, taken, offs, seq_len, seqs,
                                     total, max_q, path, accepted, new_len, bonus, None)


@pytest.mark.parametrize("call", [resize, append, attend, lambda d: accept([d], seqs=d.num_seqs)])
@pytest.mark.parametrize("kw,status", [x for x in SHAPES if not set(x[0]) & {"k_pool", "page_table", "k_scale"} and x[0] != dict(dtype=Q.DTYPE_E4M3)])
def test_bad_caches_are_refused(call, kw, status):
    if call not in (resize, append, attend) and ("num_seqs" in kw):
        # the trees' own count is looked at first
        status = {-1: "QUAIL_ERR_INVALID_ARG", 65536: "QUAIL_ERR_UNSUPPORTED_SHAPE"}[kw["num_seqs"]]
    refused(call(desc(**kw)), status)


@pytest.mark.parametrize("call", [resize, append, attend])
@pytest.mark.parametrize("kw,status", SHAPES)
def test_bad_pointers_of_caches_are_refused(call, kw, status):
    refused(call(desc(**kw)), status)


@pytest.mark.parametrize("call", [resize, append, attend])
def test_null_cache_is_refused(call):
    refused(call(None), "QUAIL_ERR_INVALID_ARG")


@pytest.mark.parametrize("kw,status", [
    (dict(prefix=8), "QUAIL_ERR_INVALID_ARG"),
    (dict(prefix=-16), "QUAIL_ERR_INVALID_ARG"),
    (dict(prefix=80), "QUAIL_ERR_INVALID_ARG"),  # past the page table
    (dict(prefix=0), "QUAIL_ERR_INVALID_ARG"),   # pages without a length
    (dict(pp=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(room=-1), "QUAIL_ERR_INVALID_ARG"),
    (dict(seq=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(pos=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(seq=None, pos=None), "QUAIL_ERR_INVALID_ARG"),  # room without a map
    (dict(seq=0x8004), "QUAIL_ERR_INVALID_ARG"),
    (dict(pos=0x9008), "QUAIL_ERR_INVALID_ARG"),
    (dict(old=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(new=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(ring=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(state=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(granted=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(offs=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(granted=0x6000), "QUAIL_ERR_INVALID_ARG"),  # written while the lengths are read
    (dict(granted=0x6100), "QUAIL_ERR_INVALID_ARG"),
])
def test_resize_refusals(kw, status):
    refused(resize(desc(), **kw), status)


def test_resize_refuses_positions_past_32_bits():
    refused(resize(desc(max_pages=(1 << 26) + 1)), "QUAIL_ERR_UNSUPPORTED_SHAPE")


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=Q.DTYPE_E4M3), "QUAIL_ERR_INVALID_ARG"),
    (dict(ld=1020), "QUAIL_ERR_INVALID_ARG"),
    (dict(ld=1016), "QUAIL_ERR_INVALID_ARG"),
    (dict(n=-1), "QUAIL_ERR_INVALID_ARG"),
    (dict(hq=129, ld=1 << 20), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(gq=0x100, eps=0.0), "QUAIL_ERR_INVALID_ARG"),
    (dict(no_rope=True), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(layout=2)), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(layout=-1)), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(rotary_dim=0)), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(rope=dict(rotary_dim=24)), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(rope=dict(rotary_dim=144)), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(rope=dict(theta=1.0)), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(theta=float("nan"))), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(scaling=4)), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(scaling=-1)), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(scaling=1, factor=0.5)), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(scaling=2, factor=float("inf"))), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(scaling=3, factor=4.0)), "QUAIL_ERR_INVALID_ARG"),  # no original length
    (dict(rope=dict(scaling=3, factor=4.0, original_len=4096.0, low=4.0, high=4.0)), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(scaling=3, factor=4.0, original_len=4096.0, low=-1.0)), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(magnitude=-1.0)), "QUAIL_ERR_INVALID_ARG"),
    (dict(rope=dict(magnitude=float("nan"))), "QUAIL_ERR_INVALID_ARG"),
    (dict(qkv=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(seq=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(pos=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(qkv=0x5004), "QUAIL_ERR_INVALID_ARG"),
    (dict(q_out=0x8004), "QUAIL_ERR_INVALID_ARG"),
])
def test_append_rope_refusals(kw, status):
    refused(append(desc(), **kw), status)


def test_append_rope_refuses_positions_past_the_exact_angles():
    refused(append(desc(max_pages=(1 << 20) + 1), rope_pos=None), "QUAIL_ERR_UNSUPPORTED_SHAPE")


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), "QUAIL_ERR_INVALID_ARG"),
    (dict(seqs=65536), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(total=-1), "QUAIL_ERR_INVALID_ARG"),
    (dict(max_q=0), "QUAIL_ERR_INVALID_ARG"),
    (dict(max_q=1025), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(total=(1 << 30) + 1), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(parent=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(offs=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(seq_len=None), "QUAIL_ERR_INVALID_ARG"),
])
def test_refusals_of_trees(kw, status):
    refused(plan(**kw), status)
    refused(accept([desc()], **kw), status)


@pytest.mark.parametrize("kw", [dict(mask=None), dict(rope_pos=None), dict(mask=0x2004)])
def test_plan_refusals(kw):
    refused(plan(**kw), "QUAIL_ERR_INVALID_ARG")


@pytest.mark.parametrize("kw", [dict(n=-1), dict(mask=None), dict(draft=None), dict(taken=None), dict(path=None),
                                dict(accepted=None), dict(new_len=None), dict(bonus=None), dict(new_len=0x1200)])
def test_accept_refusals(kw):
    refused(accept([desc()], **kw), "QUAIL_ERR_INVALID_ARG")


@pytest.mark.parametrize("pools", [dict(k_pool=0x1000, v_pool=0x8000), dict(k_pool=0x8000, v_pool=0x2000),
                                   dict(k_pool=0x2000, v_pool=0x8000), dict(k_pool=0x8000, v_pool=0x1000),
                                   dict(k_pool=0x8000, v_pool=0x8000)])
def test_accept_refuses_a_pool_that_is_there_twice(pools):
    refused(accept([desc(), desc(**pools)]), "QUAIL_ERR_INVALID_ARG")


def test_accept_refuses_too_many_layers():
    refused(accept([desc()], n=1025), "QUAIL_ERR_UNSUPPORTED_SHAPE")


def test_resize_refuses_a_cache_without_sequences():
    refused(resize(desc(num_seqs=0)), "QUAIL_ERR_INVALID_ARG")


@pytest.mark.parametrize("other", [dict(n_kv_heads=4), dict(num_pages=9), dict(page_table=0x3010), dict(max_pages=5),
                                   dict(num_seqs=2), dict(dtype=Q.DTYPE_E4M3, k_scale=0x4000, v_scale=0x4100)])
def test_accept_refuses_caches_that_differ(other):
    refused(accept([desc(), desc(**other)]), "QUAIL_ERR_INVALID_ARG")


@pytest.mark.parametrize("kw,status", [
    (dict(hq=3), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(hq=130), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(total=-1), "QUAIL_ERR_INVALID_ARG"),
    (dict(max_q=0), "QUAIL_ERR_INVALID_ARG"),
    (dict(max_q=1025), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(max_len=0), "QUAIL_ERR_INVALID_ARG"),
    (dict(max_len=65), "QUAIL_ERR_INVALID_ARG"),
    (dict(scale=-1.0), "QUAIL_ERR_INVALID_ARG"),
    (dict(scale=float("inf")), "QUAIL_ERR_INVALID_ARG"),
    (dict(total=1 << 29), "QUAIL_ERR_UNSUPPORTED_SHAPE"),
    (dict(q=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(offs=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(seq_len=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(mask=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(out=None), "QUAIL_ERR_INVALID_ARG"),
    (dict(q=0x7002), "QUAIL_ERR_INVALID_ARG"),
    (dict(out=0x9008), "QUAIL_ERR_INVALID_ARG"),
    (dict(mask=0xa004), "QUAIL_ERR_INVALID_ARG"),
    (dict(ws=None), "QUAIL_ERR_WORKSPACE"),
    (dict(ws=0x10010), "QUAIL_ERR_WORKSPACE"),
    (dict(ws_bytes=16), "QUAIL_ERR_WORKSPACE"),
])
def test_attention_tree_refusals(kw, status):
    refused(attend(desc(), **kw), status)


def test_nothing_to_do_needs_no_device():
    Q._check(append(desc(), n=0))
    Q._check(plan(total=0))
    Q._check(plan(seqs=0))
    Q._check(accept([], seqs=0))
    Q._check(attend(desc(), total=0))
    Q._check(attend(desc(num_seqs=0)))


def workspace(d, hq=32, total=100, max_q=10, max_len=4096):
    return Q.lib().quail_workspace_size_attention_tree(ctypes.byref(d), hq, total, max_q, max_len)


def test_workspace_covers_smaller_bounds():
    big = dict(n_kv_heads=8, num_pages=4096, max_pages=1 << 20)
    for dtype, more in ((Q.DTYPE_BF16, {}), (Q.DTYPE_E4M3, dict(k_scale=0x100, v_scale=0x200))):
        for seqs, total, max_q, max_len in ((64, 400, 12, 2048), (1, 64, 64, 1 << 20), (300, 3000, 100, 700)):
            most = workspace(desc(dtype=dtype, num_seqs=seqs, **big, **more), 32, total, max_q, max_len)
            assert most > 0
            for s in {1, 2, seqs // 3 + 1, seqs}:
                for t in {1, 7, total // 2, total}:
                    for q in {1, 2, max_q // 2 + 1, max_q}:
                        for n in {1, 100, 129, max_len // 3, max_len}:
                            assert workspace(desc(dtype=dtype, num_seqs=s, **big, **more), 32, t, q, n) <= most


def test_workspace_refuses_bad_bounds():
    assert workspace(desc(n_kv_heads=8, max_pages=256), max_len=4097) == 0
    assert workspace(desc(n_kv_heads=8, max_pages=256), max_q=1025) == 0
    assert workspace(desc(n_kv_heads=8, max_pages=256), hq=12) == 0


@pytest.mark.parametrize("kw", [dict(layout="other"), dict(scaling="other"), dict(magnitude=0.0), dict(magnitude=-2.0)])
def test_rope_arguments(kw):
    with pytest.raises(Q.QuailError):
        Q.Rope(1e6, **kw)
