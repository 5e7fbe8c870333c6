"""Calls that take host arrays, captured into a graph and replayed after those
arrays are gone, over documents that changed since: the same as eager calls."""
import numpy as np
import pytest

import synthetic as S
from tests import gpu_cases as C

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import trie_label_scoring_gb300 as Q
    Q.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)


def _replays_like_eager(call, outs, pools):
    """call() fills outs; captured, then replayed with other contents of the pools, beside an eager call on the same."""
    import trie_label_scoring_gb300 as Q
    call()
    Q.device_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    junk = [np.full(n, 0x7FFFFFF0, dtype=np.int32) for n in range(1, 4000, 3)]  # over what the call's own arrays left
    for _ in range(3):
        for p in pools:
            p.mul_(-0.75)
        call()
        Q.device_status()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(-3)
        graph.replay()
        Q.device_status()
        for o, x in zip(outs, want):
            assert torch.equal(o, x)
    return junk


def _docs(w):
    from trie_label_scoring_gb300.torch_inputs import kv_from_docs
    docs = S.make_docs(w, 0)
    kv = kv_from_docs(docs)
    k, v, table, lens = kv.tensors[:4]
    return docs, kv, k, v, table, lens


@pytest.mark.parametrize("m", [7, 959, 2500])  # one block of kernel arguments, its border with the node table, three
@pytest.mark.parametrize("cached", [False, True])
def test_letters_capture_and_replay(m, cached):
    import trie_label_scoring_gb300 as Q
    w = S.WORKLOADS["tiny-support10-4x128"]
    model = C.device_model(w.shape)
    docs, kv, k, v, table, lens = _docs(w)
    letters = [int(x) for x in np.random.default_rng(m).choice(w.shape.vocab, size=m, replace=False)]
    N = w.num_docs
    outs = [torch.empty((N, m), device="cuda"), torch.empty((N, m), device="cuda"),
            torch.empty((N,), dtype=torch.int32, device="cuda")]
    if cached:
        cache = Q.KVCache(k, v, table)
        n = Q.workspace_size_letters_cached(model, cache, m, docs.max_doc_len)
    else:
        n = Q.workspace_size(model, None, m, N, docs.max_doc_len, Q.MODE_LETTERS)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call():
        if cached:
            Q.classify_letters_cached(model, cache, None, lens, docs.max_doc_len, letters, 17, ws, *outs)
        else:
            Q.classify_letters(model, kv, letters, 17, N, ws, *outs)

    _replays_like_eager(call, outs, [k, v])


def test_join_capture_and_replay():
    import trie_label_scoring_gb300 as Q
    from tests.test_join import _answers, _partners
    w = S.WORKLOADS["tiny-support10-4x128"]
    model = C.device_model(w.shape)
    docs, kv, k, v, table, lens = _docs(w)
    rng = np.random.default_rng(2)
    partners = _partners(rng, w.shape.vocab)
    yes, no = _answers(rng, w.shape.vocab)
    t = Q.Trie(partners, 17, w.shape.vocab, all_nodes=True)
    N, M = w.num_docs, len(partners)
    ws = torch.empty(Q.workspace_size(model, t, len(yes) + len(no), N, docs.max_doc_len, Q.MODE_JOIN_IF),
                     dtype=torch.uint8, device="cuda")
    p = torch.empty((N, M), device="cuda")
    _replays_like_eager(lambda: Q.join_if(model, kv, t, N, yes, no, ws, p), [p], [k, v])


def test_layer_stack_capture_and_replay():
    import trie_label_scoring_gb300 as Q
    from trie_label_scoring_gb300.torch_inputs import kv_ml_from_docs, model_ml_from_bits
    mw = S.ML_WORKLOADS["tiny-L3-support10-4x128"]
    d0, ks, vs = S.make_docs_ml(mw.base, mw.n_layers, 0)
    labels = S.make_labels(mw.base, 0)
    model = model_ml_from_bits(S.make_model_ml(mw.base.shape, mw.n_layers, mw.intermediate, 0), mw.base.shape, mw.intermediate)
    kv = kv_ml_from_docs(d0, ks, vs)
    t = Q.Trie(labels.labels, labels.root_token, mw.base.shape.vocab, labels.continuation)
    N, M = len(d0.doc_len), len(labels.labels)
    ws = torch.empty(Q.workspace_size_ml(model, t, N, d0.max_doc_len), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((N, M), device="cuda"), torch.empty((N, M), device="cuda"),
            torch.empty((N,), dtype=torch.int32, device="cuda")]
    pools = [x for group in kv.tensors[:2] for x in group]
    _replays_like_eager(lambda: Q.classify_trie_tree_ml(model, kv, t, N, ws, *outs), outs, pools)


def _trie_case(seed=0):
    import trie_label_scoring_gb300 as Q
    w = S.WORKLOADS["tiny-support10-4x128"]
    docs, kv, k, v, table, lens = _docs(w)
    ls = S.make_labels(w, seed)
    trie = Q.Trie(ls.labels, ls.root_token, w.shape.vocab, ls.continuation)
    N, M = w.num_docs, len(ls.labels)
    outs = [torch.empty((N, M), device="cuda"), torch.empty((N, M), device="cuda"),
            torch.empty((N,), dtype=torch.int32, device="cuda")]
    return C.device_model(w.shape), docs, kv, [k, v], trie, N, outs


def test_trie_tree_capture_and_replay():
    import trie_label_scoring_gb300 as Q
    model, docs, kv, pools, trie, N, outs = _trie_case()
    ws = torch.empty(Q.workspace_size(model, trie, 0, N, docs.max_doc_len, Q.MODE_TRIE_TREE), dtype=torch.uint8, device="cuda")
    _replays_like_eager(lambda: Q.classify_trie_tree(model, kv, trie, N, ws, *outs), outs, pools)


def test_trie_tree_without_allocation_capture_and_replay():
    import trie_label_scoring_gb300 as Q
    model, docs, kv, pools, trie, N, outs = _trie_case()
    _replays_like_eager(lambda: Q.classify_trie_tree_noalloc(model, kv, trie, N, *outs), outs, pools)


def test_trie_decode_capture_and_replay():
    import trie_label_scoring_gb300 as Q
    w = S.WORKLOADS["tiny-support10-4x128"]
    docs, kv, k, v, table, lens = _docs(w)
    model = C.device_model(w.shape)
    trie = Q.Trie([[5, 6, 7], [5, 6, 8], [5, 9], [10, 11, 12], [10, 13]], 17, w.shape.vocab)
    N = w.num_docs
    ws = torch.empty(Q.workspace_size(model, trie, 0, N, docs.max_doc_len, Q.MODE_TRIE_DECODE), dtype=torch.uint8, device="cuda")
    cur, lab, act = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (N, N, 1))

    def call():  # greedy decoding from the root to the end
        cur.zero_()
        lab.fill_(-1)
        for _ in range(3):
            Q.classify_trie_decode_step(model, kv, trie, N, cur, lab, act, ws)

    _replays_like_eager(call, [cur, lab, act], [k, v])


def test_shortlist_capture_and_replay():
    import trie_label_scoring_gb300 as Q
    w = S.WORKLOADS["tiny-support10-4x128"]
    docs, kv, k, v, table, lens = _docs(w)
    model = C.device_model(w.shape)
    rng = np.random.default_rng(4)
    labels = [[int(a), int(b)] for a in rng.choice(w.shape.vocab, size=12, replace=False)
              for b in rng.choice(w.shape.vocab, size=5, replace=False)]
    trie = Q.Trie(labels, 17, w.shape.vocab)
    sl = Q.Shortlist(trie, 1)
    N, M = w.num_docs, len(labels)
    ws = torch.empty(Q.workspace_size_shortlist(model, trie, sl, 3, N, docs.max_doc_len), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((N, M), device="cuda"), torch.empty((N, M), device="cuda"),
            torch.empty((N,), dtype=torch.int32, device="cuda"), torch.empty((N, 3), dtype=torch.int32, device="cuda")]
    _replays_like_eager(lambda: Q.classify_trie_tree_shortlist(model, kv, trie, sl, 3, N, ws, *outs), outs, [k, v])
