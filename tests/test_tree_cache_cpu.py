"""CPU-only checks of the operators of drafted trees and bounded memory: their argument checks reject bad
calls before anything reaches a GPU, and the formulas that the GPU tests use agree with worked examples."""
import numpy as np
import pytest

from gathered_rank_gemm_gb300 import binding as B
from gathered_rank_gemm_gb300 import build
from tests import layer_ref as R
from tests import tree_ref as T
from tests.test_layer_cpu import ODD, P, _caller


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def test_tree_attention_arguments(lib):
    names = ("q qs o os lse qh cache pages kvh page d kf vf start kv table wide seqs t mq mask words scale window ws "
             "wsb status stream").split()
    base = dict(q=P, qs=512, o=P, os=512, lse=None, qh=4, cache=P, pages=10, kvh=2, page=16, d=128, kf=1.0, vf=1.0,
                start=P, kv=P, table=P, wide=10, seqs=3, t=80, mq=40, mask=P, words=2, scale=0.1, window=0, ws=P,
                wsb=1 << 30, status=None, stream=None)
    for fn in (lib.lora_kv4_tree_attention, lib.lora_kv4_tree_attention_f16):
        call = _caller(fn, names, base)
        for name in ("q", "o", "cache", "start", "kv", "table", "mask", "ws"):
            assert call(**{name: None}) == -1, name
        for kw in (dict(words=1), dict(words=0), dict(words=-1), dict(words=1 << 20), dict(mq=65), dict(d=96),
                   dict(qh=3), dict(page=20), dict(pages=0), dict(kf=0.0), dict(scale=0.0), dict(window=-1),
                   dict(wide=0), dict(seqs=0), dict(t=0), dict(mq=0), dict(mq=81), dict(qs=504)):
            assert call(**kw) == -3, kw
        for kw in (dict(q=ODD), dict(o=ODD), dict(cache=ODD), dict(ws=ODD), dict(qs=516), dict(mask=P + 2),
                   dict(lse=P + 2)):
            assert call(**kw) == -2, kw
        assert call(wsb=0) == -4


def test_accept_arguments(lib):
    names = "cache pages kvh page d start kv table wide seqs path len mp out status stream".split()
    base = dict(cache=P, pages=10, kvh=2, page=16, d=128, start=P, kv=P, table=P, wide=10, seqs=3, path=P, len=P, mp=8,
                out=P + 4096, status=None, stream=None)
    call = _caller(lib.lora_kv4_accept, names, base)
    for name in ("cache", "start", "kv", "table", "path", "len", "out"):
        assert call(**{name: None}) == -1, name
    for kw in (dict(pages=0), dict(kvh=0), dict(page=24), dict(d=32), dict(wide=0), dict(wide=1 << 28), dict(seqs=0),
               dict(seqs=65537), dict(mp=0), dict(mp=B.LORA_KV4_MAX_PATH + 1), dict(out=P), dict(out=P + 8),
               dict(out=P + 12, kv=P - 64, len=P - 64), dict(kv=P + 4096 - 8)):
        assert call(**kw) == -3, kw
    for kw in (dict(cache=ODD), dict(start=P + 2), dict(kv=P + 2), dict(table=P + 2), dict(path=P + 2), dict(len=P + 1),
               dict(out=P + 4098), dict(status=P + 2)):
        assert call(**kw) == -2, kw


def test_key_weights_arguments(lib):
    names = ("w cap q qs lse qh cache pages kvh page d kf start kv table wide seqs t mq scale window path len mp status "
             "stream").split()
    base = dict(w=P, cap=100, q=P, qs=512, lse=P, qh=4, cache=P, pages=10, kvh=2, page=16, d=128, kf=1.0, start=P, kv=P,
                table=P, wide=10, seqs=3, t=8, mq=4, scale=0.1, window=0, path=P, len=P, mp=4, status=None, stream=None)
    for fn in (lib.lora_kv4_key_weights, lib.lora_kv4_key_weights_f16):
        call = _caller(fn, names, base)
        for name in ("w", "q", "lse", "cache", "start", "kv", "table", "path", "len"):
            assert call(**{name: None}) == -1, name
        for kw in (dict(cap=0), dict(cap=1 << 31), dict(d=96), dict(qh=3), dict(qh=0), dict(kvh=0), dict(page=20),
                   dict(pages=0), dict(kf=0.0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
                   dict(window=-1), dict(window=1 << 31), dict(wide=0), dict(seqs=0), dict(t=0), dict(mq=0), dict(mq=9),
                   dict(qs=504), dict(mp=0), dict(mp=513)):
            assert call(**kw) == -3, kw
        for kw in (dict(w=P + 2), dict(q=ODD), dict(qs=516), dict(lse=P + 2), dict(cache=ODD), dict(path=P + 2),
                   dict(len=P + 2), dict(start=P + 2), dict(status=P + 1)):
            assert call(**kw) == -2, kw


def test_evict_arguments(lib):
    names = "cache pages kvh page d w pos cap kv last table wide seqs budget sink recent out status stream".split()
    base = dict(cache=P, pages=10, kvh=2, page=16, d=64, w=P, pos=P, cap=100, kv=P, last=P, table=P, wide=10, seqs=3,
                budget=10, sink=2, recent=8, out=P + 4096, status=None, stream=None)
    call = _caller(lib.lora_kv4_evict, names, base)
    for name in ("cache", "w", "pos", "kv", "last", "table", "out"):
        assert call(**{name: None}) == -1, name
    for kw in (dict(pages=0), dict(kvh=0), dict(page=24), dict(d=32), dict(cap=0), dict(cap=1 << 31), dict(wide=0),
               dict(seqs=0), dict(seqs=65537), dict(budget=0), dict(budget=1 << 31), dict(sink=-1), dict(recent=-1),
               dict(sink=3), dict(recent=9), dict(sink=11, recent=0), dict(sink=1 << 62, recent=1 << 62), dict(out=P),
               dict(out=P + 8), dict(last=P + 4100, kv=P)):
        assert call(**kw) == -3, kw
    for kw in (dict(cache=ODD), dict(w=P + 2), dict(pos=P + 2), dict(kv=P + 2), dict(last=P + 2), dict(table=P + 2),
               dict(out=P + 4098), dict(status=P + 2)):
        assert call(**kw) == -2, kw


def test_wrappers_want_cuda_tensors(lib):
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    cache = torch.zeros(1, 1, 1, 18 * 64, dtype=torch.uint8)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.lora_kv4_tree_attention(cache, q, q, None, None, None, 1, None, 0.1, None)
    with pytest.raises(ValueError, match="CUDA"):
        B.lora_kv4_accept(cache, n, n, n[:, None], n[:, None], n, n)
    with pytest.raises(ValueError, match="CUDA"):
        B.lora_kv4_key_weights(None, cache, q, None, n, n, n[:, None], 1, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        B.lora_kv4_evict(cache, None, None, n, n, n[:, None], 1, n)


# ------------------------------------------------------------------ the formulas themselves

def test_tree_visibility():
    sees = np.array([[1, 0, 0], [1, 1, 0], [1, 0, 1]], bool)  # a root with two children
    want = [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 1, 1, 0, 1]]
    assert np.array_equal(T.tree_visible(5, sees, 0), np.array(want, bool))
    # positions 2, 3, 3: a window of 2 leaves the key in front of the root, and none
    assert np.array_equal(T.tree_visible(5, sees, 2), np.array([[0, 1, 1, 0, 0], [0, 0, 1, 1, 0], [0, 0, 1, 0, 1]], bool))
    # two keys for three rows: the first row's own is not there
    assert np.array_equal(T.tree_visible(2, sees, 0), np.array([[0, 0], [1, 0], [0, 1]], bool))
    chain = np.tril(np.ones((4, 4), bool))
    for window in (0, 5):
        assert np.array_equal(T.tree_visible(9, chain, window)[:, :5], T.causal_visible(9, 4, window)[:, :5])


def test_mask_words():
    sees = np.zeros((2, 40), bool)
    sees[0, [0, 31]], sees[1, [32, 39]] = True, True
    assert T.mask_words(sees, 2).tolist() == [[-2 ** 31 + 1, 0], [0, 129]]


def test_a_path_is_causal_attention():
    """What the accepted path's rows see of a tree is what causal rows see after the move."""
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((6, 2, 8)), rng.standard_normal((20, 1, 8)), rng.standard_normal((20, 1, 8))
    sees = T.tree(rng, 6)
    path = np.nonzero(sees[5])[0]
    out, lse, _, _ = T.attention(q, k, v, 0.3, T.tree_visible(20, sees, 0))
    keys = list(range(14)) + [14 + c for c in path]
    want, wlse, _, _ = R.attention(q[path], k[keys], v[keys], 0.3, 0)
    assert np.allclose(out[path], want) and np.allclose(lse[path], wlse)
    # each row's probabilities sum to one
    w, _ = T.key_weights(np.zeros((1, len(keys))), q[path], wlse, k[keys], 0.3, 0)
    assert np.isclose(w.sum(), 2 * len(path))


def test_key_weights_by_differences():
    """d lse / d x_j = p_j: the weights of one row against central differences of lse along a score."""
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 8)), rng.standard_normal((5, 1, 8))
    lse = R.attention(q, k, k, 0.3, 0)[1]
    w, _ = T.key_weights(np.zeros((1, 5)), q, lse, k, 0.3, 0)
    for j in range(5):
        step = np.zeros((5, 1, 8))
        step[j, 0] = q[0, 0] / (q[0, 0] @ q[0, 0]) / 0.3 * 1e-5  # moves score j by 1e-5
        up, down = (R.attention(q, k + s * step, k, 0.3, 0)[1][0, 0] for s in (1, -1))
        assert abs((up - down) / 2e-5 - w[0, j]) < 1e-8


def test_evict_formula():
    w = np.array([5, 1, 3, 3, 9, 3, np.nan, 2], np.float32)
    pos = np.array([0, 3, 4, 5, 7, 9, -1, -1])
    got, p, of, to = T.evict(w, pos, 8, 12, 4, 1, 1)
    # kept: 0 (first), 7 (newest: position 12), 4 (9), 2 (3, the lowest index of three)
    assert to == [1, 3] and of == [4, 7]
    assert got.tolist()[:4] == [5, 9, 3, 2] and p.tolist() == [0, 7, 4, 12, -1, -1, -1, -1]
    assert T.evict(w, pos, 8, 12, 8, 0, 0)[1].tolist() == [0, 3, 4, 5, 7, 9, 11, 12]
