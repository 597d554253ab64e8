"""What the operators of drafted trees and bounded memory refuse before anything reaches a GPU, where that is
easily missed."""
import pytest

from gathered_rank_gemm_gb300 import binding as B
from gathered_rank_gemm_gb300 import build
from tests.test_layer_cpu import P, _caller

OUT = P + (1 << 20)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def test_new_lengths_inside_another_array(lib):
    """The kernels read every other array while the new lengths are written.  (No call here is launched: each has an
    operand that is refused, a status word at an odd address if nothing else.)"""
    names = "cache pages kvh page d start kv table wide seqs path len mp out status stream".split()
    base = dict(cache=P, pages=10, kvh=2, page=16, d=128, start=P, kv=P, table=P, wide=10, seqs=3, path=P, len=P, mp=8,
                out=OUT, status=P + 1, stream=None)
    accept = _caller(lib.lora_kv4_accept, names, base)
    assert accept() == -2
    # 4 row starts, 3 lengths, 3 x 8 rows of paths, 3 x 10 pages
    for name, words in (("start", 4), ("kv", 3), ("len", 3), ("path", 24), ("table", 30)):
        for at in (OUT - 8, OUT, OUT + 8, OUT - 4 * words + 4):
            assert accept(**{name: at}) == -3, (name, at)
        for at in (OUT - 4 * words, OUT + 12):
            assert accept(**{name: at}) == -2, (name, at)
    names = "cache pages kvh page d w pos cap kv last table wide seqs budget sink recent out status stream".split()
    base = dict(cache=P, pages=10, kvh=2, page=16, d=64, w=P, pos=P, cap=100, kv=P, last=P, table=P, wide=10, seqs=3,
                budget=10, sink=2, recent=8, out=OUT, status=P + 1, stream=None)
    evict = _caller(lib.lora_kv4_evict, names, base)
    assert evict() == -2
    for name, words in (("kv", 3), ("last", 3), ("table", 30), ("w", 600), ("pos", 600)):
        for at in (OUT - 8, OUT, OUT + 8, OUT - 4 * words + 4):
            assert evict(**{name: at}) == -3, (name, at)
        for at in (OUT - 4 * words, OUT + 12):
            assert evict(**{name: at}) == -2, (name, at)
