"""Drafted trees and bounded memory over the 4-bit cache where their contract is easily missed.  Helpers, and what
the tolerances rest on, are those of test_tree_cache_gpu.py."""
import numpy as np
import pytest

from tests import tree_ref as T
from tests.test_layer_gpu import _np, lib  # noqa: F401
from tests.test_tree_cache_gpu import _set_masks, _tree, _tree_case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rows and windows

@pytest.mark.parametrize("window", [0, 1, 2, 7])
@pytest.mark.parametrize("rows,seqs", [(9, 1), (60, 1), (140, 1), (40, 30)])
def test_nan_of_an_ancestor_further_back_than_the_window(rows, seqs, window):
    """The window hides keys in front of a tree, never its own: a NaN of V at a distant ancestor is still the row's.
    9 and 60 rows go by the decode kernel; 140 (280 packed rows), and 40 of thirty sequences (300 groups), by the other."""
    c = _tree_case([(rows, 200 + 3 * b + rows) for b in range(seqs)], 4, 2, 128, 16, "bf16", seed=300 + rows)
    c["sees"] = [np.tril(np.ones((rows, rows), bool)) for _ in range(seqs)]  # chains: as deep as they have rows
    _set_masks(c)
    node, b = 1, seqs - 1
    key = c["lengths"][b][1] - rows + node
    for x in T.entry(c["cache_np"], c["table_np"][b], 16, key, 128)[3:]:
        x[:, 2] = 0x7F  # a NaN scale of V: dimensions 32 to 47
    c["cache"] = torch.tensor(c["cache_np"]).cuda()
    _tree(c, window)
    want = np.zeros((seqs, rows, 4, 128), bool)
    want[b, c["sees"][b][:, node], :, 32:48] = True
    assert np.array_equal(np.isnan(_np(c["out"])[:seqs * rows]).reshape(want.shape), want)
