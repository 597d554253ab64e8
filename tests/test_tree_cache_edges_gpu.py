"""Drafted trees and bounded memory over the 4-bit cache where their contract is easily missed.  Helpers, and what
the tolerances rest on, are those of test_tree_cache_gpu.py."""
import math

import numpy as np
import pytest

from gathered_rank_gemm_gb300 import binding as B
from tests import tree_ref as T
from tests.test_layer_gpu import _np, lib  # noqa: F401
from tests.test_tree_cache_gpu import _set_masks, _status, _tree, _tree_case, _weights, _weights_case

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


# ------------------------------------------------------------------ rows that add nothing

@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("qh,kvh", [(1, 1), (4, 1), (8, 1), (12, 2), (5, 1)])
def test_a_key_of_nan_that_no_adding_row_sees(qh, kvh, rows):
    """A row with an lse of -infinity adds nothing, to a key of NaN neither, and what fills a tile behind the last row
    adds nothing at all: every weight but those of keys that an adding row sees keeps its bits."""
    for window in (0, 30):
        c = _weights_case([(rows, 300), (2, 40)], qh, kvh, 128, 16, "bf16", seed=310, window=window)
        first = 300 - rows - (window - 1 if window else 100)  # in a window, the first row alone sees it
        for x in T.entry(c["cache_np"], c["table_np"][0], 16, first, 128)[2:3]:
            x[:] = 0x7F  # a key of NaN
        c["cache"] = torch.tensor(c["cache_np"]).cuda()
        c["lse"][:1 if window else rows] = -math.inf
        _weights(c)
        got = c["w"].cpu().numpy()
        assert np.array_equal(got[0, :, first].view(np.int32), c["w_np"][0, :, first].view(np.int32)), (window, got[0, :, first])
        assert np.isfinite(got).all()
        if not window:
            assert np.array_equal(got[0, :, :300 - rows], c["w_np"][0, :, :300 - rows])
            assert (got[0, :, 300 - rows:300] == 0).all()


@pytest.mark.parametrize("rows", [1, 40])
def test_a_key_of_nan_and_paths_that_name_no_row(rows):
    c = _weights_case([(rows, 300), (2, 40)], 4, 1, 64, 16, "bf16", seed=311, paths=True)
    for x in T.entry(c["cache_np"], c["table_np"][0], 16, 17, 64)[2:3]:
        x[:] = 0x7F
    c["cache"] = torch.tensor(c["cache_np"]).cuda()
    c["path"][0] = -3
    status = _status()
    _weights(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_LENGTH
    got = c["w"].cpu().numpy()
    assert np.array_equal(got[0, :, :300 - rows], c["w_np"][0, :, :300 - rows]) and (got[0, :, 300 - rows:300] == 0).all()
