"""Drafted trees and bounded memory over the 4-bit cache where their contract is easily missed.  Helpers, and what
the tolerances rest on, are those of test_tree_cache_gpu.py."""
import math

import numpy as np
import pytest

from gathered_rank_gemm_gb300 import binding as B
from tests import layer_ref as R
from tests import tree_ref as T
from tests.test_layer_gpu import DTYPES, FP32, K_SCALE, _i32, _np, lib  # noqa: F401
from tests.test_tree_cache_gpu import (_accept, _evict, _evict_case, _evict_check, _formula, _keys, _set_masks,
                                       _status, _tree, _tree_case, _tree_check, _weights, _weights_case,
                                       _weights_check)

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


# ------------------------------------------------------------------ paths and windows

def _path_visible(n, m, window):
    """What the rows of a path see: as the tree's attention has it, which hides keys in front of the tree only."""
    return T.tree_visible(n, np.tril(np.ones((m, m), bool)), window)


@pytest.mark.parametrize("window", [1, 2, 5, 30, 300])
@pytest.mark.parametrize("lengths,qh,kvh,d", [
    ([(9, 60), (3, 40), (1, 7), (6, 6), (0, 20)], 2, 2, 64), ([(12, 200), (40, 300), (7, 30)], 8, 2, 128),
    ([(300, 900), (100, 110), (64, 700)], 4, 1, 64), ([(130, 100), (70, 70)], 5, 1, 128)])
def test_paths_longer_than_the_window(lengths, qh, kvh, d, window):
    """Rows of a path give weight to what their lse counts: all of their ancestors, and the keys in front that the
    window leaves."""
    c = _weights_case(lengths, qh, kvh, d, 16, "bf16", seed=320 + window, paths=True)
    c["window"] = window
    q, lse, want, size = _np(c["q"]), c["lse"].cpu().numpy(), [], []
    for b, (m, n) in enumerate(lengths):
        r, k = c["rows_of"][b], _keys(c, b)[0]
        if m:
            visible = _path_visible(n, m, window)
            x = np.einsum("rhd,khd->rhk", q[r], np.repeat(k, qh // kvh, 1)) / math.sqrt(d)
            x = np.where(visible[:, None], x, -np.inf)
            with np.errstate(divide="ignore"):
                lse[r] = np.log(np.exp(x).sum(-1))
            full = np.zeros((kvh, max(n, c["capacity"])))
            full[:, :c["capacity"]] = c["w_np"][b]
            w, s = _formula(q[r], lse[r].astype(np.float64), k, 1 / math.sqrt(d), visible, full)
        else:
            w, s = c["w_np"][b].astype(np.float64), np.zeros(c["w_np"][b].shape)
        want.append(w), size.append(s)
    c["lse"].copy_(torch.tensor(lse))
    _weights(c)
    got = c["w"].cpu().numpy()
    for b, (m, n) in enumerate(lengths):
        tol = FP32 * size[b] + 2.0 ** -22 * np.abs(want[b])
        bad = ~(np.abs(got[b] - want[b]) <= tol)
        assert not bad.any(), (b, m, n, bad.sum(), np.argwhere(bad)[:4], got[b][bad][:4], want[b][bad][:4])


@pytest.mark.parametrize("rows", [10, 90])
def test_a_row_of_a_path_gives_away_a_weight_of_one_in_any_window(rows):
    """Tree attention, acceptance and weights one behind the other: every row on the path gives one a head."""
    for window in (0, 1, 3, 50):
        c = _tree_case([(rows, 60 + rows), (rows // 2, 200)], 8, 2, 128, 16, "bf16", seed=330 + rows)
        rng = np.random.default_rng(rows)
        c["sees"] = [T.tree(rng, m, deep=0.9) for m, _ in c["lengths"]]
        _set_masks(c)
        _tree(c, window)
        paths = [np.nonzero(s[s.sum(1).argmax()])[0].tolist() for s in c["sees"]]
        assert len(paths[0]) > rows // 3
        wide = max(map(len, paths))
        path, length, kv = _i32([p + [-1] * (wide - len(p)) for p in paths]), _i32([len(p) for p in paths]), _i32([0, 0])
        _accept(dict(c, path=path, len=length, out=kv))
        w = torch.zeros(2, 2, 200, device="cuda")
        B.lora_kv4_key_weights(w, c["cache"], c["q"], c["lse"], c["start"], kv, c["table"], c["max_q"], 1 / math.sqrt(128),
                               window=window, k_scale=K_SCALE, path=path, path_len=length)
        total = w.double().sum(-1).cpu()
        want = torch.tensor([4.0 * len(p) for p in paths])[:, None].expand(-1, 2)
        # lse and the scores are off by 2^-16 of sum |q k|, at most 60 here with 1 + |lse|
        assert ((total - want).abs() <= want * FP32 * 64).all(), (window, total, want)


def _random_case(lengths, qh, kvh, d, page, dtype, seed=0, window=0, paths=False, capacity=None, grow=1.0):
    """As _weights_case, with codes drawn as such (quick for many keys) and keys of about 1.4 K_SCALE * 32."""
    rng = np.random.default_rng(seed)
    per = [-(-n // page) for _, n in lengths]
    order, wide = rng.permutation(sum(per) + 3), max(1, max(per))
    table = np.full((len(per), wide), -7, np.int64)
    at = 0
    for b, x in enumerate(per):
        table[b, :x] = order[at:at + x]
        at += x
    cache = rng.integers(0, 256, (len(order), kvh, page // 16, 18 * d), dtype=np.uint8)
    cache[..., 16 * d:] = rng.integers(0x50, 0x5C, cache[..., 16 * d:].shape, dtype=np.uint8)  # scales of 8 to 22
    behind = 8 if paths else 0
    start = np.concatenate([[0], np.cumsum([m + behind for m, _ in lengths])])
    rows = int(start[-1]) + 2
    q = torch.tensor(rng.standard_normal((rows, qh, d)) * grow, dtype=torch.float32).to(DTYPES[dtype]).cuda()
    capacity = capacity or max(1, max(n for _, n in lengths))
    w = rng.random((len(lengths), kvh, capacity)).astype(np.float32)
    c = dict(lengths=lengths, q=q, cache_np=cache, cache=torch.tensor(cache).cuda(), table_np=table, table=_i32(table),
             start=_i32(start), start_np=start, kv=_i32([n for _, n in lengths]), page=page, dtype=dtype, rows=rows, qh=qh,
             kvh=kvh, d=d, max_q=max(1, max(m for m, _ in lengths)), out=torch.full_like(q, 7), window=window, path=None,
             len=None, capacity=capacity, w_np=w, w=torch.tensor(w).cuda(),
             rows_of=[np.arange(a, a + m) for a, (m, _) in zip(start, lengths)])
    if paths:
        spread = [np.sort(rng.permutation(m + behind)[:m]) for m, _ in lengths]
        path = np.full((len(lengths), c["max_q"] + 1), -3, np.int64)
        for b, p in enumerate(spread):
            path[b, :len(p)] = p
        c["path"], c["len"] = _i32(path), _i32([m for m, _ in lengths])
        c["rows_of"] = [a + p for a, p in zip(start, spread)]
    c["lse"] = torch.full((rows, qh), 7.0, device="cuda")
    return c


def _sight(c, b):
    m, n = c["lengths"][b]
    return T.tree_visible(n, np.tril(np.ones((m, m), bool)), c["window"]) if c["path"] is not None else \
        T.causal_visible(n, m, c["window"])


def _random_weights_check(c, some=None):
    """_weights_check of every key head (or of those in `some`) by itself, with the lse that the rows have."""
    g, d = c["qh"] // c["kvh"], c["d"]
    heads = range(c["kvh"]) if some is None else some
    q, lse = _np(c["q"]), c["lse"].cpu().numpy()
    keys = {(b, h): R.read_cache(c["cache_np"][:, h:h + 1], c["table_np"][b][:-(-n // c["page"])], n, c["page"], d)[0] * K_SCALE
            for b, (m, n) in enumerate(c["lengths"]) if m and n for h in heads}
    for b, h in keys:
        r, see = c["rows_of"][b], _sight(c, b)
        for i in range(h * g, h * g + g):
            x = np.where(see, q[r, i] @ keys[b, h][:, 0].T / math.sqrt(d), -np.inf)
            top = np.where(see.any(1), x.max(1), 0)
            with np.errstate(divide="ignore"):
                lse[r, i] = top + np.log(np.exp(x - top[:, None]).sum(1))
    c["lse"].copy_(torch.tensor(lse))
    status = _status()
    _weights(c, status=status)
    assert status[0].item() == 0
    got = c["w"].cpu().numpy()
    for b, (m, n) in enumerate(c["lengths"]):
        for h in heads:
            if not (m and n):
                assert np.array_equal(got[b, h], c["w_np"][b, h])
                continue
            r = c["rows_of"][b]
            full = c["w_np"][b, h:h + 1].astype(np.float64)
            want, size = _formula(q[r, h * g:h * g + g], lse[r, h * g:h * g + g].astype(np.float64), keys[b, h],
                                  1 / math.sqrt(d), _sight(c, b), full)
            # (fp32 holds no term below 2^-126: the exponential gives 0 there, m * g times at most)
            bad = ~(np.abs(got[b, h] - want[0]) <= FP32 * size[0] + 2.0 ** -22 * np.abs(want[0]) + m * g * 2.0 ** -126)
            assert not bad.any(), (b, h, m, n, bad.sum(), np.argwhere(bad)[:4], got[b, h][bad][:4], want[0][bad][:4])
            assert np.array_equal(got[b, h, n:], c["w_np"][b, h, n:])


# ------------------------------------------------------------------ scores of tens and hundreds

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lengths,qh,kvh,d", [([(1, 900), (3, 400), (8, 300)], 4, 1, 128), ([(60, 700), (100, 130)], 4, 2, 64)])
@pytest.mark.parametrize("grow", [30.0, 200.0])
def test_key_weights_of_large_scores(lengths, qh, kvh, d, grow, dtype):
    """Scores of tens and hundreds whose products cancel: each term of a weight is known to within 2^-16 of
    1 + |lse| + sum |q k|, which the check allows."""
    c = _random_case(lengths, qh, kvh, d, 16, dtype, seed=370, grow=grow)
    _random_weights_check(c)
    assert c["lse"][:c["start_np"][-1]].abs().max() > 2 * grow


# ------------------------------------------------------------------ the same bits

@pytest.mark.parametrize("paths", [None, True])
@pytest.mark.parametrize("lengths,qh,kvh", [
    ([(1, 900), (3, 333), (8, 700), (1, 50), (2, 350)], 8, 2), ([(1, 900), (3, 333), (64, 700), (1, 50), (200, 350)], 8, 2),
    ([(1 + b % 3 * 20, 300 + 7 * b) for b in range(40)], 4, 1)])
def test_a_sequences_weights_are_the_same_bits_in_any_batch(lengths, qh, kvh, paths):
    """Alone with the batch's bound on the rows, a sequence's weights are what they are in the batch."""
    c = _weights_case(lengths, qh, kvh, 128, 16, "bf16", seed=340, paths=paths)
    _weights(c)
    some = range(len(lengths)) if len(lengths) < 10 else (0, 1, 2, 20, 39)
    for b in some:
        r = torch.arange(int(c["start_np"][b]), int(c["start_np"][b + 1]), device="cuda")
        q, lse = torch.zeros_like(c["q"]), torch.zeros_like(c["lse"])
        q[:len(r)], lse[:len(r)] = c["q"][r], c["lse"][r]
        w = torch.tensor(c["w_np"][b:b + 1]).cuda()
        _weights({**c, "w": w, "q": q, "lse": lse, "start": _i32([0, len(r)]), "kv": c["kv"][b:b + 1],
                  "table": c["table"][b:b + 1], "path": c["path"][b:b + 1] if paths else None,
                  "len": c["len"][b:b + 1] if paths else None})
        assert torch.equal(w[0].view(torch.int32), c["w"][b].view(torch.int32)), b


@pytest.mark.parametrize("lengths,qh,kvh,d,window,dtype", [
    ([(15, 700)], 32, 8, 128, 0, "bf16"), ([(9 + b % 56, 500 + 100 * b) for b in range(32)], 32, 8, 128, 0, "bf16"),
    ([(33 + b % 5, 200 + 240 * b) for b in range(20)], 24, 4, 64, 2048, "f16"), ([(60, 30000), (50, 20000)], 8, 8, 128, 0, "bf16")])
def test_tree_attention_repeats_itself(lengths, qh, kvh, d, window, dtype):
    """In one workspace and in others, behind calls that leave other data on the chip."""
    c = _random_case(lengths, qh, kvh, d, 16, dtype, seed=350)
    c["sees"], c["words"] = [T.tree(np.random.default_rng(b), m) for b, (m, _) in enumerate(lengths)], 2
    _set_masks(c)
    ws = _tree(c, window)
    first = c["out"].clone(), c["lse"].clone()
    other = _random_case([(70, 900), (3, 4000)], 8, 2, 64, 16, "f16", seed=351)
    other["sees"], other["words"] = [np.tril(np.ones((m, m), bool)) for m, _ in other["lengths"]], 3
    _set_masks(other)
    for i in range(8):
        _tree(other)
        c["out"].fill_(7)
        _tree(c, window, **({} if i % 2 else dict(workspace=ws)))
        assert torch.equal(c["out"].view(torch.int16), first[0].view(torch.int16)), i
        assert torch.equal(c["lse"].view(torch.int32), first[1].view(torch.int32)), i


# ------------------------------------------------------------------ how items of many rows are shared out

def _items(c, few=32, keys=256):
    """Pairs of a sequence and a tile of 256 keys, and items a CTA: pairs times key heads over the SMs."""
    pairs = 0
    for m, n in c["lengths"]:
        if m * (c["qh"] // c["kvh"]) > few:
            first = max(0, n - m - c["window"] + 1) if c["window"] else 0
            pairs += max(0, -(-n // keys) - first // keys)
    return pairs, pairs * c["kvh"] / torch.cuda.get_device_properties(0).multi_processor_count


def _ragged(seqs, rows=40, least=300, spread=401):
    """Sequences of `rows` rows, some with few and some without any between them."""
    return [((0, 1, 2, rows, rows, rows, rows - 3)[b % 7] if b else 0, least + b * 131 % spread) for b in range(seqs)]


@pytest.mark.parametrize("paths", [False, True])
def test_more_pairs_than_are_sorted(paths):
    """Equal runs of all items: across key tiles and sequences."""
    c = _random_case(_ragged(420), 2, 1, 64, 16, "bf16", seed=360, paths=paths)
    pairs, each = _items(c)
    assert pairs > 512 and 2 < each <= 16
    _random_weights_check(c)


@pytest.mark.parametrize("paths", [False, True])
def test_more_pairs_than_are_sorted_in_a_window(paths):
    c = _random_case(_ragged(700, least=500), 3, 1, 64, 32, "f16", seed=361, paths=paths, window=170)
    assert _items(c)[0] > 512
    _random_weights_check(c)


def test_more_pairs_than_are_sorted_of_many_heads():
    """... across the heads of a sequence, whose tiles are cut by the ends of runs."""
    c = _random_case(_ragged(420, least=280, spread=300), 4, 4, 64, 16, "bf16", seed=362)
    pairs, each = _items(c)
    assert pairs > 512 and 4 < each <= 16
    _random_weights_check(c, some=(0, 1, 3))


@pytest.mark.parametrize("paths,window", [(False, 0), (True, 0), (False, 6000)])
def test_more_items_than_are_dealt(paths, window):
    """Few pairs, so many heads that a CTA has more than 16 items: runs across tiles and heads."""
    c = _random_case([(40, 9000), (2, 400), (34, 7000), (0, 90), (50, 6000)], 32, 32, 64, 64, "bf16", seed=363, paths=paths,
                     window=window)
    pairs, each = _items(c)
    assert pairs <= 512 and (each > 16) == (window == 0)
    _random_weights_check(c, some=(0, 1, 13, 30, 31))


@pytest.mark.parametrize("paths,window", [(False, 0), (True, 0), (True, 90), (False, 90)])
def test_pairs_that_one_lane_each_places(paths, window):
    """161 to 512 pairs in order of their rows, and a few rounds of dealing."""
    c = _random_case(_ragged(240, rows=70), 2, 2, 64, 16, "bf16", seed=364, paths=paths, window=window)
    pairs, each = _items(c)
    assert 160 < pairs <= 512 and 2 < each <= 16
    _random_weights_check(c)


@pytest.mark.parametrize("paths,window", [(False, 0), (True, 0), (False, 2000)])
def test_several_rounds_of_dealing(paths, window):
    """Items of one to eight row tiles, up to 16 rounds of them."""
    c = _random_case([(500, 6000), (40, 9000), (3, 700), (200, 3000), (90, 2000)], 16, 16, 64, 64, "f16", seed=365,
                     paths=paths, window=window)
    pairs, each = _items(c)
    assert pairs <= 160 and 3 < each <= 16
    _random_weights_check(c, some=(0, 7, 15))


# ------------------------------------------------------------------ captured calls

def _captured(call, before, after, check):
    """Captures call(before), replays it over the tensors of `after`, which are of the same shapes, and checks those."""
    call(before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(before)
    for name in ("cache", "q", "start", "kv", "table", "mask", "path", "len", "lse", "w", "out", "pos", "last"):
        if isinstance(before.get(name), torch.Tensor):
            before[name].copy_(after[name])
    graph.replay()
    check({**after, **{n: before[n] for n in ("cache", "out", "lse", "w", "pos") if n in before}})


@pytest.mark.parametrize("first,then", [([(140, 300), (20, 200)], [(60, 295), (100, 200)]), ([(30, 40), (1, 16)], [(1, 33), (30, 7)])])
def test_tree_attention_in_a_graph_over_other_lengths(first, then):
    a, b = (_tree_case(x, 4, 2, 128, 16, "bf16", seed=380 + i, words=5) for i, x in enumerate((first, then)))
    a["max_q"] = b["max_q"] = max(m for m, _ in first)
    space = torch.zeros(B.lora_kv4_attention_workspace_size(2, a["rows"], a["max_q"], 4, 2, 128), dtype=torch.uint8, device="cuda")
    _captured(lambda c: _tree(c, workspace=space), a, b, _tree_check)


@pytest.mark.parametrize("paths", [None, True])
@pytest.mark.parametrize("first,then", [([(140, 300), (20, 200)], [(60, 295), (100, 200)]), ([(300, 700), (3, 90)], [(3, 699), (300, 90)])])
def test_key_weights_of_many_rows_in_a_graph_over_other_lengths(first, then, paths):
    a, b = (_weights_case(x, 8, 2, 64, 16, "f16", seed=390 + i, paths=paths, capacity=700) for i, x in enumerate((first, then)))
    assert a["max_q"] >= b["max_q"] and a["q"].shape == b["q"].shape
    if paths:  # as wide as the first's paths
        b["path"] = torch.nn.functional.pad(b["path"], (0, a["path"].shape[1] - b["path"].shape[1]), value=-3)
    b["max_q"] = a["max_q"]
    _captured(_weights, a, b, _weights_check)


@pytest.mark.parametrize("first,then,heads,budget", [([9000, 40], [40, 9000], 2, 2000), ([300, 2100], [2090, 305], 8, 300)])
def test_eviction_in_a_graph_over_other_lengths(first, then, heads, budget):
    """By a cluster of CTAs a head, and by single ones."""
    a, b = (_evict_case(x, heads, 64, 16, seed=400 + i, capacity=max(first)) for i, x in enumerate((first, then)))
    for x in (a, b):  # pages for the longest in every sequence
        wide = -(-max(first) // 16)
        x["table_np"] = np.arange(2 * wide).reshape(2, wide)
        x["cache_np"] = np.random.default_rng(wide).integers(0, 256, (2 * wide, heads, 1, 18 * 64), dtype=np.uint8)
        x["table"], x["cache"] = _i32(x["table_np"]), torch.tensor(x["cache_np"]).cuda()
    b["out"] = a["out"]
    _captured(lambda c: _evict(c, budget, 4, 30), a, b, lambda c: _evict_check(c, budget, 4, 30))
