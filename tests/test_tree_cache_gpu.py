"""Drafted trees and bounded memory over the 4-bit cache on the GPU: tree attention, the accepted path, the
keys' weights and eviction, against their formulas in 64 bits on the CPU.

What the tolerances rest on is said in test_layer_gpu.py: a 16-bit output is rounded once, a probability once to
fp16, everything else happens in fp32 (2^-16 of the magnitudes that are summed).  A key's weight is a
sum of probabilities exp(x - lse) in fp32, each off by 2^-16 of (1 + sum |q k| + |lse|) of it.  Moves are exact."""
import math

import numpy as np
import pytest

from gathered_rank_gemm_gb300 import binding as B
from tests import layer_ref as R
from tests import tree_ref as T
from tests.test_layer_gpu import (BOTTOM, FP32, HALF_UNIT, K_SCALE, V_SCALE, _attend_case, _i32, _np,  # noqa: F401
                                  lib)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(4, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ tree attention

def _tree_case(lengths, qh, kvh, d, page, dtype, seed=0, words=None, **more):
    c = _attend_case(lengths, qh, kvh, d, page, dtype, seed=seed, **more)
    rng = np.random.default_rng(seed + 1000)
    c["sees"] = [T.tree(rng, m) for m, _ in lengths]
    c["words"] = words or -(-c["max_q"] // 32)
    _set_masks(c)
    return c


def _set_masks(c, stray=0):
    rows = [T.mask_words(s, c["words"]) for s in c["sees"]]
    mask = np.concatenate(rows + [np.full((c["rows"] - sum(map(len, rows)), c["words"]), -1, np.int32)])
    if stray:  # bits from m on count for nothing
        for b, (m, _) in enumerate(c["lengths"]):
            off = np.zeros((1, 32 * c["words"]), bool)
            off[0, m:] = True
            mask[c["start_np"][b]:c["start_np"][b + 1]] |= T.mask_words(off, c["words"])
    c["mask"] = _i32(mask)


def _tree(c, window=0, scale=None, **more):
    size = B.lora_kv4_attention_workspace_size(len(c["lengths"]), c["rows"], c["max_q"], c["qh"], c["kvh"], c["d"])
    ws = more.pop("workspace", None)
    if ws is None:
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    B.lora_kv4_tree_attention(c["cache"], c["q"], c["out"], c["start"], c["kv"], c["table"], c["max_q"], c["mask"],
                              scale or 1 / math.sqrt(c["d"]), ws, window=window, k_scale=K_SCALE, v_scale=V_SCALE,
                              lse=c["lse"], **more)
    return ws


def _keys(c, b, n=None):
    n = c["lengths"][b][1] if n is None else n
    k, v = R.read_cache(c["cache_np"], c["table_np"][b][:-(-n // c["page"])], n, c["page"], c["d"])
    return k * K_SCALE, v * V_SCALE


def _tree_check(c, window=0, some=None, gone=()):
    q, out, lse = _np(c["q"]), _np(c["out"]), c["lse"].cpu().numpy().astype(np.float64)
    for b, (m, n) in enumerate(c["lengths"]):
        if m == 0:
            continue
        k, v = _keys(c, b)
        pick = np.arange(m) if some is None or m <= some else np.unique(np.linspace(0, m - 1, some).astype(int))
        r = c["start_np"][b] + pick
        visible = T.tree_visible(n, c["sees"][b], window)[pick]
        for page in gone:
            visible[:, page * c["page"]:(page + 1) * c["page"]] = False
        want, wlse, size, span = T.attention(q[r], k, v, 1 / math.sqrt(c["d"]), visible)
        tol = HALF_UNIT[c["dtype"]] * np.abs(want) + BOTTOM[c["dtype"]] + \
            (2.0 ** -11 + FP32 + FP32 * span[..., None]) * size + 2.0 ** -25 * size.max(initial=0) * max(1, n) ** 0.5
        bad = ~(np.abs(out[r] - want) <= tol)
        assert not bad.any(), (b, m, n, bad.sum(), np.argwhere(bad)[:3], out[r][bad][:3], want[bad][:3])
        none = np.isneginf(wlse)
        assert np.array_equal(np.isneginf(lse[r]), none)
        err = np.abs(lse[r][~none] - wlse[~none])
        assert (err <= FP32 * (1 + span[~none] + np.abs(wlse[~none]))).all(), (b, m, n, err.max())
        assert (out[r][none] == 0).all()
    last = c["start_np"][-1]
    assert (c["out"][last:] == 7).all() and (c["lse"][last:] == 7).all(), "a row past the last sequence was written"


TREES = [
    # lengths (rows, keys), q heads, kv heads, d, page
    ([(1, 1)], 1, 1, 128, 16), ([(1, 40)], 4, 1, 64, 16), ([(2, 2), (3, 17), (4, 33)], 4, 2, 128, 16),
    ([(5, 700), (0, 20), (2, 31)], 8, 8, 64, 32), ([(15, 700)], 32, 8, 128, 16), ([(8, 300), (7, 45)], 20, 4, 128, 48),
    ([(4, 2000), (1, 77)], 16, 2, 64, 1024), ([(16, 16), (16, 15), (16, 3)], 4, 4, 128, 16),
    ([(33, 40), (31, 100), (32, 32)], 8, 2, 128, 16), ([(64, 600), (9, 1500)], 4, 1, 64, 64), ([(65, 65)], 4, 2, 64, 16),
    ([(100, 500), (37, 130), (1, 60)], 6, 2, 128, 32), ([(200, 333), (0, 0), (64, 64)], 8, 8, 128, 16),
    ([(130, 100), (2, 1), (40, 0)], 5, 1, 128, 16), ([(60, 3000), (50, 2000)], 2, 2, 128, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", range(len(TREES)))
def test_tree_attention(shape, dtype):
    c = _tree_case(*TREES[shape], dtype, seed=shape)
    status = _status()
    _tree(c, status=status)
    _tree_check(c, some=60)
    assert status[0].item() == 0


@pytest.mark.parametrize("window", [1, 2, 17, 40, 300])
@pytest.mark.parametrize("shape", [2, 3, 4, 8, 9, 11, 13])
def test_tree_attention_in_a_window(shape, window):
    c = _tree_case(*TREES[shape], "bf16", seed=50 + shape)
    _tree(c, window)
    _tree_check(c, window, some=40)


@pytest.mark.parametrize("shape", [2, 5, 8, 11, 13])
def test_masks_of_any_kind(shape):
    """Rows that see nothing of the tree, all of it, not themselves; bits behind the tree; spare words."""
    c = _tree_case(*TREES[shape], "bf16", seed=70 + shape, words=7)
    rng = np.random.default_rng(shape)
    for s in c["sees"]:
        if len(s):
            s[:] = rng.random(s.shape) < 0.4
            s[rng.integers(len(s))] = False
            s[rng.integers(len(s))] = True
    for stray in (0, 1):
        for window in (0, 30):
            _set_masks(c, stray)
            _tree(c, window)
            _tree_check(c, window, some=60)


@pytest.mark.parametrize("lengths", [[(3, 4), (2, 2)], [(40, 41), (70, 70)]])
def test_rows_without_any_key(lengths):
    """Empty masks and no key in front, or a window that ends before it."""
    c = _tree_case([lengths[0], (lengths[1][0], lengths[1][0])], 4, 1, 64, 16, "bf16", seed=3)
    for s in c["sees"]:
        s[0] = False
    c["sees"][1][:] = False
    _set_masks(c)
    _tree(c)
    _tree_check(c)
    _tree(c, window=1)
    _tree_check(c, window=1)


def test_a_chain_is_causal_attention():
    """Chains of drafted tokens by both calls: the same rows over the same keys, to the bit where the
    kernels split them alike (no windows, the same ends)."""
    for lengths in ([(5, 300), (3, 90)], [(70, 500), (33, 200)]):
        c = _tree_case(lengths, 8, 2, 128, 16, "bf16", seed=9)
        c["sees"] = [np.tril(np.ones((m, m), bool)) for m, _ in lengths]
        _set_masks(c)
        _tree(c, window=120)
        _tree_check(c, window=120)
        got = c["out"].float()
        ws = torch.zeros(B.lora_kv4_attention_workspace_size(2, c["rows"], c["max_q"], 8, 2, 128), dtype=torch.uint8,
                         device="cuda")
        B.lora_kv4_attention(c["cache"], c["q"], c["out"], c["start"], c["kv"], c["table"], c["max_q"],
                             1 / math.sqrt(128), ws, window=1000, k_scale=K_SCALE, v_scale=V_SCALE)
        chain = c["out"].float().clone()
        _tree(c, window=1000)
        # two roundings of the output, two of the probabilities of values of at most 6
        assert ((c["out"].float() - chain).abs() <= 2.0 ** -7 * chain.abs() + 2.0 ** -9 * 6).all()
        assert not torch.equal(got, chain)


@pytest.mark.parametrize("lengths", [[(20, 30000), (3, 9000)], [(100, 9000)]])
def test_tree_attention_over_long_keys(lengths):
    c = _tree_case(lengths, 4, 1, 128, 64, "bf16", seed=7)
    ws = _tree(c)
    _tree_check(c, some=6)
    first = c["out"].clone(), c["lse"].clone()
    for _ in range(3):  # the same workspace, the same bits
        _tree(c, workspace=ws)
        assert torch.equal(c["out"], first[0]) and torch.equal(c["lse"], first[1])


@pytest.mark.parametrize("window", [0, 400])
def test_trees_that_go_by_either_kernel(window):
    """Few sequences, in a table with room for many keys: short ones, long ones and single rows, each by the
    kernel that its own length calls for."""
    c = _tree_case([(40, 300), (1, 30000), (40, 30000), (3, 5000), (0, 9), (37, 40)], 4, 1, 128, 64, "bf16", seed=21)
    _tree(c, window)
    _tree_check(c, window, some=8)


def test_tree_attention_of_many_sequences_and_strided_rows():
    rng = np.random.default_rng(18)
    lengths = [(int(rng.integers(0, 20)), int(rng.integers(0, 90))) for _ in range(400)]
    lengths[7], lengths[300] = (70, 150), (120, 1000)
    c = _tree_case(lengths, 4, 2, 64, 16, "f16", seed=18, pad=24)
    c["out"] = torch.full((c["rows"], 4 * 64 + 40), 7, dtype=torch.float16, device="cuda")[:, :256].unflatten(1, (4, 64))
    _tree(c)
    _tree_check(c, some=30)


@pytest.mark.parametrize("rows", [4, 60])
def test_nan_values_reach_only_rows_that_see_them(rows):
    c = _tree_case([(rows, 200)], 4, 2, 128, 16, "bf16", seed=22)
    node = rows // 2
    key = 200 - rows + node
    for x in T.entry(c["cache_np"], c["table_np"][0], 16, key, 128)[3:]:
        x[:, 2] = 0x7F  # a NaN scale of V: dimensions 32 to 47
    c["cache"] = torch.tensor(c["cache_np"]).cuda()
    _tree(c)
    out = _np(c["out"])[:rows]
    nan = np.isnan(out)
    want = np.zeros(out.shape, bool)
    want[c["sees"][0][:, node], :, 32:48] = True
    assert np.array_equal(nan, want) and 0 < c["sees"][0][:, node].sum() < rows


def test_tree_attention_of_what_only_the_data_shows():
    c = _tree_case([(6, 300), (50, 400)], 4, 2, 64, 16, "bf16", seed=30)
    status = _status()
    table = c["table"].clone()
    table[0, 3], table[1, 3] = -5, c["cache"].shape[0]
    c["table"] = table
    _tree(c, status=status)
    _tree_check(c, gone=[3])
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_SLOT
    c["max_q"] = 20
    c["out"].fill_(7)
    _tree(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_LENGTH | B.LORA_STATUS_BAD_SLOT
    assert (c["out"][26:] == 7).all() and torch.isfinite(c["out"][:26].float()).all()


# ------------------------------------------------------------------ the accepted path

def _path_case(paths, heads, d, page, drafted, keys, seed=0, wide=None):
    rng = np.random.default_rng(seed)
    per = [-(-n // page) for n in keys]
    pages = sum(per) + 3
    order = rng.permutation(pages)
    table = np.full((len(keys), max(1, max(per))), -7, np.int64)
    at = 0
    for b, m in enumerate(per):
        table[b, :m] = order[at:at + m]
        at += m
    cache = rng.integers(0, 256, (pages, heads, page // 16, 18 * d), dtype=np.uint8)
    wide = wide or max(1, max(len(p) for p in paths))
    path = np.full((len(paths), wide), -9, np.int64)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    return dict(cache_np=cache, cache=torch.tensor(cache).cuda(), table_np=table, table=_i32(table), page=page, d=d,
                start=_i32(np.concatenate([[0], np.cumsum(drafted)])), kv=_i32(keys), path=_i32(path),
                len=_i32([len(p) for p in paths]), out=_i32([-1] * len(paths)), paths=paths, drafted=drafted, keys=keys)


def _accept(c, **more):
    B.lora_kv4_accept(c["cache"], c["start"], c["kv"], c["table"], c["path"], c["len"], c["out"], **more)


def _accept_check(c):
    want = c["cache_np"].copy()
    for b, path in enumerate(c["paths"]):
        base = c["keys"][b] - c["drafted"][b]
        T.move(want, c["table_np"][b], c["page"], c["d"], [base + x for x in path], [base + i for i in range(len(path))])
        assert c["out"][b].item() == base + len(path)
    got = c["cache"].cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,page", [(1, 16), (3, 32), (8, 48), (32, 64)])
def test_accept(heads, page, d):
    rng = np.random.default_rng(heads)
    drafted, keys, paths = [], [], []
    for _ in range(20):
        m = int(rng.integers(0, 70))
        sees = T.tree(rng, m)
        drafted.append(m)
        keys.append(m + int(rng.integers(0, 200)))
        paths.append([int(x) for x in np.nonzero(sees[rng.integers(m)])[0]] if m and rng.random() < 0.9 else [])
    c = _path_case(paths, heads, d, page, drafted, keys, seed=heads + d)
    status = _status()
    _accept(c, status=status)
    _accept_check(c)
    assert status[0].item() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_accept_of_any_order_and_repeats(d):
    rng = np.random.default_rng(4)
    paths = [[3, 2, 1, 0], [5, 5, 5], [1, 0], [int(x) for x in rng.permutation(300)], list(range(40)),
             [int(x) for x in rng.integers(0, 512, 512)]]
    c = _path_case(paths, 5, d, 16, [4, 6, 2, 300, 40, 512], [4, 60, 33, 1000, 41, 700], seed=4)
    _accept(c)
    _accept_check(c)


def test_accept_of_what_only_the_data_shows():
    c = _path_case([[0, 2], [1, 3], [2], [0, 1, 2]], 2, 64, 16, [3, 4, 3, 4], [40, 50, 60, 30], seed=5, wide=3)
    status = _status()
    c["path"][0, 1], c["path"][1, 0] = 3, -2  # no such rows
    _accept(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_LENGTH
    c["paths"][0], c["paths"][1] = [0, 1], [0, 3]  # left where they are
    _accept_check(c)
    c = _path_case([[1, 2, 3], [1], [3], [2]], 2, 64, 16, [4, 2, 4, 3], [20, 18, 60, 30], seed=6)
    c["len"] = _i32([9, -1, 1, 1])
    c["kv"] = _i32([20, 18, 60, 10 ** 6])
    _accept(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_LENGTH | B.LORA_STATUS_BAD_SLOT
    room = c["table"].shape[1] * 16  # the last sequence's keys behind its pages are not there
    assert c["out"].tolist() == [19, 16, 57, room - 3 + 1]
    c["paths"][1], c["paths"][3], c["out"] = [], [], _i32([19, 16, 57, 27])
    _accept_check(c)


# ------------------------------------------------------------------ the keys' weights

def _weights_case(lengths, qh, kvh, d, page, dtype, seed=0, window=0, paths=None, capacity=None, some=None, **more):
    """A batch with the lse that its rows have; with paths, lengths are those after the acceptance and
    each sequence has 8 rows more in q than its path names."""
    c = _attend_case(lengths, qh, kvh, d, page, dtype, seed=seed, **more)
    rng = np.random.default_rng(seed + 5)
    c["capacity"] = capacity or max(1, max(n for _, n in lengths))
    c["w_np"] = rng.random((len(lengths), kvh, c["capacity"])).astype(np.float32)
    c["w"] = torch.tensor(c["w_np"]).cuda()
    c["window"], c["path"], c["len"] = window, None, None
    c["rows_of"] = [np.arange(c["start_np"][b], c["start_np"][b + 1]) for b in range(len(lengths))]
    if paths:
        spread = [np.sort(rng.permutation(m + 8)[:m]) for m, _ in lengths]
        start = np.concatenate([[0], np.cumsum([m + 8 for m, _ in lengths])])
        rows = int(start[-1]) + 2
        q = rng.standard_normal((rows, qh, d))
        c["q"] = torch.tensor(q, dtype=torch.float32).to(c["q"].dtype).cuda()
        c["start"], c["start_np"], c["rows"] = _i32(start), start, rows
        wide = max(m for m, _ in lengths) + 1
        path = np.full((len(lengths), wide), -3, np.int64)
        for b, p in enumerate(spread):
            path[b, :len(p)] = p
        c["path"], c["len"] = _i32(path), _i32([m for m, _ in lengths])
        c["rows_of"] = [start[b] + p for b, p in enumerate(spread)]
        c["max_q"] = max(m for m, _ in lengths)
    q = _np(c["q"])
    lse = rng.standard_normal((c["rows"], qh))
    for b, (m, n) in enumerate(lengths):
        if m and n:
            k, v = _keys(c, b)
            x = np.einsum("rhd,khd->rhk", q[c["rows_of"][b]], np.repeat(k, qh // kvh, 1)) / math.sqrt(d)
            x = np.where(T.causal_visible(n, m, window)[:, None], x, -np.inf)
            top = x.max(-1)
            with np.errstate(divide="ignore", invalid="ignore"):
                lse[c["rows_of"][b]] = np.where(np.isneginf(top), -np.inf, top + np.log(np.exp(
                    x - np.where(np.isneginf(top), 0, top)[..., None]).sum(-1)))
        else:
            lse[c["rows_of"][b]] = -np.inf
    c["lse"] = torch.tensor(lse, dtype=torch.float32).cuda()
    return c


def _weights(c, **more):
    B.lora_kv4_key_weights(c["w"], c["cache"], c["q"], c["lse"], c["start"], c["kv"], c["table"], c["max_q"],
                           1 / math.sqrt(c["d"]), **{"window": c["window"], "k_scale": K_SCALE, "path": c["path"],
                                                     "path_len": c["len"], **more})


def _formula(q, lse, k, scale, visible, w):
    """T.key_weights of many rows at once."""
    g = q.shape[1] // k.shape[1]
    new, size = w.astype(np.float64), np.zeros(w.shape)
    m, n = visible.shape
    new[:, max(0, n - m):n] = 0
    for h in range(q.shape[1]):
        x, span = q[:, h] @ k[:, h // g].T * scale, np.abs(q[:, h]) @ np.abs(k[:, h // g]).T * scale
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(visible & ~np.isneginf(lse[:, h])[:, None], np.exp(x - lse[:, h, None]), 0)
        new[h // g, :n] += p.sum(0)
        size[h // g, :n] += (p * (1 + span + np.where(p > 0, np.abs(lse[:, h, None]), 0))).sum(0)
    return new, size


def _weights_check(c):
    q, lse, got = _np(c["q"]), c["lse"].cpu().numpy().astype(np.float64), c["w"].cpu().numpy()
    for b, (m, n) in enumerate(c["lengths"]):
        cap = c["capacity"]
        if m == 0:
            assert np.array_equal(got[b], c["w_np"][b])
            continue
        full = np.zeros((c["kvh"], max(n, cap)))
        full[:, :cap] = c["w_np"][b]
        k, _ = _keys(c, b)
        r = c["rows_of"][b]
        want, size = _formula(q[r], lse[r], k, 1 / math.sqrt(c["d"]), T.causal_visible(n, m, c["window"]), full)
        tol = FP32 * size + 2.0 ** -22 * np.abs(want)
        bad = ~(np.abs(got[b] - want[:, :cap]) <= tol[:, :cap])
        assert not bad.any(), (b, m, n, bad.sum(), np.argwhere(bad)[:4], got[b][bad][:4], want[:, :cap][bad][:4])
        assert np.array_equal(got[b][:, n:], c["w_np"][b][:, n:]), "a weight behind the last key was written"
        if c["window"]:
            lo = max(0, n - m - c["window"] + 1)
            assert np.array_equal(got[b][:, :lo], c["w_np"][b][:, :lo])


WEIGHTS = [
    ([(1, 1)], 1, 1, 128, 16), ([(1, 15), (1, 16), (1, 17), (1, 0)], 4, 2, 64, 16), ([(1, 700)], 32, 8, 128, 16),
    ([(1, n) for n in (5, 257, 1000, 31, 511, 64)], 8, 1, 128, 64), ([(2, 300), (0, 45), (3, 3)], 20, 4, 128, 48),
    ([(4, 100), (1, 3), (5, 2), (2, 0)], 8, 2, 64, 32), ([(7, 300), (2, 310)], 6, 3, 64, 16),
    ([(16, 16), (1, 2000)], 4, 4, 128, 1024), ([(33, 40), (1, 100), (8, 600)], 8, 2, 128, 16),
    ([(70, 70), (65, 200)], 4, 2, 64, 64), ([(130, 500), (3, 900)], 5, 1, 128, 32),
    ([(300, 290), (129, 129), (1, 700), (5, 0)], 6, 2, 128, 16), ([(257, 600)], 2, 2, 64, 16),
    ([(520, 900)], 3, 1, 128, 64), ([(400, 1500), (31, 257)], 16, 2, 128, 16), ([(128, 128)], 1, 1, 128, 16),
    ([(129, 1000)], 24, 1, 64, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", range(len(WEIGHTS)))
def test_key_weights(shape, dtype):
    c = _weights_case(*WEIGHTS[shape], dtype, seed=shape)
    status = _status()
    _weights(c, status=status)
    _weights_check(c)
    assert status[0].item() == 0


@pytest.mark.parametrize("window", [1, 16, 100, 1000])
@pytest.mark.parametrize("shape", [3, 4, 5, 8, 10, 11, 13])
def test_key_weights_in_a_window(shape, window):
    c = _weights_case(*WEIGHTS[shape], "bf16", seed=30 + shape, window=window)
    _weights(c)
    _weights_check(c)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", range(2, 12))
def test_key_weights_of_paths(shape, dtype):
    c = _weights_case(*WEIGHTS[shape], dtype, seed=60 + shape, paths=True)
    _weights(c)
    _weights_check(c)


@pytest.mark.parametrize("shape", [2, 8, 11])
def test_key_weights_add_up(shape):
    """A second call adds the same to the older keys, and a third begins the newest anew."""
    c = _weights_case(*WEIGHTS[shape], "bf16", seed=80 + shape)
    _weights(c)
    _weights_check(c)
    c["w_np"] = c["w"].cpu().numpy()
    _weights(c)
    _weights_check(c)


def test_key_weights_do_not_depend_on_the_batch():
    """A sequence alone and among others: the same bits."""
    lengths = [(1, 900), (3, 333), (64, 700), (1, 50), (200, 350)]
    c = _weights_case(lengths, 8, 2, 128, 16, "bf16", seed=90)
    _weights(c)
    for b, (m, n) in enumerate(lengths):
        r = slice(int(c["start_np"][b]), int(c["start_np"][b + 1]))
        w = torch.tensor(c["w_np"][b:b + 1]).cuda()
        B.lora_kv4_key_weights(w, c["cache"], c["q"][r], c["lse"][r], _i32([0, m]), c["kv"][b:b + 1],
                               c["table"][b:b + 1], min(m, c["max_q"]), 1 / math.sqrt(128), k_scale=K_SCALE)
        same = torch.equal(w[0], c["w"][b])
        # (which kernel has a sequence may follow the bound on the rows: then within both roundings)
        assert same or (w[0] - c["w"][b]).abs().max() <= FP32 * 32 * (1 + c["w"][b].abs().max())
    again = torch.tensor(c["w_np"]).cuda()
    c["w"], first = again, c["w"]
    _weights(c)
    assert torch.equal(c["w"], first)


@pytest.mark.parametrize("seqs", [31, 33, 255, 256, 257, 600])
def test_key_weights_of_many_sequences(seqs):
    rng = np.random.default_rng(seqs)
    lengths = [(int(rng.integers(0, 4)), int(rng.integers(0, 60))) for _ in range(seqs)]
    lengths[0] = lengths[-1] = (0, 5)
    lengths[seqs // 2] = (1, 3000)
    lengths[3] = (90, 130)
    c = _weights_case(lengths, 4, 2, 64, 16, "f16", seed=seqs)
    _weights(c)
    _weights_check(c)


def test_key_weights_of_strided_rows_and_a_spare_capacity():
    c = _weights_case([(3, 200), (80, 300)], 4, 2, 128, 16, "bf16", seed=91, pad=24, capacity=1000)
    _weights(c)
    _weights_check(c)


@pytest.mark.parametrize("rows", [1, 100])
def test_key_weights_of_what_only_the_data_shows(rows):
    status = _status()
    c = _weights_case([(rows, 300), (2, 90)], 4, 2, 64, 16, "bf16", seed=92, capacity=200)
    _weights(c, status=status)  # keys from 200 on have no weight
    _weights_check(c)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_LENGTH
    c = _weights_case([(rows, 300), (2, 90)], 4, 2, 64, 16, "bf16", seed=93)
    c["table"][0, 2] = -1
    _weights(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_SLOT
    gone = c["w"][0, :, 32:48].clone()
    fresh = 300 - rows
    want = torch.tensor(c["w_np"][0, :, 32:48]).cuda()
    want[:, max(0, fresh - 32):] = 0
    assert torch.equal(gone, want)
    c["w"][0, :, 32:48] = torch.tensor(_formula(
        _np(c["q"])[c["rows_of"][0]], c["lse"].cpu().numpy().astype(np.float64)[c["rows_of"][0]], _keys(c, 0)[0], 1 / 8,
        T.causal_visible(300, rows, 0), c["w_np"][0])[0][:, 32:48])
    _weights_check(c)


@pytest.mark.parametrize("bound", [1, 5, 70])
def test_rows_beyond_the_bound_add_nothing(bound):
    c = _weights_case([(6, 100), (90, 200)], 4, 2, 64, 16, "bf16", seed=94)
    status = _status()
    c["max_q"] = bound
    _weights(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_LENGTH
    for b, (m, n) in enumerate(c["lengths"]):  # as if they had no lse
        c["lse"][int(c["start_np"][b]) + min(m, bound):int(c["start_np"][b + 1])] = -math.inf
    _weights_check(c)


@pytest.mark.parametrize("rows", [2, 90])
def test_key_weights_of_rows_without_lse_and_of_nan(rows):
    c = _weights_case([(rows, 300)], 4, 2, 128, 16, "bf16", seed=95)
    c["lse"][0] = -math.inf
    _weights(c)
    _weights_check(c)
    c["w"].copy_(torch.tensor(c["w_np"]))
    c["lse"][1, 2] = math.nan  # a head of the second key head
    _weights(c)
    got = torch.isnan(c["w"][0]).cpu()
    at = 300 - rows + 1
    assert not got[0].any() and got[1, :at + 1].all() and not got[1, at + 1:].any()


@pytest.mark.parametrize("paths", [None, True])
@pytest.mark.parametrize("lengths", [[(5, 200), (4, 90), (7, 60)], [(90, 300), (70, 200), (131, 140)]])
def test_key_weights_of_a_sequence_beside_rows_of_nan(lengths, paths):
    """Another sequence's rows, those off the path, and those of no sequence may hold anything."""
    c = _weights_case(lengths, 6, 2, 64, 16, "bf16", seed=96, paths=paths)
    _weights(c)
    first = c["w"].clone()
    own = np.concatenate([c["rows_of"][0], c["rows_of"][2]])
    others = torch.tensor(np.setdiff1d(np.arange(c["rows"]), own)).cuda()
    assert len(others) > lengths[1][0]
    for q, lse in ((math.nan, 1.0), (math.inf, 1.0), (1.0, math.nan), (1.0, math.inf), (math.nan, math.nan)):
        c["q"][others], c["lse"][others] = q, lse
        c["w"].copy_(torch.tensor(c["w_np"]))
        _weights(c)
        for b in (0, 2):
            assert torch.equal(c["w"][b].view(torch.int32), first[b].view(torch.int32)), (q, lse, b)


@pytest.mark.parametrize("paths", [None, True])
@pytest.mark.parametrize("qh,kvh", [(100, 1), (65, 1), (44, 2), (26, 1), (34, 1), (6, 1), (130, 1)])
def test_key_weights_behind_a_call_of_nan(qh, kvh, paths):
    """What an earlier call has left in a tile's columns behind the last row is not read."""
    c = _weights_case([(60, 300), (1, 90), (30, 100)], qh, kvh, 64, 16, "bf16", seed=97, paths=paths)
    c["q"][c["rows"] - 1] = 2.0
    for value in (math.nan, 3e38, -3e38):
        e = _weights_case([(150, 6000)], 8, 8, 64, 16, "bf16", seed=98)  # more items than SMs, full tiles
        e["q"][:] = value
        _weights(e)
        c["w"].copy_(torch.tensor(c["w_np"]))
        _weights(c)
        _weights_check(c)


def test_key_weights_behind_the_attention():
    """lse as lora_kv4_attention leaves it: every row gives away a weight of one."""
    c = _weights_case([(1, 3000), (5, 700), (200, 260), (1, 1)], 8, 2, 128, 64, "bf16", seed=96)
    ws = torch.zeros(B.lora_kv4_attention_workspace_size(4, c["rows"], c["max_q"], 8, 2, 128), dtype=torch.uint8, device="cuda")
    B.lora_kv4_attention(c["cache"], c["q"], c["out"], c["start"], c["kv"], c["table"], c["max_q"], 1 / math.sqrt(128),
                         ws, k_scale=K_SCALE, v_scale=V_SCALE, lse=c["lse"])
    c["w"].zero_()
    _weights(c)
    total = c["w"].double().sum(-1).cpu()
    want = torch.tensor([4.0 * m for m, _ in c["lengths"]])[:, None].expand(-1, 2)
    # lse and the scores are off by 2^-16 of sum |q k|, at most 30 here
    assert ((total - want).abs() <= want * FP32 * 64).all(), total


# ------------------------------------------------------------------ eviction

def _evict_case(keys, heads, d, page, kind="spread", seed=0, capacity=None, held=None):
    rng = np.random.default_rng(seed)
    c = _path_case([[] for _ in keys], heads, d, page, [0] * len(keys), keys, seed=seed)
    cap = capacity or max(1, max(keys))
    shape = (len(keys), heads, cap)
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 4, shape).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":
        w = rng.standard_normal(shape).astype(np.float32)
        for x in (np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38):
            w[rng.random(shape) < 0.05] = x
    pos = np.full(shape, -1, np.int64)
    last = []
    for b, n in enumerate(keys):
        h = int((held if held is not None else rng.random()) * n)  # keys that an earlier call has left
        for k in range(heads):
            pos[b, k, :h] = rng.permutation(3 * max(h, 1))[:h]
        last.append(3 * max(h, 1) + (n - h))
    c.update(w_np=w, pos_np=pos, w=torch.tensor(w).cuda(), pos=_i32(pos), last=_i32(last), last_np=last, cap=cap)
    return c


def _evict(c, budget, sink=0, recent=0, **more):
    B.lora_kv4_evict(c["cache"], c["w"], c["pos"], c["kv"], c["last"], c["table"], budget, c["out"], sink=sink,
                     recent=recent, **more)


def _evict_check(c, budget, sink=0, recent=0):
    cache, w, pos = c["cache_np"].copy(), c["w_np"].copy(), c["pos_np"].copy()
    moves = 0
    for b, n in enumerate(c["keys"]):
        for h in range(w.shape[1]):
            w[b, h], pos[b, h], of, to = T.evict(w[b, h], pos[b, h], n, c["last_np"][b], budget, sink, recent)
            T.move(cache, c["table_np"][b], c["page"], c["d"], of, to, h)
            moves += len(of)
    assert c["out"].tolist() == [min(n, budget) for n in c["keys"]]
    got = c["pos"].cpu().numpy()
    assert np.array_equal(got, pos), (np.argwhere(got != pos)[:5], got[got != pos][:5], pos[got != pos][:5])
    assert np.array_equal(c["w"].cpu().numpy().view(np.int32), w.view(np.int32))
    got = c["cache"].cpu().numpy()
    assert np.array_equal(got, cache), f"{(got != cache).sum()} bytes differ"
    return moves


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("keys,heads,d,page,budget,sink,recent", [
    ([1, 2, 3, 0], 1, 64, 16, 1, 0, 0), ([40, 41, 39, 80], 3, 128, 16, 40, 4, 10), ([300], 8, 128, 32, 299, 0, 1),
    ([257, 255, 256, 600], 2, 64, 48, 256, 0, 256), ([1000, 30], 4, 128, 16, 100, 0, 0), ([700, 513], 2, 64, 64, 5, 3, 2),
    ([2100, 2049], 8, 128, 16, 2048, 4, 128), ([900], 2, 128, 1024, 450, 450, 0), ([5000, 3000], 2, 64, 16, 2500, 4, 64)])
def test_evict(keys, heads, d, page, budget, sink, recent, kind):
    c = _evict_case(keys, heads, d, page, kind, seed=budget)
    status = _status()
    _evict(c, budget, sink, recent, status=status)
    assert _evict_check(c, budget, sink, recent) >= 0
    assert status[0].item() == 0


@pytest.mark.parametrize("kind", ["spread", "ties"])
@pytest.mark.parametrize("keys,budget", [([15000], 7000), ([40000, 13000], 2000), ([14000], 13500), ([12289], 12288),
                                         ([60000], 43000), ([4096], 2000), ([4097], 4000)])
def test_evict_of_long_sequences(keys, budget, kind):
    """More keys than shared memory holds, more moves than are listed at a time."""
    c = _evict_case(keys, 2, 64, 64, kind, seed=budget, held=0.3)
    _evict(c, budget, 16, 100)
    assert _evict_check(c, budget, 16, 100) > 0


@pytest.mark.parametrize("kind", ["spread", "ties"])
@pytest.mark.parametrize("seqs,most,budget", [(20, 2600, 1200), (20, 900, 300), (62, 700, 300), (16, 3000, 900),
                                              (17, 5000, 4900)])
def test_evict_of_many_heads(seqs, most, budget, kind):
    """As many heads as SMs, some more and some fewer; of one sequence one key goes, of another all but the budget."""
    rng = np.random.default_rng(seqs + most)
    keys = [int(x) for x in rng.integers(1, most + 1, seqs)]
    keys[0], keys[-1], keys[3] = most, budget + 1, budget
    c = _evict_case(keys, 8, 64, 16, kind, seed=budget)
    status = _status()
    _evict(c, budget, 4, 20, status=status)
    assert _evict_check(c, budget, 4, 20) > 0
    assert status[0].item() == 0


def test_evict_again_and_again():
    """Steps of a few new keys: the positions of those that stay, and the newest, are kept."""
    c = _evict_case([64, 50], 2, 64, 16, seed=8, held=0.0)
    rng = np.random.default_rng(8)
    cap = 96
    c["cap"], keys, last = cap, [64, 50], [63, 49]
    c["table_np"] = np.array([[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11]])
    c["table"] = _i32(c["table_np"])
    c["cache_np"] = rng.integers(0, 256, (12, 2, 1, 18 * 64), dtype=np.uint8)
    c["cache"] = torch.tensor(c["cache_np"]).cuda()
    c["w_np"], c["pos_np"] = np.zeros((2, 2, cap), np.float32), np.full((2, 2, cap), -1, np.int64)
    c["pos"] = _i32(c["pos_np"])
    for step in range(12):
        new = int(rng.integers(1, 30))
        keys, last = [k + new for k in keys], [x + new for x in last]
        c["w_np"] += rng.random(c["w_np"].shape).astype(np.float32)
        c["w"] = torch.tensor(c["w_np"]).cuda()
        c["keys"], c["last_np"], c["kv"], c["last"] = keys, last, _i32(keys), _i32(last)
        _evict(c, 60, 2, 16)
        _evict_check(c, 60, 2, 16)
        c["w_np"], c["pos_np"] = c["w"].cpu().numpy(), c["pos"].cpu().numpy().astype(np.int64)
        c["cache_np"], keys = c["cache"].cpu().numpy(), c["out"].tolist()
        for b in range(2):
            for h in range(2):
                held = set(c["pos_np"][b, h, :keys[b]].tolist())
                assert len(held) == keys[b] and {0, 1} | set(range(last[b] - 15, last[b] + 1)) <= held


def test_evict_of_what_only_the_data_shows():
    c = _evict_case([60, 90], 2, 64, 16, seed=9, capacity=100)
    status = _status()
    c["kv"] = _i32([60, 2000])  # clamped to the table
    c["last_np"] = [c["last_np"][0], 2000]
    c["last"] = _i32(c["last_np"])
    _evict(c, 50, status=status)
    assert B.lora_read_status(status) & B.LORA_STATUS_BAD_LENGTH
    assert c["out"].tolist() == [50, 50]
    c = _evict_case([60, 90], 2, 64, 16, seed=10)
    c["table"][1] = -1  # nothing to move to or from: weights and positions go on
    _evict(c, 50, 0, 20, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_SLOT
    want = c["cache_np"].copy()
    for h in range(2):
        _, _, of, to = T.evict(c["w_np"][0, h], c["pos_np"][0, h], 60, c["last_np"][0], 50, 0, 20)
        T.move(want, c["table_np"][0], 16, 64, of, to, h)
        w, pos, _, _ = T.evict(c["w_np"][1, h], c["pos_np"][1, h], 90, c["last_np"][1], 50, 0, 20)
        assert np.array_equal(c["w"][1, h].cpu().numpy(), w) and np.array_equal(c["pos"][1, h].cpu().numpy(), pos)
    assert np.array_equal(c["cache"].cpu().numpy(), want)
    c = _evict_case([90], 2, 64, 16, seed=11)  # positions that no step leaves
    for last in (-5, -2 ** 31, 2 ** 31 - 1):
        c["last_np"], c["last"] = [last], _i32([last])
        _evict(c, 50, 5, 20)
        assert c["out"].tolist() == [50]


# ------------------------------------------------------------------ sizes at the ends

HEADS = [  # (q heads, key heads): packed rows that fill no tile, or more heads than a tile has rows
    (100, 1), (130, 1), (256, 1), (14, 2), (128, 128)]


@pytest.mark.parametrize("qh,kvh", HEADS)
def test_tree_attention_of_many_heads(qh, kvh):
    c = _tree_case([(1, 60), (3, 200), (9, 30)], qh, kvh, 64, 16, "bf16", seed=qh)
    _tree(c)
    _tree_check(c)


@pytest.mark.parametrize("paths", [False, True])
@pytest.mark.parametrize("qh,kvh", HEADS)
def test_key_weights_of_many_heads(qh, kvh, paths):
    c = _weights_case([(1, 60), (3, 600), (9, 30), (40, 300)], qh, kvh, 64, 16, "bf16", seed=qh, paths=paths)
    _weights(c)
    _weights_check(c)


@pytest.mark.parametrize("seqs", [1500, 3000])
def test_many_sequences(seqs):
    """Of every operator, more sequences than a CTA has threads."""
    rng = np.random.default_rng(seqs)
    lengths = [(int(rng.integers(0, 9)), int(rng.integers(0, 40))) for _ in range(seqs)]
    lengths[1] = (45, 60)
    c = _tree_case(lengths, 2, 1, 64, 16, "bf16", seed=seqs)
    _tree(c)
    _tree_check(c)
    c = _weights_case(lengths, 2, 1, 64, 16, "bf16", seed=seqs)
    _weights(c)
    _weights_check(c)
    c = _evict_case([n for _, n in lengths], 1, 64, 16, seed=seqs)
    _evict(c, 17, 1, 3)
    assert _evict_check(c, 17, 1, 3) > seqs
    paths = [[int(x) for x in rng.permutation(m)[:rng.integers(0, m + 1)]] for m, _ in lengths]
    c = _path_case(paths, 2, 64, 16, [m for m, _ in lengths], [m + n for m, n in lengths], seed=seqs)
    _accept(c)
    _accept_check(c)


def test_pages_past_four_gigabytes():
    """The same work on the last pages of a cache whose offsets pass 32 bits: the same bits."""
    far = 62000
    big = torch.empty(far + 300, 8, 4, 18 * 128, dtype=torch.uint8, device="cuda")
    assert far * big[0].numel() > 1 << 32
    t = _tree_case([(5, 700), (60, 900)], 16, 8, 128, 64, "bf16", seed=1)
    w = _weights_case([(5, 700), (60, 900), (1, 300)], 16, 8, 128, 64, "bf16", seed=2)
    a = _path_case([[1, 3], list(range(5, 45)), [3, 2, 1]], 8, 128, 64, [5, 60, 4], [700, 900, 100], seed=3)
    e = _evict_case([700, 5000], 8, 128, 64, seed=4)

    def moved(c):
        pages = c["cache"].shape[0]
        big[far:far + pages] = c["cache"]
        return {**c, "cache": big, "table": torch.where(c["table"] >= 0, c["table"] + far, c["table"])}, slice(far, far + pages)

    _tree(t)
    want = t["out"].clone()
    t["out"].fill_(7)
    _tree(moved(t)[0])
    assert torch.equal(t["out"], want)
    _weights(w)
    want = w["w"].clone()
    w["w"].copy_(torch.tensor(w["w_np"]))
    _weights(moved(w)[0])
    assert torch.equal(w["w"], want)
    m, at = moved(a)
    _accept(m)
    _accept_check({**a, "cache": big[at]})
    m, at = moved(e)
    _evict(m, 600, 4, 50)
    _evict_check({**e, "cache": big[at]}, 600, 4, 50)


# ------------------------------------------------------------------ the wrappers' refusals

def test_refusals():
    c = _tree_case([(3, 40)], 4, 2, 64, 16, "bf16")
    with pytest.raises(ValueError, match="tree_mask"):
        B.lora_kv4_tree_attention(c["cache"], c["q"], c["out"], c["start"], c["kv"], c["table"], 3, c["mask"].long(), 0.1,
                                  c["cache"])
    with pytest.raises(ValueError, match="tree_mask"):
        B.lora_kv4_tree_attention(c["cache"], c["q"], c["out"], c["start"], c["kv"], c["table"], 3, c["mask"][:2], 0.1,
                                  c["cache"])
    with pytest.raises(B.LoraError):
        B.lora_kv4_tree_attention(c["cache"], c["q"], c["out"], c["start"], c["kv"], c["table"], 3, c["mask"], 0.1,
                                  torch.zeros(16, dtype=torch.uint8, device="cuda"))
    p = _path_case([[1]], 2, 64, 16, [3], [40])
    for name in ("path", "len", "out", "table", "kv", "start"):
        with pytest.raises(ValueError):
            _accept({**p, name: p[name].long()})
    with pytest.raises(B.LoraError):
        _accept({**p, "out": p["kv"]})
    w = _weights_case([(3, 40)], 4, 2, 64, 16, "bf16")
    for name in ("w", "lse"):
        with pytest.raises(ValueError):
            _weights({**w, name: w[name].double()})
    with pytest.raises(ValueError, match="path"):
        _weights({**w, "path": p["path"]})
    with pytest.raises(ValueError, match="weights"):
        _weights({**w, "w": w["w"][:, :1]})
    e = _evict_case([40], 2, 64, 16)
    for name in ("w", "pos", "last", "kv", "out"):
        with pytest.raises(ValueError):
            _evict({**e, name: e[name].double()}, 10)
    for kw in (dict(budget=0), dict(budget=10, sink=6, recent=5), dict(budget=10, recent=-1)):
        with pytest.raises(B.LoraError):
            _evict(e, **kw)
    with pytest.raises(B.LoraError):
        _evict({**e, "out": e["kv"]}, 10)
    with pytest.raises(ValueError, match="budget"):
        _evict(e, 10.5)


# ------------------------------------------------------------------ together

def test_a_step_of_a_server_under_a_graph():
    """Append, tree attention, acceptance, weights and eviction, captured once and replayed over steps with
    other lengths, trees and paths, against the formulas on what the cache holds before each."""
    rng = np.random.default_rng(77)
    seqs, qh, kvh, d, page, budget, sink, recent = 3, 4, 2, 64, 16, 70, 2, 8
    rows, words, wide = 24, 1, 8  # pages a sequence
    cap = wide * page
    cache = torch.zeros(seqs * wide + 1, kvh, 1, 18 * d, dtype=torch.uint8, device="cuda")
    table_np = rng.permutation(seqs * wide).reshape(seqs, wide)
    q, k, v, out = (torch.zeros(rows, h, d, dtype=torch.bfloat16, device="cuda") for h in (qh, kvh, kvh, qh))
    lse = torch.zeros(rows, qh, device="cuda")
    table, n = _i32(table_np), _i32([0])
    slots, start, kv, kv2, kv3 = _i32([-1] * rows), _i32([0] * (seqs + 1)), *(_i32([0] * seqs) for _ in range(3))
    mask, path, plen, last = _i32(np.zeros((rows, words))), _i32(np.zeros((seqs, 8))), _i32([0] * seqs), _i32([0] * seqs)
    w, pos = torch.zeros(seqs, kvh, cap, device="cuda"), _i32(np.full((seqs, kvh, cap), -1))
    ws = torch.zeros(B.lora_kv4_attention_workspace_size(seqs, rows, 8, qh, kvh, d), dtype=torch.uint8, device="cuda")
    status = _status()
    scale = 1 / math.sqrt(d)

    def step():
        B.lora_kv4_append(cache, k, v, slots, n, k_scale=K_SCALE, v_scale=V_SCALE, status=status)
        B.lora_kv4_tree_attention(cache, q, out, start, kv, table, 8, mask, scale, ws, k_scale=K_SCALE, v_scale=V_SCALE,
                                  lse=lse, status=status)
        B.lora_kv4_accept(cache, start, kv, table, path, plen, kv2, status=status)
        B.lora_kv4_key_weights(w, cache, q, lse, start, kv2, table, 8, scale, k_scale=K_SCALE, path=path, path_len=plen,
                               status=status)
        B.lora_kv4_evict(cache, w, pos, kv2, last, table, budget, kv3, sink=sink, recent=recent, status=status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    w.zero_(), pos.fill_(-1)
    have, at, evicted = [0] * seqs, [0] * seqs, 0
    for _ in range(70):
        drafted = [int(rng.integers(0, 9)) for _ in range(seqs)]
        trees = [T.tree(rng, m) for m in drafted]
        paths = [[int(x) for x in np.nonzero(t[rng.integers(len(t))])[0]] if len(t) else [] for t in trees]
        paths = [p if len(p) > 1 or rng.random() < 0.7 else [] for p in paths]
        total = sum(drafted)
        start.copy_(_i32(np.concatenate([[0], np.cumsum(drafted)])))
        n.fill_(total)
        where = [table_np[b][j // page] * page + j % page for b, m in enumerate(drafted) for j in range(have[b], have[b] + m)]
        slots.copy_(_i32(where + [-1] * (rows - total)))
        for t in (q, k, v):
            t.copy_(torch.tensor(rng.standard_normal(tuple(t.shape)), dtype=torch.float32))
        kv.copy_(_i32([h + m for h, m in zip(have, drafted)]))
        mask[:total].copy_(_i32(np.concatenate([T.mask_words(t, 1) for t in trees]).reshape(total, 1)))
        plen.copy_(_i32([len(p) for p in paths]))
        path.copy_(_i32([p + [-1] * (8 - len(p)) for p in paths]))
        last.copy_(_i32([a + len(p) - 1 for a, p in zip(at, paths)]))
        before, w_np, pos_np = cache.cpu().numpy(), w.cpu().numpy(), pos.cpu().numpy().astype(np.int64)
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert status[0].item() == 0
        # the cache after the append, from the formula
        for t, part, factor in ((k, 0, K_SCALE), (v, 1, V_SCALE)):
            code, s8 = R.quantise32(_np(t).astype(np.float32), factor)
            for i, slot in enumerate(where):
                e = T.entry(before, np.arange(cache.shape[0]), page, slot, d)
                e[part][:], e[2 + part][:] = R.pack(code[i]), s8[i]
        row = 0
        for b, (m, p) in enumerate(zip(drafted, paths)):
            nk = have[b] + m
            kk, vv = (x * f for x, f in zip(R.read_cache(before, table_np[b], nk, page, d), (K_SCALE, V_SCALE)))
            r = slice(row, row + m)
            row += m
            want, wlse, size, span = T.attention(_np(q)[r], kk, vv, scale, T.tree_visible(nk, trees[b], 0))
            tol = HALF_UNIT["bf16"] * np.abs(want) + (2.0 ** -11 + FP32 + FP32 * span[..., None]) * size + \
                2.0 ** -25 * size.max(initial=0) * max(nk, 1) ** 0.5
            assert (np.abs(_np(out)[r] - want) <= tol).all()
            T.move(before, table_np[b], page, d, [have[b] + x for x in p], [have[b] + i for i in range(len(p))])
            nk = have[b] + len(p)
            kk = R.read_cache(before, table_np[b], nk, page, d)[0] * K_SCALE
            rr = np.array(p, int) + r.start
            left = min(nk, budget)
            if len(p):
                new, size = _formula(_np(q)[rr], lse.cpu().numpy().astype(np.float64)[rr], kk, scale,
                                     T.causal_visible(nk, len(p), 0), w_np[b])
                tolw = FP32 * size + 2.0 ** -22 * np.abs(new)
            else:
                new, tolw = w_np[b].astype(np.float64), np.zeros(w_np[b].shape)
            got_w, got_pos = w.cpu().numpy()[b], pos.cpu().numpy()[b]
            for h in range(kvh):
                # which keys stay may hang on the last bits of two weights: take them from the positions
                named = pos_np[b, h].copy()
                for j in range(nk):
                    if named[j] < 0:
                        named[j] = at[b] + len(p) - 1 - (nk - 1 - j)
                place = {int(x): j for j, x in enumerate(named[:nk])}
                of = [place[int(x)] for x in got_pos[h, :left]]
                assert len(set(of)) == left
                assert (np.abs(got_w[h, :left] - new[h, of]) <= tolw[h, of]).all()
                if nk > budget:
                    evicted += 1
                    gone = sorted(set(range(nk)) - set(of))
                    free = [j for j in range(nk) if not (named[j] < sink or named[j] > at[b] + len(p) - 1 - recent)]
                    assert set(gone) <= set(free)
                    kept = [j for j in of if j in set(free)]
                    assert min(new[h, kept]) >= max(new[h, gone]) - 2 * max(tolw[h, gone].max(), tolw[h, kept].max())
                    holes = [j for j in range(budget) if j in set(gone)]
                    movers = [j for j in range(budget, nk) if j in set(of)]
                    assert [of[j] for j in holes] == movers
                    T.move(before, table_np[b], page, d, movers, holes, h)
            at[b] += len(p)
            have[b] = left
        assert kv3.tolist() == have
        assert np.array_equal(cache.cpu().numpy(), before)
    assert evicted > 10


@pytest.mark.parametrize("rows", [3, 100])
def test_a_tree_attention_that_gives_up_says_so_and_the_next_is_whole(rows):
    c = _tree_case([(rows, 900), (2, 300)], 8, 2, 128, 16, "bf16", seed=40)
    status = _status()
    assert B.lora_testing_inject_timeout(True) is False
    try:
        ws = _tree(c, status=status)
        torch.cuda.synchronize()
    finally:
        assert B.lora_testing_inject_timeout(False) is True
    assert B.lora_read_status(status) == B.LORA_STATUS_TIMEOUT
    assert (c["out"] == 7).all()
    _tree(c, workspace=ws, status=status)
    _tree_check(c, some=30)
    assert B.lora_read_status(status) == 0


@pytest.mark.parametrize("paths", [False, True])
def test_key_weights_that_give_up_say_so_and_the_next_are_whole(paths):
    c = _weights_case([(60, 900), (300, 700)], 8, 2, 128, 16, "bf16", seed=41, paths=paths)
    status = _status()
    assert B.lora_testing_inject_timeout(True) is False
    try:
        _weights(c, status=status)
        torch.cuda.synchronize()
    finally:
        assert B.lora_testing_inject_timeout(False) is True
    assert B.lora_read_status(status) == B.LORA_STATUS_TIMEOUT
    assert np.array_equal(c["w"].cpu().numpy(), c["w_np"])
    _weights(c, status=status)
    _weights_check(c)
    assert B.lora_read_status(status) == 0


def test_two_streams():
    """Calls on two streams at once, and on a stream given by its handle: each has its own results."""
    one, two = (_weights_case([(1, 3000), (60, 500)], 8, 2, 128, 16, "bf16", seed=s) for s in (97, 98))
    ev = [_evict_case([900, 700], 4, 128, 16, seed=s) for s in (1, 2)]
    trees = [_tree_case([(5, 900), (50, 400)], 8, 2, 128, 16, "bf16", seed=s) for s in (3, 4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    spaces = [torch.zeros(B.lora_kv4_attention_workspace_size(2, c["rows"], c["max_q"], 8, 2, 128), dtype=torch.uint8,
                          device="cuda") for c in trees]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, c, t, ws in zip(streams, (one, two), trees, spaces):
            c["w"].record_stream(s)
            with torch.cuda.stream(s):
                c["w"].copy_(torch.tensor(c["w_np"]))
            _weights(c, stream=s)
            _tree(t, workspace=ws, stream=s.cuda_stream)
    for s, c in zip(streams, ev):
        _evict(c, 500, 4, 30, stream=s)
    torch.cuda.synchronize()
    for c in (one, two):
        _weights_check(c)
    for c in trees:
        _tree_check(c, some=30)
    for c in ev:
        _evict_check(c, 500, 4, 30)
