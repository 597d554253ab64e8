"""The operators around a layer's LoRA products where their contract is easily missed.  Helpers, and what
the tolerances rest on, are those of test_layer_gpu.py."""
import math

import numpy as np
import pytest

from gathered_rank_gemm_gb300 import binding as B
from tests import layer_ref as R
from tests.test_layer_gpu import (BOTTOM, FP32, HALF_UNIT, K_SCALE, V_SCALE, _append, _append_case,  # noqa: F401
                                  _append_check, _attend, _attend_case, _attend_check, _i32, _norm_case,
                                  _norm_check, _np, lib)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scores of any finite size

def _sequences(c):
    """Each sequence's rows of q, out and lse, and its keys and values in 64 bits."""
    for b, (m, n) in enumerate(c["lengths"]):
        r = slice(c["start_np"][b], c["start_np"][b + 1])
        k, v = R.read_cache(c["cache_np"], c["table_np"][b][:-(-n // c["page"])], n, c["page"], c["d"])
        yield (m, n, _np(c["q"])[r], _np(c["out"])[r], c["lse"].cpu().numpy().astype(np.float64)[r],
               k * K_SCALE, v * V_SCALE)


def _check_single_keys(c, scale):
    """Rows whose largest score leads by so much that its key has all the weight: the score's own
    rounding in fp32 (2^-16 of sum |q k|, as everywhere) is far below the lead."""
    checked = 0
    for m, n, q, out, lse, k, v in _sequences(c):
        for i in range(m):
            pos = n - m + i
            for h in range(c["qh"] if pos >= 0 else 0):
                g = h // (c["qh"] // c["kvh"])
                x = k[:pos + 1, g] @ q[i, h] * scale
                span = (np.abs(k[:pos + 1, g]) @ np.abs(q[i, h])).max() * scale
                best = int(x.argmax())
                if len(x) > 1 and x[best] - np.partition(x, -2)[-2] < max(100.0, FP32 * span):
                    continue
                want = v[best, g]
                assert (np.abs(out[i, h] - want) <= (HALF_UNIT[c["dtype"]] + FP32) * np.abs(want) + BOTTOM[c["dtype"]]).all(), \
                    (n, i, h, x[best], out[i, h][:3], want[:3])
                assert abs(lse[i, h] - x[best]) <= FP32 * span, (n, i, h, lse[i, h], x[best])
                checked += 1
    return checked


FAR = [2.0 ** 20, 2.0 ** 24, 2.0 ** 26, 2.0 ** 28, 2.0 ** 60]  # times q k of about 10
CHUNKS = [[(140, 300)], [(300, 290), (70, 600)]]
FEW = [[(1, 200), (2, 30)], [(1, 3000)], [(4, 700), (1, 90)], [(1, 500 + 7 * i) for i in range(40)]]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", FAR)
@pytest.mark.parametrize("lengths", CHUNKS + FEW)
def test_attention_of_large_scores(lengths, scale, dtype):
    """Past 2^27 the rounding of a score alone is more than fp16 holds as a power of two."""
    c = _attend_case(lengths, 4, 2, 128, 16, dtype, seed=31)
    _attend(c, scale=scale)
    total = sum(max(0, min(m, n)) for m, n in lengths) * 4
    assert _check_single_keys(c, scale) > 0.9 * total


@pytest.mark.parametrize("scale", FAR + [-1.0])
@pytest.mark.parametrize("lengths", CHUNKS + FEW)
def test_attention_of_equal_keys(lengths, scale):
    """Keys that are all the same share the weight equally, however large their score is."""
    c = _attend_case(lengths, 4, 2, 128, 16, "bf16", seed=32)
    if scale < 0:  # large negative scores
        scale = 2.0 ** 28
        c["q"].copy_(-c["q"].abs())
        c["cache_np"][..., :64] &= 0x77  # the first key of a block is above 0
    codes, _, scales, _ = R.sections(c["cache_np"], 128)
    first = c["table_np"][0][0]
    codes[:] = codes[first, :, 0, 0].copy()[:, None, None]
    scales[:] = scales[first, :, 0, 0].copy()[:, None, None]
    assert np.array_equal(R.sections(c["cache_np"], 128)[0], codes)
    c["cache"] = torch.tensor(c["cache_np"]).cuda()
    _attend(c, scale=scale)
    for m, n, q, out, lse, k, v in _sequences(c):
        for i in range(max(0, m - n), m):
            cut = n - m + i + 1
            for h in range(4):
                vv = v[:cut, h // 2]
                want, size = vv.mean(0), np.abs(vv).mean(0)
                tol = HALF_UNIT["bf16"] * np.abs(want) + (2.0 ** -11 + FP32) * size + 2.0 ** -25 * size.max() * cut ** 0.5
                assert (np.abs(out[i, h] - want) <= tol).all(), (n, i, h, out[i, h][:3], want[:3])
                span = np.abs(k[0, h // 2]) @ np.abs(q[i, h]) * scale
                assert abs(lse[i, h] - (k[0, h // 2] @ q[i, h] * scale + math.log(cut))) <= FP32 * (1 + span)


# ------------------------------------------------------------------ pages that are not there

def _check_without(c, gone, some=None):
    """The last row of each sequence against the formula over the keys that are there."""
    scale = 1 / math.sqrt(c["d"])
    for b, (m, n, q, out, lse, k, v) in enumerate(_sequences(c)):
        if m == 0:
            continue
        there = np.ones(n, bool)
        for a in gone.get(b, ()):
            there[a * c["page"]:(a + 1) * c["page"]] = False
        want, wlse, size, span = R.attention(q[-1:], k[there], v[there], scale, 0)
        tol = HALF_UNIT[c["dtype"]] * np.abs(want) + (2.0 ** -11 + FP32 + FP32 * span[..., None]) * size + \
            2.0 ** -25 * size.max() * n ** 0.5
        assert (np.abs(out[-1:] - want) <= tol).all(), (b, n, np.abs(out[-1:] - want).max())
        assert (np.abs(lse[-1:] - wlse) <= FP32 * (1 + span + np.abs(wlse))).all(), (b, n, lse[-1:] - wlse)


def _pool_case(lengths, qh, kvh, d, page, dtype, seed, pool=600):
    """Long sequences whose pages are drawn, many times each, from a few."""
    rows, pages = sum(m for m, _ in lengths), -(-pool // page)
    c = _attend_case([(rows, pages * page)], qh, kvh, d, page, dtype, seed=seed)
    rng = np.random.default_rng(seed)
    table = c["table_np"][0][rng.integers(0, pages, (len(lengths), max(-(-n // page) for _, n in lengths)))]
    start = np.concatenate([[0], np.cumsum([m for m, _ in lengths])])
    return dict(c, lengths=lengths, table=_i32(table), table_np=table, start=_i32(start), start_np=start,
                kv=_i32([n for _, n in lengths]), max_q=max(m for m, _ in lengths))


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("heads", [1, 32])
@pytest.mark.parametrize("lengths,keys", [
    ([(1, 1500)], [600]), ([(1, 9000)], [600, 5000, 8990]), ([(1, 20000), (1, 25000)], [4000, 8128, 17000, 19990]),
    ([(1, 3000 + 10 * i) for i in range(20)], [700, 2000, 2900]), ([(12, 30000), (1, 600)], [100, 5000, 29000]),
    ([(40, 5000)], [600, 3000, 4800])])
def test_attention_masks_pages_that_are_not_there_wherever_they_are(lengths, keys, heads, page):
    """Near and far from the beginning of what one warp, or one CTA, reads of a sequence."""
    c = _pool_case(lengths, heads, heads, 64, page, "bf16", seed=33)
    gone = {b: [j // page for j in keys if j < n] for b, (_, n) in enumerate(lengths)}
    for b, pages in gone.items():
        for i, a in enumerate(pages):
            c["table"][b, a] = -1 if i % 2 else c["cache"].shape[0]
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    _attend(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_SLOT
    _check_without(c, gone)


@pytest.mark.parametrize("page", [16, 32, 48])
@pytest.mark.parametrize("window", [1, 17, 100, 300])
@pytest.mark.parametrize("lengths", [[(1, 900), (1, 60)], [(5, 700)], [(140, 500), (70, 1000)], [(300, 1200), (1, 400)]])
def test_pages_in_front_of_a_window_are_not_looked_up(lengths, window, page):
    """A server gives such pages to others: their entries may hold anything."""
    c = _attend_case(lengths, 4, 2, 64, page, "bf16", seed=34)
    for b, (m, n) in enumerate(lengths):
        c["table"][b, :max(0, n - m - window + 1) // page] = -1
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    _attend(c, window, status=status)
    assert B.lora_read_status(status) == 0
    _attend_check(c, window, some=20)


# ------------------------------------------------------------------ the ends of the ranges

@pytest.mark.parametrize("lengths", [[(1, 200), (2, 30)], [(140, 300)]])
def test_attention_of_queries_of_next_to_nothing(lengths):
    """Scores that underflow are all 0: the keys that a row sees share the weight."""
    c = _attend_case(lengths, 4, 2, 64, 16, "bf16", seed=35)
    c["q"].mul_(2.0 ** -120)
    _attend(c, scale=1e-12)
    _attend_check(c, scale=1e-12, some=20)


@pytest.mark.parametrize("lengths", [[(8, 3), (3, 3), (1, 1)], [(140, 100), (1, 5)], [(300, 290)]])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 200])
def test_attention_in_a_window_of_any_size(lengths, window):
    c = _attend_case(lengths, 4, 2, 128, 16, "bf16", seed=36)
    _attend(c, window)
    _attend_check(c, 0, some=25)  # wider than any sequence: no window at all


@pytest.mark.parametrize("rows", [1, 60])
def test_attention_of_as_many_keys_as_an_integer_holds(rows):
    """2^31 - 16 keys in a window of 300, every page the same one."""
    page, wide, window = 16, 2 ** 27 - 1, 300
    c = _attend_case([(rows, page)], 4, 2, 64, page, "bf16", seed=37)
    c["table"] = torch.full((1, wide), int(c["table_np"][0, 0]), dtype=torch.int32, device="cuda")
    c["kv"] = _i32([wide * page])
    _attend(c, window)
    got, lse = _np(c["out"]), c["lse"].cpu().numpy().astype(np.float64)
    k, v = (np.tile(x, (400 // page, 1, 1)) for x in R.read_cache(c["cache_np"], c["table_np"][0][:1], page, page, 64))
    q = _np(c["q"])
    for i in range(rows):
        cut = slice(0, 400 - rows + i + 1)
        want, wlse, size, span = R.attention(q[i:i + 1], k[cut] * K_SCALE, v[cut] * V_SCALE, 0.125, window)
        tol = HALF_UNIT["bf16"] * np.abs(want) + (2.0 ** -11 + FP32 + FP32 * span[..., None]) * size + 2.0 ** -25 * size.max() * 20
        assert (np.abs(got[i] - want[0]) <= tol[0]).all(), (i, got[i, 0, :3], want[0, 0, :3])
        assert (np.abs(lse[i] - wlse[0]) <= FP32 * (1 + span[0] + np.abs(wlse[0]))).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("weight", [20.3, 25.1])
@pytest.mark.parametrize("lengths", [[(1, 1 << 17), (1, 900)], [(1, 1 << 17)] * 304, [(70, 1 << 17)] * 160])
def test_attention_of_one_key_above_a_long_flat_tail(lengths, weight, dtype):
    """The first key weighs 1, each other one 2^-20.3 (all of them 10 %) or 2^-25.1 (0.4 %), all of one sign in
    V.  Next to a sum of 1 an fp32 accumulator of the tensor cores keeps multiples of 2^-23, so a key may
    lose that much; a probability's own rounding (2^-25) lies below.  (Many sequences: one that is cut has
    its first key in one of its runs only.)"""
    c = _pool_case(lengths, 1, 1, 64, 16, dtype, seed=38, pool=32)
    codes, vcodes, scales, vscales = R.sections(c["cache_np"], 64)
    codes[:], vcodes[:], scales[:], vscales[:] = 0, 0x22, 0x38, 0x38  # K 0, V 1
    first, tail = c["table_np"].min(), c["table_np"].max()
    assert first != tail
    codes[first, :, 0, 0, :8] = 0x22  # a key of 1 in each of the first 16 dimensions
    c["table_np"][:] = tail
    c["table_np"][:, 0] = first
    c["table"], c["cache"] = _i32(c["table_np"]), torch.tensor(c["cache_np"]).cuda()
    c["q"].fill_(1)
    scale = weight * math.log(2) / (16 * K_SCALE)
    _attend(c, scale=scale)
    out, lse = _np(c["out"]) / V_SCALE, c["lse"].cpu().numpy()
    for b, (m, n) in enumerate(lengths):
        for i in {0, m // 2, m - 1}:
            keys, row = n - m + i + 1, c["start_np"][b] + i
            tol = HALF_UNIT[dtype] + 2.0 ** -11 + 2.0 ** -23 * keys
            assert (np.abs(out[row] - 1) <= tol).all(), (keys, out[row, 0, :2])
            want = weight * math.log(2) + math.log1p((keys - 1) * 2.0 ** -weight)
            assert abs(lse[row, 0] - want) <= FP32 * (1 + 2 * want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lengths", [[(6, 700), (2, 90)], [(200, 900)]])
def test_an_infinite_query_leaves_the_other_rows_as_they_are(lengths, dtype):
    c = _attend_case(lengths, 4, 2, 128, 16, dtype, seed=39)
    _attend(c)
    want = c["out"].clone()
    other = torch.ones_like(want, dtype=torch.bool)
    for i, h, sign in ((1, 1, 1), (3, 2, -1), (5, 0, 1)):
        c["q"][i, h, 7 * h] = sign * math.inf
        other[i, h] = False
    _attend(c)
    assert torch.equal(c["out"][other], want[other])


# ------------------------------------------------------------------ the norm's range and its codes

@pytest.mark.parametrize("hidden,groups", [(8, 1), (512, 4), (4096, 32), (11008, 1), (32768, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_norm_of_rows_whose_squares_leave_the_range(hidden, groups, dtype):
    x, _, w, out, nt = _norm_case(8, 8, hidden, groups, dtype, False, seed=41)
    factors = [2.0 ** 60, 2.0 ** 100, 2.0 ** 122, 2.0 ** -70, 2.0 ** -110, 1.0, 2.0 ** 63, 2.0 ** -62] if dtype == "bf16" \
        else [2.0 ** 12, 2.0 ** -20, 1.0, 2.0 ** -8, 2.0 ** 10, 2.0 ** -14, 2.0 ** 4, 2.0 ** 8]
    x.mul_(torch.tensor(factors, device="cuda", dtype=torch.float64).to(x.dtype)[:, None])
    for eps in (0.0, 1e-30):
        B.lora_add_rmsnorm(x, w, eps, nt, **out)
        _norm_check(x, None, w, out, 8, groups, dtype, eps=eps)


@pytest.mark.parametrize("hidden,groups", [(4096, 32), (8192, 64), (11008, 86)])
def test_norm_codes_are_the_nearest(hidden, groups):
    """Rows of +-1, so that mean(z^2) is 1 and n is the weight, and weights of t times the middle between two
    codes in a group whose scale is t: a quotient that is off by its last bit takes the wrong code."""
    rows = 4
    g = torch.Generator().manual_seed(42)
    t = (torch.randint(16, 32, (groups, 1), generator=g) * 2 + 1).float()  # 33, 35, ... 63
    w = t * (torch.randint(8, 16, (groups, 128), generator=g) * 2 + 1) / 16 * 2.0 ** torch.randint(-4, 5, (groups, 128), generator=g)
    w[:, 5] = 448 * t[:, 0]
    w = w.flatten().half()
    x = (torch.randint(0, 2, (rows, hidden), generator=g) * 2.0 - 1).half()
    out = dict(y=torch.zeros(rows, hidden, dtype=torch.float16, device="cuda"),
               y8=torch.zeros(rows, hidden, device="cuda").to(torch.float8_e4m3fn),
               y8_scale=torch.zeros(rows, groups, device="cuda"))
    B.lora_add_rmsnorm(x.cuda(), w.cuda(), 0.0, _i32([rows]), **out)
    n = (x.float() * w.float()).numpy()
    assert np.array_equal(_np(out["y"]), n)
    s = np.repeat(out["y8_scale"].cpu().numpy(), 128, 1)
    assert (np.abs(s / np.repeat(t.numpy(), 128, 0).T - 1) <= 2.0 ** -23).all()
    want = np.sign(n) * R.E4M3[R.to_e4m3(np.abs(n / s))]  # the quotient rounded once to fp32
    off = int((want != _np(out["y8"])).sum())
    assert off == 0, f"{off} of {n.size} codes are not the nearest"


@pytest.mark.parametrize("groups", [1, 4])
def test_norm_keeps_the_sign_of_a_zero_and_the_ends_of_a_scale(groups):
    x, _, w, out, nt = _norm_case(4, 4, 512, groups, "bf16", False, seed=45)
    w.abs_()
    x[0, ::3], x[0, 1::3] = -0.0, 0.0
    x[1] = -0.0
    x[2, 5] = math.inf  # a mean of infinity: the others are 0
    x[3, ::2] = 0.0
    B.lora_add_rmsnorm(x, w, 1e-5, nt, **out)
    code = out["y8"].view(torch.uint8)
    assert (code[0, ::3] == 0x80).all() and (code[0, 1::3] == 0).all() and (code[1] == 0x80).all()
    assert torch.equal(torch.signbit(out["y"][:2].float()), torch.signbit(x[:2].float()))
    n = out["y"][2].float()
    assert torch.isnan(n[5]) and (n[:5] == 0).all() and (n[6:] == 0).all()
    _norm_check(x[3:], None, w, {k: v[3:] for k, v in out.items()}, 1, groups, "bf16")
    # weights whose group's largest n, and its scale, are infinite: finite n / infinity is 0
    w = torch.full((512,), 2.0 ** 127, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(4, 512, dtype=torch.bfloat16, device="cuda")
    x[:, 7] = 200.0
    w[9:] = 1.0
    B.lora_add_rmsnorm(x, w, 1e-5, nt, **out)
    n, s, y8 = out["y"].float(), out["y8_scale"], out["y8"].float()
    assert torch.isinf(n[:, 7]).all() and torch.isinf(s[:, 0]).all()
    assert torch.isnan(y8[:, 7]).all() and (y8[:, 9:128] == 0).all() and (y8[:, :7] == 0).all()


# ------------------------------------------------------------------ the append's zeros

@pytest.mark.parametrize("d", [64, 128])
def test_append_keeps_the_sign_of_a_zero(d):
    c = _append_case(6, 6, 1, 2, d, 16, 0, False, "bf16", seed=43)
    c["slots"] = _i32(np.arange(6))
    for x in ("k", "v"):
        t = c[x]
        t[0, :, ::3] = -0.0
        t[1, :, ::3] = 0.0
        t[2] = -0.0          # a block of zeros has scale 0 and codes 0
        t[3, :, 1:16] = -0.0
        t[4, :, 5] = -1e-30  # rounds to -0
    _append(c)
    _append_check(c, 6, d, 16, "bf16")


# ------------------------------------------------------------------ refusals come before the launch

class _NotAStream:
    cuda_stream = "none"


@pytest.mark.parametrize("stream", ["0", 1.5, object(), _NotAStream()])
def test_a_wrong_stream_is_refused_and_nothing_is_launched(stream):
    x, r, w, out, nt = _norm_case(4, 4, 256, 2, "bf16")
    c = _append_case(4, 4, 2, 1, 64, 16, 64, False, "bf16")
    a = _attend_case([(1, 20)], 4, 2, 64, 16, "bf16")
    with pytest.raises(ValueError):
        B.lora_add_rmsnorm(x, w, 1e-5, nt, residual=r, stream=stream, **out)
    with pytest.raises(ValueError):
        _append(c, stream=stream)
    with pytest.raises(ValueError):
        _attend(a, stream=stream)
    torch.cuda.synchronize()
    assert all((t.float() == 7).all() for t in out.values())
    assert (c["cache"] == 0xA5).all() and (c["q_out"] == 7).all()
    assert (a["out"] == 7).all() and (a["lse"] == 7).all()


def test_a_truth_value_that_has_none_is_refused():
    c = _append_case(4, 4, 2, 1, 64, 16, 64, False, "bf16")
    c["interleaved"] = np.zeros(2)  # its truth is ambiguous
    with pytest.raises(ValueError):
        _append(c)
    torch.cuda.synchronize()
    assert (c["cache"] == 0xA5).all() and (c["q_out"] == 7).all()


# ------------------------------------------------------------------ bounded waits

@pytest.mark.parametrize("heads", [(32, 32), (64, 4)])
def test_a_call_that_gives_up_ends_soon(heads):
    """One wait of 1 ms (the test hook's) and one for what was in flight, however many parts a warp has left:
    some 26 here.  (Through the hook nothing is in flight, so that wait runs out as well.)"""
    qh, kvh = heads
    c = _pool_case([(1, 40)] * (64000 // kvh), qh, kvh, 64, 16, "bf16", seed=44, pool=48)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = _attend(c, status=status)
    want = c["out"].clone()
    c["out"].fill_(7)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    assert B.lora_testing_inject_timeout(True) is False
    try:
        begin.record()
        _attend(c, workspace=ws, status=status)
        end.record()
        assert B.lora_read_status(status) == B.LORA_STATUS_TIMEOUT
    finally:
        assert B.lora_testing_inject_timeout(False) is True
    assert begin.elapsed_time(end) < 10.0
    assert (c["out"] == 7).all()
    _attend(c, workspace=ws, status=status)
    assert B.lora_read_status(status) == 0
    assert torch.equal(c["out"], want)
