"""The operators around a layer's LoRA products on the GPU: the norm, the append to the 4-bit
paged cache and the attention over it, against their formulas in 64 bits on the CPU.

Tolerances come from the roundings that the contract names: a 16-bit output is rounded once (half
a unit in the last place: at most 2^-8 relative in bf16, 2^-11 in fp16, plus half the smallest subnormal in fp16), an e4m3
code once (2^-4 relative, 2^-10 at the bottom), a probability once to fp16 (2^-11, and 2^-25 at the
bottom), everything else happens in fp32 (sums of at most 2^15 terms: 2^-24 * sqrt(terms), taken as
2^-16)."""
import math

import numpy as np
import pytest

from gathered_rank_gemm_gb300 import binding as B
from tests import layer_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
BOTTOM = {"bf16": 1e-38, "f16": 2.0 ** -25}
FP32 = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gathered_rank_gemm_gb300 import build
    build.build()
    return B.load()


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _close(got, want, rel, absolute, what):
    bad = ~(np.abs(got - want) <= absolute + rel * np.abs(want))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first {got[bad][:3]} want {want[bad][:3]}"


# ------------------------------------------------------------------ norm

def _norm_case(rows, n, hidden, groups, dtype, residual=True, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    x = torch.randn(rows, hidden + pad, generator=g).to(dt).cuda()[:, :hidden]
    r = (2 * torch.randn(rows, hidden + pad, generator=g)).to(dt).cuda()[:, :hidden] if residual else None
    w = (1 + 0.1 * torch.randn(hidden, generator=g)).to(dt).cuda()
    out = dict(residual_out=torch.full((rows, hidden + pad), 7, dtype=dt, device="cuda")[:, :hidden],
               y=torch.full((rows, hidden + pad), 7, dtype=dt, device="cuda")[:, :hidden],
               y8=torch.full((rows, hidden), 7.0, device="cuda").to(torch.float8_e4m3fn),
               y8_scale=torch.full((rows, groups), 7.0, device="cuda"))
    return x, r, w, out, _i32([n])


def _norm_check(x, r, w, out, n, groups, dtype, eps=1e-5):
    z, want, scale = R.norm(_np(x[:n]), None if r is None else _np(r[:n]), _np(w), eps, groups)
    _close(_np(out["residual_out"][:n]), z, HALF_UNIT[dtype] + FP32, BOTTOM[dtype], "residual_out")
    _close(_np(out["y"][:n]), want, HALF_UNIT[dtype] + FP32, BOTTOM[dtype], "y")
    _close(_np(out["y8_scale"][:n]), scale, FP32, 0, "y8_scale")
    wide = np.repeat(scale, want.shape[1] // groups, 1)
    _close(_np(out["y8"][:n]), want / wide, 2.0 ** -4 + FP32, 2.0 ** -10, "y8")
    for name, t in out.items():
        assert (t[n:].float() == 7).all(), f"{name}: a row past n was written"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,n,hidden,groups", [
    (1, 1, 8, 1), (1, 1, 128, 1), (3, 2, 136, 1), (5, 5, 4096, 32), (9, 9, 2048, 1), (4, 3, 5000, 1),
    (3, 3, 8320, 65), (2, 2, 11008, 86), (2, 2, 16392, 1), (3, 2, 32768, 256), (2, 2, 32768, 1), (700, 699, 264, 1),
    (300, 300, 1024, 8), (64, 0, 256, 2)])
def test_norm(rows, n, hidden, groups, dtype):
    x, r, w, out, nt = _norm_case(rows, n, hidden, groups, dtype, seed=hidden)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    B.lora_add_rmsnorm(x, w, 1e-5, nt, residual=r, status=status, **out)
    _norm_check(x, r, w, out, n, groups, dtype)
    assert status[0].item() == 0


@pytest.mark.parametrize("hidden,groups", [(520, 1), (4096, 32), (4096, 1)])
def test_norm_of_strided_rows_and_without_a_residual(hidden, groups):
    for residual in (True, False):
        x, r, w, out, nt = _norm_case(37, 35, hidden, groups, "bf16", residual, pad=24, seed=3)
        B.lora_add_rmsnorm(x, w, 1e-5, nt, residual=r, **out)
        _norm_check(x, r, w, out, 35, groups, "bf16")


@pytest.mark.parametrize("hidden,groups", [(4096, 32), (1000, 1)])
def test_norm_in_place_and_with_some_outputs_only(hidden, groups):
    x, r, w, out, nt = _norm_case(20, 20, hidden, groups, "bf16", seed=5)
    want = {k: v.clone() for k, v in out.items()}
    B.lora_add_rmsnorm(x, w, 1e-5, nt, residual=r, **want)
    r2, x2 = r.clone(), x.clone()
    B.lora_add_rmsnorm(x2, w, 1e-5, nt, residual=r2, residual_out=r2, y=x2)
    assert torch.equal(r2, want["residual_out"]) and torch.equal(x2, want["y"])
    B.lora_add_rmsnorm(x, w, 1e-5, nt, residual=r, y8=out["y8"], y8_scale=out["y8_scale"])
    assert torch.equal(out["y8"].view(torch.uint8), want["y8"].view(torch.uint8))
    assert torch.equal(out["y8_scale"], want["y8_scale"])
    x3 = x.clone()
    B.lora_add_rmsnorm(x3, w, 1e-5, nt, residual=r, residual_out=x3)
    assert torch.equal(x3, want["residual_out"])


def test_norm_of_zeros_huge_values_and_nan():
    x, _, w, out, nt = _norm_case(5, 5, 512, 4, "bf16", False)
    x[0] = 0
    x[1, 7] = math.nan
    x[2] = 1e18
    x[3] = 1e-18
    B.lora_add_rmsnorm(x, w, 0.0, nt, **out)
    y, s = out["y"].float(), out["y8_scale"]
    assert torch.isnan(y[0]).all()  # 0 / sqrt(0): eps is 0 here
    assert torch.isnan(y[1]).all() and torch.isnan(s[1]).all() and torch.isnan(out["y8"][1].float()).all()
    assert torch.isfinite(y[2:]).all() and torch.isfinite(s[2:]).all()
    B.lora_add_rmsnorm(x, w, 1e-5, nt, **out)
    assert (out["y"][0] == 0).all() and (out["y8"][0].float() == 0).all()
    assert (out["y8_scale"][0] == 2.0 ** -100).all()


def test_norm_clamps_n_and_says_so():
    x, r, w, out, _ = _norm_case(6, 6, 256, 1, "bf16")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    B.lora_add_rmsnorm(x, w, 1e-5, _i32([9]), residual=r, status=status, **out)
    _norm_check(x, r, w, out, 6, 1, "bf16")
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_NUM_TOKENS
    B.lora_add_rmsnorm(x, w, 1e-5, _i32([-1]), residual=r, status=status, **out)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_NUM_TOKENS


# ------------------------------------------------------------------ append

def _append_case(rows, n, qh, kvh, d, page, rope_dim, interleaved, dtype, seed=0):
    rng = np.random.default_rng(seed)
    dt = DTYPES[dtype]
    qkv = torch.tensor(rng.standard_normal((rows, (qh + 2 * kvh) * d)), dtype=torch.float32).to(dt).cuda()
    q, k, v = (a.unflatten(1, (-1, d)) for a in qkv.split([qh * d, kvh * d, kvh * d], 1))
    positions = rng.integers(0, 500, rows)
    pages = -(-rows // page) + 2
    slots = rng.permutation(pages * page)[:rows]
    slots[rng.random(rows) < 0.1] = -1
    rope = None
    if rope_dim:
        angle = np.arange(500)[:, None] / 10000.0 ** (np.arange(0, rope_dim, 2) / rope_dim)
        rope = torch.tensor(np.concatenate([np.cos(angle), np.sin(angle)], 1), dtype=torch.float32, device="cuda")
    cache = torch.full((pages, kvh, page // 16, 18 * d), 0xA5, dtype=torch.uint8, device="cuda")
    return dict(q=q, k=k, v=v, positions=_i32(positions), slots=_i32(slots), rope=rope, cache=cache,
                q_out=torch.full((rows, qh, d), 7, dtype=dt, device="cuda"),
                k_held=torch.full((rows, kvh, d), 7, dtype=dt, device="cuda"),
                v_held=torch.full((rows, kvh, d), 7, dtype=dt, device="cuda"), n=_i32([n]), interleaved=interleaved)


def _append(c, **more):
    B.lora_kv4_append(c["cache"], c["k"], c["v"], c["slots"], c["n"], q=c["q"], q_out=c["q_out"],
                      positions=c["positions"], rope=c["rope"], interleaved=c["interleaved"], k_scale=1 / 32,
                      v_scale=0.01, **{"k_held": c["k_held"], "v_held": c["v_held"], **more})


def _append_check(c, n, d, page, dtype, live=None):
    slots = c["slots"].cpu().numpy()[:n]
    pos = c["positions"].cpu().numpy()[:n]
    live = np.ones(n, bool) if live is None else live
    q, k, v = (_np(c[x][:n]) for x in "qkv")
    k32 = k.astype(np.float32)
    if c["rope"] is not None:
        cos, sin = np.split(c["rope"].cpu().numpy()[np.clip(pos, 0, 499)], 2, -1)
        q = R.rotate(q, cos, sin, c["interleaved"])
        k32 = R.rotate(k32, cos, sin, c["interleaved"], np.float32)
    _close(_np(c["q_out"][:n])[live], q[live], HALF_UNIT[dtype] + FP32, 2.0 ** -20, "q_out")
    cache = np.full(c["cache"].shape, 0xA5, np.uint8)
    kept = live & (slots >= 0)
    for x, factor, part, held in ((k32, 1 / 32, 0, "k_held"), (v.astype(np.float32), 0.01, 1, "v_held")):
        code, s8 = R.quantise32(x, factor)
        for t in np.nonzero(kept)[0]:
            blk = cache[slots[t] // page, :, slots[t] % page // 16]
            r = slots[t] % 16
            blk[:, 8 * d * part + r * d // 2:8 * d * part + (r + 1) * d // 2] = R.pack(code[t])
            s0 = (16 + part) * d
            blk[:, s0 + r * d // 16:s0 + (r + 1) * d // 16] = s8[t]
        want = R.values(code, s8) * np.float64(np.float32(factor))
        _close(_np(c[held][:n])[kept], want[kept], HALF_UNIT[dtype] + FP32, BOTTOM[dtype], held)
        assert (c[held][:n][torch.tensor(~kept)] == 7).all()
    got = c["cache"].cpu().numpy()
    assert np.array_equal(got, cache), f"{(got != cache).sum()} bytes of the cache differ"
    for name in ("q_out", "k_held", "v_held"):
        assert (c[name][n:] == 7).all(), f"{name}: a row past n was written"


@pytest.mark.parametrize("rows,n,qh,kvh,d,page,rope_dim,interleaved,dtype", [
    (1, 1, 32, 32, 128, 16, 128, False, "bf16"), (1, 1, 1, 1, 64, 16, 64, True, "f16"),
    (40, 37, 8, 2, 128, 32, 128, True, "bf16"), (40, 40, 6, 3, 64, 64, 32, False, "bf16"),
    (65, 65, 4, 4, 128, 48, 96, False, "f16"), (300, 299, 12, 2, 64, 16, 64, False, "bf16"),
    (33, 33, 5, 1, 128, 128, 64, True, "bf16"), (17, 0, 2, 1, 64, 16, 64, False, "bf16"),
    (50, 50, 4, 2, 128, 1024, 0, False, "f16")])
def test_append(rows, n, qh, kvh, d, page, rope_dim, interleaved, dtype):
    c = _append_case(rows, n, qh, kvh, d, page, rope_dim, interleaved, dtype, seed=rows + d)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    _append(c, status=status)
    _append_check(c, n, d, page, dtype)
    assert status[0].item() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotates_q_in_place_and_needs_no_q(interleaved):
    c = _append_case(30, 30, 4, 2, 128, 16, 128, interleaved, "bf16")
    _append(c)
    whole = c["cache"].clone()
    want = c["q_out"].clone()
    c["cache"].fill_(0xA5)
    B.lora_kv4_append(c["cache"], c["k"], c["v"], c["slots"], c["n"], q=c["q"], q_out=c["q"],
                      positions=c["positions"], rope=c["rope"], interleaved=interleaved, k_scale=1 / 32,
                      v_scale=0.01)
    assert torch.equal(c["q"], want) and torch.equal(c["cache"], whole)
    c["cache"].fill_(0xA5)
    B.lora_kv4_append(c["cache"], c["k"], c["v"], c["slots"], c["n"], positions=c["positions"], rope=c["rope"],
                      interleaved=interleaved, k_scale=1 / 32, v_scale=0.01)
    assert torch.equal(c["cache"], whole)


def test_append_of_zeros_ties_nan_infinity_and_extremes():
    c = _append_case(8, 8, 1, 1, 64, 16, 0, False, "bf16", seed=9)
    c["slots"] = _i32(np.arange(8))
    ties = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0])
    for x in ("k", "v"):
        t = c[x][:, 0]
        t[0] = 0
        t[1, :16] = ties.to(t)
        t[1, 16:32] = ties.to(t) * 2.0 ** -5
        t[2, 3] = math.nan
        t[3, 20] = math.inf
        t[3, 40] = -math.inf
        t[4] = 3e38
        t[5] = 1e-38
        t[6] *= 1e-4
        t[7] *= 100
    _append(c, k_held=None, v_held=None)
    c["k_held"].fill_(7)
    got = c["cache"].cpu().numpy()
    for x, factor, part in (("k", 1 / 32, 0), ("v", 0.01, 1)):
        code, s8 = R.quantise32(_np(c[x][:, 0]).astype(np.float32), factor)
        assert np.array_equal(R.sections(got, 64)[part][0, 0, 0, :8], R.pack(code))
        assert np.array_equal(R.sections(got, 64)[2 + part][0, 0, 0, :8], s8)


def test_append_refuses_what_only_the_data_shows():
    c = _append_case(12, 12, 2, 1, 64, 16, 64, False, "bf16", seed=2)
    pos, slots = c["positions"].clone(), c["slots"].clone()
    c["positions"][3], c["positions"][5] = 500, -1
    c["slots"][7] = c["cache"].shape[0] * 16
    c["slots"][8] = -2
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    _append(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_SLOT | B.LORA_STATUS_BAD_POSITION
    live = np.ones(12, bool)
    live[[3, 5]] = False
    assert (c["q_out"][[3, 5]] == 7).all()
    c["slots"][7], c["slots"][8] = -1, -1
    _append_check(c, 12, 64, 16, "bf16", live)


# ------------------------------------------------------------------ attention

K_SCALE, V_SCALE = 1 / 32, 1 / 64


def _attend_case(lengths, qh, kvh, d, page, dtype, seed=0, spread=1.0, pad=0, grow=None):
    rng = np.random.default_rng(seed)
    dt = DTYPES[dtype]
    per = [-(-n // page) for _, n in lengths]
    pages = sum(per) + 3
    order = rng.permutation(pages)
    wide = max(1, max(per))
    table = np.full((len(per), wide), -7, np.int64)  # entries behind a sequence's pages are not read
    at = 0
    for b, m in enumerate(per):
        table[b, :m] = order[at:at + m]
        at += m
    k = [rng.standard_normal((n, kvh, d)) * spread for _, n in lengths]
    v = [rng.standard_normal((n, kvh, d)) for _, n in lengths]
    if grow:  # keys that grow along a sequence, by powers of two from 1 to 2^grow
        k = [x * 2.0 ** np.linspace(0, grow, len(x))[:, None, None] for x in k]
    cache = R.build_cache(k, v, pages, table, page, K_SCALE, V_SCALE)
    rows = sum(m for m, _ in lengths) + 2
    q = torch.tensor(rng.standard_normal((rows, qh * d + pad)), dtype=torch.float32).to(dt).cuda()
    q = q[:, :qh * d].unflatten(1, (qh, d))
    start = np.concatenate([[0], np.cumsum([m for m, _ in lengths])])
    return dict(lengths=lengths, q=q, cache=torch.tensor(cache).cuda(), cache_np=cache, table_np=table,
                table=_i32(table), start=_i32(start), start_np=start, kv=_i32([n for _, n in lengths]), page=page,
                max_q=max(1, max(m for m, _ in lengths)), out=torch.full((rows, qh, d), 7, dtype=dt, device="cuda"),
                lse=torch.full((rows, qh), 7.0, device="cuda"), dtype=dtype, rows=rows, qh=qh, kvh=kvh, d=d)


def _attend(c, window=0, scale=None, **more):
    size = B.lora_kv4_attention_workspace_size(len(c["lengths"]), c["rows"], c["max_q"], c["qh"], c["kvh"], c["d"])
    ws = more.pop("workspace", None)
    if ws is None:
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    B.lora_kv4_attention(c["cache"], c["q"], c["out"], c["start"], c["kv"], c["table"], c["max_q"],
                         scale or 1 / math.sqrt(c["d"]), ws, window=window, k_scale=K_SCALE, v_scale=V_SCALE,
                         lse=c["lse"], **more)
    return ws


def _attend_check(c, window=0, scale=None, some=None):
    """Every row against the formula (or, for long sequences, the rows `some` picks of each)."""
    scale = scale or 1 / math.sqrt(c["d"])
    q, out, lse = _np(c["q"]), _np(c["out"]), c["lse"].cpu().numpy().astype(np.float64)
    for b, (m, n) in enumerate(c["lengths"]):
        k, v = R.read_cache(c["cache_np"], c["table_np"][b][:-(-n // c["page"])], n, c["page"], c["d"])
        rows = slice(c["start_np"][b], c["start_np"][b + 1])
        pick = np.arange(m) if some is None or m <= some else np.unique(np.linspace(0, m - 1, some).astype(int))
        for i in pick if some is not None else [None]:
            if i is None:
                qq, cut, r = q[rows], n, rows
            else:  # row i alone: it is the last of a sequence of its own keys
                cut = max(0, n - m + i + 1)
                r = slice(rows.start + i, rows.start + i + 1)
                qq = q[r]
            want, wlse, size, span = R.attention(qq, k[:cut] * K_SCALE, v[:cut] * V_SCALE, scale, window)
            tol = HALF_UNIT[c["dtype"]] * np.abs(want) + BOTTOM[c["dtype"]] + \
                (2.0 ** -11 + FP32 + FP32 * span[..., None]) * size + 2.0 ** -25 * size.max(initial=0) * max(1, cut) ** 0.5
            bad = ~(np.abs(out[r] - want) <= tol)
            assert not bad.any(), (b, m, n, i, bad.sum(), out[r][bad][:3], want[bad][:3])
            none = np.isneginf(wlse)
            assert np.array_equal(np.isneginf(lse[r]), none)
            err = np.abs(lse[r][~none] - wlse[~none])
            assert (err <= FP32 * (1 + span[~none] + np.abs(wlse[~none]))).all(), (b, m, n, err.max())
            assert (out[r][none] == 0).all()
    last = c["start_np"][-1]
    assert (c["out"][last:] == 7).all() and (c["lse"][last:] == 7).all(), "a row past the last sequence was written"


SHAPES = [
    # lengths (rows, keys), q heads, kv heads, d, page
    ([(1, 1)], 1, 1, 128, 16), ([(1, 1)], 1, 1, 64, 16), ([(1, 15), (1, 16), (1, 17)], 4, 2, 128, 16),
    ([(1, 33), (1, 0), (1, 129), (1, 64)], 8, 8, 64, 32), ([(1, 700)], 32, 8, 128, 16),
    ([(1, n) for n in (5, 257, 1000, 31, 511, 64)], 8, 1, 128, 64), ([(1, 300), (1, 45)], 20, 4, 128, 48),
    ([(1, 200), (1, 77)], 12, 1, 64, 16), ([(1, 130), (1, 95)], 24, 1, 128, 16), ([(1, 2000)], 64, 2, 64, 1024),
    ([(4, 100), (1, 3), (0, 50), (3, 3), (5, 2), (2, 0)], 8, 2, 128, 16),
    ([(7, 300), (2, 310)], 6, 3, 64, 16), ([(3, 1000), (8, 900)], 5, 1, 128, 32),
    ([(16, 16)], 4, 4, 64, 16), ([(33, 40), (1, 100)], 8, 2, 128, 16), ([(70, 70), (65, 200)], 4, 2, 64, 64),
    ([(130, 500)], 4, 1, 128, 32), ([(300, 290), (129, 129), (1, 700), (5, 0)], 6, 2, 128, 16),
    ([(257, 600)], 2, 2, 64, 16), ([(200, 333), (0, 0), (64, 64)], 8, 8, 128, 16),
    ([(520, 900)], 3, 1, 128, 64), ([(140, 150), (90, 700)], 10, 2, 64, 32),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention(shape, dtype):
    lengths, qh, kvh, d, page = SHAPES[shape]
    c = _attend_case(lengths, qh, kvh, d, page, dtype, seed=shape)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    _attend(c, status=status)
    _attend_check(c, some=40)
    assert status[0].item() == 0


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 1000])
@pytest.mark.parametrize("shape", [3, 5, 10, 11, 17, 18, 21])
def test_attention_in_a_window(shape, window):
    lengths, qh, kvh, d, page = SHAPES[shape]
    c = _attend_case(lengths, qh, kvh, d, page, "bf16", seed=100 + shape)
    _attend(c, window)
    _attend_check(c, window, some=25)


@pytest.mark.parametrize("lengths", [[(1, 40000), (1, 7)], [(1, 9000), (2, 20000), (1, 0)], [(130, 9000)]])
def test_attention_over_long_keys(lengths):
    c = _attend_case(lengths, 4, 1, 128, 64, "bf16", seed=7)
    ws = _attend(c)
    _attend_check(c, some=6)
    first = c["out"].clone(), c["lse"].clone()
    for _ in range(3):  # the same workspace, the same bits
        _attend(c, workspace=ws)
        assert torch.equal(c["out"], first[0]) and torch.equal(c["lse"], first[1])


@pytest.mark.parametrize("lengths", [[(1, 500), (1, 90)], [(3, 333)], [(150, 400)]])
@pytest.mark.parametrize("spread", [30.0, 1e-3])
def test_attention_of_peaked_and_flat_rows(lengths, spread):
    c = _attend_case(lengths, 8, 2, 128, 16, "bf16", seed=11, spread=spread)
    c["q"].mul_(3)
    _attend(c)
    _attend_check(c, some=20)


@pytest.mark.parametrize("grow", [12, -12])
@pytest.mark.parametrize("lengths", [[(1, 3000)], [(3, 700), (1, 90)], [(150, 1500)], [(300, 700), (40, 300)]])
def test_attention_of_scores_that_grow_or_fall_along_the_keys(lengths, grow):
    """The running reference has to move again and again, or never."""
    c = _attend_case(lengths, 4, 2, 128, 16, "bf16", seed=17, spread=2.0 ** (-grow / 2), grow=grow)
    _attend(c)
    _attend_check(c, some=20)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("chunks", [False, True])
def test_attention_of_many_sequences(chunks, d):
    """More sequences than a CTA has threads; with chunks, some of them go to each kernel."""
    rng = np.random.default_rng(18)
    lengths = [(int(rng.integers(0, 4)), int(rng.integers(0, 60))) for _ in range(1100)]
    if chunks:
        for b in range(5, 1100, 90):
            lengths[b] = (int(rng.integers(30, 140)), int(rng.integers(1, 200)))
    c = _attend_case(lengths, 2, 1, d, 16, "bf16", seed=18)
    _attend(c)
    _attend_check(c)


@pytest.mark.parametrize("seqs", [31, 32, 33, 192, 193, 256, 257, 385])
@pytest.mark.parametrize("rows", [1, 2, 9])
def test_attention_where_the_walk_over_sequences_changes(seqs, rows):
    """Sequences of a warp's lanes, of a CTA's threads, of several a thread; empty ones among them,
    the first and the last too; a few long ones, so that items are whole, and cut."""
    rng = np.random.default_rng(seqs)
    lengths = [(int(rng.integers(0, rows + 1)), int(rng.integers(0, 40))) for _ in range(seqs)]
    lengths[0] = lengths[-1] = (0, 5)
    c = _attend_case(lengths, 4, 2, 128, 16, "bf16", seed=seqs)
    _attend(c)
    _attend_check(c)
    lengths[seqs // 2] = (1, 3000)
    c = _attend_case(lengths, 4, 2, 64, 16, "f16", seed=seqs)
    _attend(c)
    _attend_check(c)


@pytest.mark.parametrize("bound", [1, 4, 100])
def test_rows_beyond_the_bound_get_no_output(bound):
    c = _attend_case([(3, 60), (130, 300), (1, 9)], 4, 2, 64, 16, "bf16", seed=19)
    c["max_q"] = bound
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    _attend(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_LENGTH
    got, lse = c["out"].clone(), c["lse"].clone()
    c["max_q"] = 130
    _attend(c)
    _attend_check(c, some=20)
    kept = torch.zeros(c["rows"], dtype=torch.bool, device="cuda")
    for b, (m, _) in enumerate(c["lengths"]):
        kept[c["start_np"][b]:c["start_np"][b] + min(m, bound)] = True
    assert (got[~kept] == 7).all() and (lse[~kept] == 7).all()
    # the same rows by the same formula, whichever kernel had them: two roundings of the output and
    # two of the probabilities (2^-11 of values of at most 6) apart, and as much for the sums
    diff = (got[kept].float() - c["out"][kept].float()).abs()
    assert (diff <= 2.0 ** -7 * c["out"][kept].float().abs() + 2.0 ** -9 * 6).all()


@pytest.mark.parametrize("rows", [1, 140])
def test_sequences_that_share_pages(rows):
    """A common beginning in common pages, as prefix reuse leaves it."""
    c = _attend_case([(rows, 300), (rows, 300), (rows, 280)], 4, 2, 128, 32, "bf16", seed=20)
    for t in (c["table"], c["table_np"]):
        t[1:, :6] = t[0, :6]
    _attend(c)
    _attend_check(c, some=15)


def test_two_streams_with_a_workspace_each():
    one = _attend_case([(1, 2500), (1, 900)], 8, 2, 128, 16, "bf16", seed=24)
    two = _attend_case([(140, 400), (2, 800)], 8, 2, 128, 16, "bf16", seed=25)
    cases = (one, two)
    spaces = [_attend(c) for c in cases]
    want = [c["out"].clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, ws, s in zip(cases, spaces, streams):
            _attend(c, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c["out"], w)
        _attend_check(c, some=10)


@pytest.mark.parametrize("factor", [2.0 ** 60, 2.0 ** -60])
@pytest.mark.parametrize("lengths", [[(1, 200), (2, 30)], [(140, 300)]])
def test_attention_of_queries_far_from_one(lengths, factor):
    c = _attend_case(lengths, 4, 2, 64, 16, "bf16", seed=12)
    c["q"].mul_(factor)
    scale = 1 / math.sqrt(64) / factor
    _attend(c, scale=scale)
    _attend_check(c, scale=scale, some=20)


def test_attention_of_strided_rows_on_another_stream():
    for lengths in ([(1, 100), (2, 30), (1, 513)], [(200, 300), (1, 40)]):
        c = _attend_case(lengths, 8, 4, 128, 16, "bf16", seed=13, pad=64)
        wide = torch.full((c["rows"], 8 * 128 + 8), 7, dtype=torch.bfloat16, device="cuda")
        c["out"] = wide[:, :1024].unflatten(1, (8, 128))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        _attend(c, stream=side)
        side.synchronize()
        _attend_check(c, some=20)
        assert (wide[:, 1024:] == 7).all()


@pytest.mark.parametrize("lengths", [[(1, 300), (1, 90)], [(140, 200), (1, 60)]])
def test_attention_of_data_that_does_not_fit(lengths):
    c = _attend_case(lengths, 4, 2, 128, 16, "bf16", seed=14)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    # a page outside the cache: its keys are masked
    c["table"][0, 2] = c["cache"].shape[0]
    _attend(c, status=status)
    assert B.lora_read_status(status) == B.LORA_STATUS_BAD_SLOT
    gone = np.ones(lengths[0][1], bool)
    gone[32:48] = False
    k, v = R.read_cache(c["cache_np"], c["table_np"][0], lengths[0][1], 16, 128)
    last = lengths[0][0] - 1
    want, wlse, size, span = R.attention(_np(c["q"][last:last + 1]), k[gone] * K_SCALE, v[gone] * V_SCALE, 1 / math.sqrt(128), 0)
    assert (np.abs(_np(c["out"][last:last + 1]) - want) <= HALF_UNIT['bf16'] * np.abs(want) + 2.0 ** -10 * size).all()
    # more keys than the table holds: clamped
    c = _attend_case(lengths, 4, 2, 128, 16, "bf16", seed=15)
    c["kv"][0] = 1 << 30
    c["kv"][1] = -5
    _attend(c, status=status)
    assert B.lora_read_status(status) & B.LORA_STATUS_BAD_LENGTH
    assert (c["out"][c["start_np"][1]:c["start_np"][2]] == 0).all()


def test_attention_in_a_graph_follows_its_data():
    """One captured call serves other lengths, pages and inputs (the host gives bounds only)."""
    a = _attend_case([(1, 900), (1, 40), (1, 1)], 8, 2, 128, 16, "bf16", seed=16)
    ws = _attend(a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            _attend(a, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    _attend_check(a)
    a["kv"].copy_(_i32([300, 0, 1]))
    a["lengths"] = [(1, 300), (1, 0), (1, 1)]
    a["q"].mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    _attend_check(a)


def test_offsets_past_32_bits():
    """A cache of more than 4 GB: append to its last pages, then attend to them."""
    kvh, d, page = 8, 128, 64
    pages = (5 << 30) // (kvh * page // 16 * 18 * d)
    cache = torch.zeros((pages, kvh, page // 16, 18 * d), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(5)
    n = 100
    own = np.array([pages - 1, pages - 3])
    j = np.arange(n)
    slots = own[j // page] * page + j % page
    assert slots[0] * kvh * 18 * d // 16 > 1 << 32
    k, v = (torch.tensor(rng.standard_normal((n, kvh, d)), dtype=torch.float32).bfloat16().cuda() for _ in range(2))
    B.lora_kv4_append(cache, k, v, _i32(slots), _i32([n]), k_scale=K_SCALE, v_scale=V_SCALE)
    for m in (1, n):
        q = torch.tensor(rng.standard_normal((m, 16, d)), dtype=torch.float32).bfloat16().cuda()
        out = torch.empty_like(q)
        ws = torch.zeros(B.lora_kv4_attention_workspace_size(1, m, m, 16, kvh, d), dtype=torch.uint8, device="cuda")
        B.lora_kv4_attention(cache, q, out, _i32([0, m]), _i32([n]), _i32([own]), m, 0.1, ws, k_scale=K_SCALE,
                             v_scale=V_SCALE)
        kk, vv = R.read_cache(cache[torch.tensor(own)].cpu().numpy(), [0, 1], n, page, d)
        want, _, size, _ = R.attention(_np(q), kk * K_SCALE, vv * V_SCALE, 0.1, 0)
        assert (np.abs(_np(out) - want) <= HALF_UNIT["bf16"] * np.abs(want) + 2.0 ** -10 * size).all()


# ------------------------------------------------------------------ refusals of the wrappers

def test_wrappers_refuse_wrong_operands():
    x, r, w, out, nt = _norm_case(4, 4, 256, 2, "bf16")
    for bad in (dict(residual=r.half()), dict(residual=r[:, :128]), dict(y=out["y"].cpu()),
                dict(y8=out["y8"], y8_scale=None), dict(y8=out["y8"], y8_scale=out["y8_scale"].half())):
        with pytest.raises(ValueError):
            B.lora_add_rmsnorm(x, w, 1e-5, nt, **{"y": out["y"], **bad})
    with pytest.raises(ValueError):
        B.lora_add_rmsnorm(x.float(), w, 1e-5, nt, y=out["y"])
    with pytest.raises(ValueError):
        B.lora_add_rmsnorm(x.t(), w, 1e-5, nt, y=out["y"])
    with pytest.raises(B.LoraError):
        B.lora_add_rmsnorm(x, w, 1e-5, nt)  # no output at all
    c = _append_case(4, 4, 2, 1, 64, 16, 64, False, "bf16")
    with pytest.raises(ValueError):
        B.lora_kv4_append(c["cache"], c["k"], c["v"].half(), c["slots"], c["n"])
    with pytest.raises(ValueError):
        B.lora_kv4_append(c["cache"], c["k"], c["v"], c["slots"].long(), c["n"])
    with pytest.raises(ValueError):
        B.lora_kv4_append(c["cache"], c["k"], c["v"], c["slots"], c["n"], rope=c["rope"])
    with pytest.raises(B.LoraError):
        B.lora_kv4_append(c["cache"], c["k"], c["v"], c["slots"], c["n"], k_scale=0.0)
    a = _attend_case([(1, 20)], 4, 2, 64, 16, "bf16")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    args = (a["cache"], a["q"], a["out"], a["start"], a["kv"], a["table"])
    with pytest.raises(ValueError):
        B.lora_kv4_attention(*args[:2], a["out"].half(), *args[3:], 1, 0.1, ws)
    with pytest.raises(ValueError):
        B.lora_kv4_attention(*args[:3], a["start"][:1], *args[4:], 1, 0.1, ws)
    with pytest.raises(B.LoraError):
        B.lora_kv4_attention(*args, 1, 0.0, ws)
    with pytest.raises(B.LoraError):
        B.lora_kv4_attention(*args, 1, 0.1, ws, window=-1)
    with pytest.raises(B.LoraError):
        B.lora_kv4_attention(*args, 1, 0.1, ws[:16])
    with pytest.raises(B.LoraError):
        B.lora_kv4_attention(*args, 99, 0.1, ws)


# ------------------------------------------------------------------ NaN where a row must not look

@pytest.mark.parametrize("lengths,window", [([(1, 80), (6, 100)], 0), ([(6, 100)], 20), ([(140, 300)], 0),
                                            ([(140, 300), (4, 90)], 50), ([(300, 310)], 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_in_the_cache_stays_with_the_rows_that_see_it(lengths, window, d):
    """A NaN scale of K takes the rows that see its key; one of V their 16 dimensions."""
    c = _attend_case(lengths, 4, 2, d, 16, "bf16", seed=21)
    b = len(lengths) - 1
    m, n = lengths[b]
    key = n - 3 if m < 10 else n - m // 2
    page, r = c["table_np"][b][key // 16], key % 16
    clean = c["cache"].clone()
    _attend(c, window)
    want = c["out"].clone()
    rows = torch.arange(m, device="cuda") + int(c["start_np"][b])
    pos = torch.arange(n - m, n, device="cuda")
    sees = (pos >= key) & ((pos - window < key) if window else torch.ones_like(pos, dtype=torch.bool))
    # V: the second 16 dimensions of key head 1
    c["cache"].copy_(clean)
    c["cache"][page, 1, 0, 17 * d + r * d // 16 + 1] = 0x7F
    _attend(c, window)
    got = c["out"]
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[rows[sees], 2:, 16:32] = True
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], want[~bad])
    # K: any block of it
    c["cache"].copy_(clean)
    c["cache"][page, 1, 0, 16 * d + r * d // 16] = 0xFF
    _attend(c, window)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[rows[sees], 2:] = True
    assert torch.isnan(c["out"][bad]).all()
    assert torch.equal(c["out"][~bad], want[~bad])


@pytest.mark.parametrize("lengths", [[(3, 50)], [(140, 200)]])
def test_queries_that_are_not_finite_keep_to_their_rows(lengths):
    c = _attend_case(lengths, 4, 2, 64, 16, "bf16", seed=22)
    _attend(c)
    want = c["out"].clone()
    c["q"][1, 1, 5] = math.nan
    c["q"][2, 3, 0] = math.inf
    _attend(c)
    other = torch.ones_like(want, dtype=torch.bool)
    other[1, 1] = False
    other[2, 3] = False
    assert torch.isnan(c["out"][1, 1]).all()
    assert torch.equal(c["out"][other], want[other])


# ------------------------------------------------------------------ bounded waits

@pytest.mark.parametrize("lengths", [[(1, 3000), (1, 90), (1, 0)], [(2, 40)], [(140, 900), (1, 60)]])
def test_attention_gives_up_a_wait_and_recovers(lengths):
    """Through the test hook: the call ends, says so, writes nothing, and the next call on the same
    workspace is right."""
    c = _attend_case(lengths, 8, 2, 128, 16, "bf16", seed=23)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = _attend(c, status=status)
    torch.cuda.synchronize()
    c["out"].fill_(7)
    c["lse"].fill_(7)
    assert B.lora_testing_inject_timeout(True) is False
    try:
        _attend(c, workspace=ws, status=status)
        assert B.lora_read_status(status) == B.LORA_STATUS_TIMEOUT
    finally:
        assert B.lora_testing_inject_timeout(False) is True
    assert (c["out"] == 7).all() and (c["lse"] == 7).all()
    _attend(c, workspace=ws, status=status)
    assert B.lora_read_status(status) == 0
    _attend_check(c, some=10)
