"""CPU-only checks of the operators around a layer's LoRA products: their argument checks reject
bad calls before anything reaches a GPU, and the 64-bit formulas that the GPU tests use agree with
worked examples."""
import ctypes

import numpy as np
import pytest

from gathered_rank_gemm_gb300 import binding as B
from gathered_rank_gemm_gb300 import build
from tests import layer_ref as R

P, ODD = 0x10000, 0x10004  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def _caller(fn, names, base):
    def call(**kw):
        d = dict(base, **kw)
        assert set(d) == set(names)
        return fn(*[d[n] for n in names])
    return call


def test_norm_arguments(lib):
    names = ("x xs r rs w eps h ro ros y ys y8 y8s sc group n t status stream").split()
    base = dict(x=P, xs=256, r=P, rs=256, w=P, eps=1e-5, h=256, ro=P, ros=256, y=P, ys=256, y8=P, y8s=256, sc=P,
                group=128, n=P, t=8, status=None, stream=None)
    for fn in (lib.lora_add_rmsnorm, lib.lora_add_rmsnorm_f16):
        call = _caller(fn, names, base)
        for name in ("x", "w", "n", "sc"):
            assert call(**{name: None}) == -1, name
        assert call(y=None, y8=None, ro=None) == -1
        for kw in (dict(h=0), dict(h=252), dict(h=32776), dict(group=64), dict(group=0), dict(t=0), dict(t=1 << 23),
                   dict(xs=248), dict(rs=8), dict(ros=8), dict(ys=8), dict(y8s=8), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(h=264, xs=264, rs=264, ros=264, ys=264, y8s=264)):
            assert call(**kw) == -3, kw
        for kw in (dict(x=ODD), dict(r=ODD), dict(w=ODD), dict(ro=ODD), dict(y=ODD), dict(y8=ODD), dict(xs=260),
                   dict(y8s=260), dict(n=P + 2), dict(status=P + 2)):
            assert call(**kw) == -2, kw


def test_append_arguments(lib):
    names = ("q qs qo qos qh k ks v vs rope mp rd il pos slots cache pages kvh page d kf vf kh vh n t status "
             "stream").split()
    base = dict(q=P, qs=512, qo=P, qos=512, qh=4, k=P, ks=256, v=P, vs=256, rope=P, mp=100, rd=128, il=0, pos=P,
                slots=P, cache=P, pages=10, kvh=2, page=16, d=128, kf=1.0, vf=1.0, kh=None, vh=None, n=P, t=8,
                status=None, stream=None)
    for fn in (lib.lora_kv4_append, lib.lora_kv4_append_f16):
        call = _caller(fn, names, base)
        for name in ("k", "v", "slots", "cache", "n", "qo", "pos"):
            assert call(**{name: None}) == -1, name
        for kw in (dict(d=96), dict(d=32), dict(kvh=0), dict(kvh=257), dict(page=8), dict(page=24), dict(page=1040),
                   dict(pages=0), dict(pages=1 << 28), dict(kf=0.0), dict(vf=-1.0), dict(kf=float("inf")), dict(kf=1e-40),
                   dict(qh=0), dict(qh=300), dict(rd=16), dict(rd=160), dict(rd=48), dict(mp=0), dict(qs=504),
                   dict(qos=8), dict(ks=248), dict(vs=0), dict(t=0)):
            assert call(**kw) == -3, kw
        for kw in (dict(q=ODD), dict(qo=ODD), dict(k=ODD), dict(v=ODD), dict(cache=ODD), dict(rope=ODD), dict(kh=ODD),
                   dict(vh=ODD), dict(qs=516), dict(ks=260), dict(slots=P + 2), dict(pos=P + 1), dict(n=P + 2)):
            assert call(**kw) == -2, kw


def test_attention_arguments(lib):
    names = ("q qs o os lse qh cache pages kvh page d kf vf start kv table wide seqs t mq scale window ws wsb status "
             "stream").split()
    base = dict(q=P, qs=512, o=P, os=512, lse=None, qh=4, cache=P, pages=10, kvh=2, page=16, d=128, kf=1.0, vf=1.0,
                start=P, kv=P, table=P, wide=10, seqs=3, t=8, mq=4, scale=0.1, window=0, ws=P, wsb=1 << 30,
                status=None, stream=None)
    for fn in (lib.lora_kv4_attention, lib.lora_kv4_attention_f16):
        call = _caller(fn, names, base)
        for name in ("q", "o", "cache", "start", "kv", "table", "ws"):
            assert call(**{name: None}) == -1, name
        for kw in (dict(d=96), dict(qh=3), dict(qh=0), dict(qh=512), dict(kvh=0), dict(page=20), dict(pages=0),
                   dict(kf=0.0), dict(vf=float("nan")), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
                   dict(window=-1), dict(wide=0), dict(seqs=0), dict(seqs=65537), dict(t=0), dict(mq=0), dict(mq=9),
                   dict(qs=504), dict(os=504)):
            assert call(**kw) == -3, kw
        for kw in (dict(q=ODD), dict(o=ODD), dict(cache=ODD), dict(ws=ODD), dict(qs=516), dict(table=P + 2),
                   dict(lse=P + 2)):
            assert call(**kw) == -2, kw
        assert call(wsb=0) == -4
    size = B.lora_kv4_attention_workspace_size
    assert size(3, 8, 4, 4, 2, 128) > 0
    assert size(0, 8, 4, 4, 2, 128) == 0 and size(3, 8, 9, 4, 2, 128) == 0 and size(3, 8, 4, 4, 3, 128) == 0


def test_wrappers_want_cuda_tensors(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.lora_add_rmsnorm(x, x[0], 1e-5, torch.zeros(1, dtype=torch.int32), y=x)
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    cache = torch.zeros(1, 1, 1, 18 * 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.lora_kv4_append(cache, k, k, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.lora_kv4_attention(cache, k, k, None, None, None, 1, 0.1, None)


# ------------------------------------------------------------------ the formulas themselves

def test_formats():
    assert R.E4M3[0x7E] == 448 and R.E4M3[1] == 2.0 ** -9 and R.E4M3[0x38] == 1.0 and np.isnan(R.E4M3[0x7F])
    assert list(R.to_e4m3([0, 448, 1e9, np.nan, 1.0625, 1.1875, 2.0 ** -10])) == [0, 0x7E, 0x7E, 0x7F, 0x38, 0x3A, 0]
    ties = np.array([[6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6.0]])
    code, s8 = R.quantise32(ties, 1.0)
    assert s8[0, 0] == 0x38
    assert list(R.values(code, s8)[0]) == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, -6]
    assert np.array_equal(R.unpack(R.pack(code)), code)


def test_quantisation_keeps_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 128))
    code, s8 = R.quantise32(x, 0.25)
    got = R.values(code, s8) * 0.25
    step = np.repeat(R.E4M3[s8], 16, -1) * 0.25
    assert (np.abs(got - x) <= step * (1 + 1e-6)).all()  # half of the widest gap (4 to 6)


def test_cache_round_trip():
    rng = np.random.default_rng(1)
    k, v = [rng.standard_normal((21, 2, 64))], [rng.standard_normal((21, 2, 64))]
    table = np.array([[2, 0]])
    cache = R.build_cache(k, v, 3, table, 16, 0.5, 0.25)
    kk, vv = R.read_cache(cache, table[0], 21, 16, 64)
    for got, x, f in ((kk, k[0], 0.5), (vv, v[0], 0.25)):
        assert np.array_equal(got, R.values(*R.quantise32(x, f)))


def test_attention_formula_by_differences():
    """out = sum p v and d lse / d x_j = p_j: the formula against central differences of lse."""
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((1, 1, 8)), rng.standard_normal((5, 1, 8)), rng.standard_normal((5, 1, 8))
    out, lse, _, _ = R.attention(q, k, v, 0.3, 0)
    grad = np.zeros(8)
    for i in range(8):
        for sign in (1, -1):
            qq = q.copy()
            qq[0, 0, i] += sign * 1e-5
            grad[i] += sign * R.attention(qq, k, v, 0.3, 0)[1][0, 0] / 2e-5
    same, _, _, _ = R.attention(q, k, k, 0.3, 0)  # sum p k, so d lse / d q = scale * that
    assert np.allclose(grad, 0.3 * same[0, 0], atol=1e-8)
    assert np.allclose(out[0, 0], np.exp(k[:, 0] @ q[0, 0] * 0.3 - lse[0, 0]) @ v[:, 0])
    assert (R.attention(q, k, v, 0.3, 2)[0] == R.attention(q, k[3:], v[3:], 0.3, 0)[0]).all()
