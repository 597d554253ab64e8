"""The example of a decoder layer's attention half, run as a user runs it, against the same steps in
plain PyTorch in fp32 (over the values that the cache holds)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gathered_rank_gemm_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


# bf16 roundings (2^-9 rms of a rounding is about 2^-9 / sqrt(3)) of x, y, q, o and the output, each
# carried on by a product of norm about one: about 5 * 2^-9; twice that is allowed
TOLERANCE = 2.0 ** -5.5


@pytest.mark.parametrize("shape", [dict(), dict(q_heads=4, kv_heads=4, head_dim=128, page_size=32, rank=8),
                                   dict(q_heads=16, kv_heads=1, head_dim=64, max_tokens=300)])
def test_layer(example, shape):
    layer = example.Layer(**shape)
    worst, steps, status = example.check(layer, prompts=[37, 100, 5, 64], chunk=48, new_tokens=4)
    assert steps > 4 and status == 0
    assert worst < TOLERANCE
