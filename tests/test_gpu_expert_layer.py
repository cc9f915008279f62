"""The example layer: 8-bit serving and a 16-bit training step against the
same formulas in 32 bits (autograd).

E4M3 values carry a rounding error of up to 2^-4, uniformly spread about
2^-5.8 of them in the mean square; an output of the serving path sums
products of two such factors twice over, four roundings, so the relative
error in the norm stays below 4 * 2^-5 = 0.125.  The training path rounds its
intermediate rows to bfloat16 (2^-8 at most) at some eight places: below
8 * 2^-8 = 0.032.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,width,hidden", [(1000, 8, 512, 768), (1, 4, 128, 128),
                                                         (37, 16, 384, 200)])
def test_expert_layer(tokens, experts, width, hidden):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixed_precision_dense_02_gb300 import build
    build.build()
    from mixed_precision_dense_02_gb300 import expert_layer
    for name, e in expert_layer.demo(tokens, experts, width, hidden).items():
        assert e < (0.125 if name == "served output" else 0.032), (name, e)
