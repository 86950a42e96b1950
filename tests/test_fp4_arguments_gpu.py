"""Arguments of the 4-bit calls that contradict one another or the definition: refused, not answered in part."""
import pytest

import ternary_weight_bit_w2a8_b200 as bn

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

MX, NV = bn.BITNET_FP4_MX, bn.BITNET_FP4_NV


@pytest.fixture(scope="module")
def operands():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ternary_weight_bit_w2a8_b200 import build
    build.build()
    x = torch.ones(4, 256, dtype=torch.bfloat16, device="cuda")
    w, ws = bn.bitnet_fp4_quant(torch.ones(8, 256, device="cuda"), NV)
    a, sa = bn.bitnet_fp4_quant(x, NV)
    return x, a, sa, w, ws


# each call with a scale in one of its places
SCALED = {
    "tensor_scale": lambda o, g: bn.bitnet_fp4_tensor_scale(o[0], g=g),
    "quant": lambda o, g: bn.bitnet_fp4_quant(o[0], NV, g=g),
    "dequant": lambda o, g: bn.bitnet_fp4_dequant(o[1], o[2], 256, NV, g=g),
    "gemm_ga": lambda o, g: bn.bitnet_fp4_gemm(*o[1:], 256, NV, ga=g),
    "gemm_gw": lambda o, g: bn.bitnet_fp4_gemm(*o[1:], 256, NV, gw=g),
    "linear_ga": lambda o, g: bn.bitnet_fp4_linear(o[0], o[3], o[4], NV, ga=g),
    "linear_gw": lambda o, g: bn.bitnet_fp4_linear(o[0], o[3], o[4], NV, gw=g),
}


@pytest.mark.parametrize("call", list(SCALED))
@pytest.mark.parametrize("shape", [(0,), (2,), (4, 1), (8,)])
def test_a_scale_is_one_value(operands, call, shape):
    """A scale per token or per row is not what these calls compute with."""
    with pytest.raises(ValueError, match="one value"):
        SCALED[call](operands, torch.ones(shape, device="cuda"))


@pytest.mark.parametrize("call", list(SCALED))
def test_one_value_of_any_shape_is_a_scale(operands, call):
    many = torch.ones(3, device="cuda")
    for g in (torch.ones((), device="cuda"), torch.ones(1, 1, device="cuda"), many[1:2]):
        SCALED[call](operands, g)


# each call with an output and a type asked for
TYPED = {
    "dequant": lambda o, y, t: bn.bitnet_fp4_dequant(o[1], o[2], 256, NV, y=y, dtype=t),
    "gemm": lambda o, y, t: bn.bitnet_fp4_gemm(*o[1:], 256, NV, y=y, dtype=t),
    "linear": lambda o, y, t: bn.bitnet_fp4_linear(o[0], o[3], o[4], NV, y=y, dtype=t),
}


@pytest.mark.parametrize("call", list(TYPED))
def test_the_type_asked_for_is_that_of_y(operands, call):
    cols = 256 if call == "dequant" else 8
    y = torch.empty(4, cols, dtype=torch.float16, device="cuda")
    assert TYPED[call](operands, y, torch.float16).data_ptr() == y.data_ptr()
    assert TYPED[call](operands, y, None).data_ptr() == y.data_ptr()
    for t in (torch.bfloat16, torch.float32, torch.int8, "float16"):
        with pytest.raises(ValueError, match="dtype"):
            TYPED[call](operands, y, t)
