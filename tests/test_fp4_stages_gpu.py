"""Products over every number of stages of k around the depths of the kernels' rings (3 to 8 stages): what a CTA waits for
before it leaves, where its ring has not gone round, has just done so, and has done so several times.  A wait on the
wrong phase would run out (1 s) and be reported."""
import pytest

import ternary_weight_bit_w2a8_b200 as bn

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ternary_weight_bit_w2a8_b200 import build
    build.build()


# clusters over k and one CTA to a tile; tokens quantised in the launch; pairs with a tile each, with a range of k of
# one, and with several tiles
SHAPES = [("gemm", 1, 300), ("gemm", 20, 21000), ("linear", 3, 300), ("linear", 16, 33000), ("gemm", 130, 2500),
          ("gemm", 70, 64), ("gemm", 700, 7000)]


@pytest.mark.parametrize("fmt", [bn.BITNET_FP4_MX, bn.BITNET_FP4_NV])
@pytest.mark.parametrize("call,M,N", SHAPES)
def test_every_number_of_stages(fmt, call, M, N):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    for stages in list(range(1, 19)) + [24, 25, 33, 47, 64]:
        K = 256 * stages - (128 if stages % 2 else 0)  # (the last one may hold half)
        x = torch.randn(M, K, device="cuda", generator=gen)
        w, ws = bn.bitnet_fp4_quant(torch.randn(N, K, device="cuda", generator=gen), fmt)
        a, sa = bn.bitnet_fp4_quant(x, fmt)
        if call == "gemm":
            y = bn.bitnet_fp4_gemm(a, sa, w, ws, K, fmt)
        else:
            y = bn.bitnet_fp4_linear(x, w, ws, fmt)
        assert bn.bitnet_get_device_error() == bn.BITNET_OK, stages
        # the values read back are exact, and so are their products in 64 bits
        av, wv = (bn.bitnet_fp4_dequant(c, s, K, fmt, dtype=torch.float32).double() for c, s in ((a, sa), (w, ws)))
        want, mag = av @ wv.t(), av.abs() @ wv.abs().t()
        tol = want.abs() * 2.0 ** -8 + mag * (K / 16 + 16) * 2.0 ** -22  # half a step of bf16, and the fp32 sums'
        assert bool(((y.double() - want).abs() <= tol).all()), stages


@pytest.mark.parametrize("fmt", [bn.BITNET_FP4_MX, bn.BITNET_FP4_NV])
@pytest.mark.parametrize("N", [64, 128, 192, 256, 384])
def test_every_number_of_tiles(fmt, N):
    """One, two and three tiles to a pair of the 74, and one pair with one more: which uses of the accumulators are
    handed back."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    for K in (128, 1300):
        w, ws = bn.bitnet_fp4_quant(torch.randn(N, K, device="cuda", generator=gen), fmt)
        wv = bn.bitnet_fp4_dequant(w, ws, K, fmt, dtype=torch.float32).double()
        for tiles in (1, 73, 74, 75, 147, 148, 149, 222, 223):
            M = 256 * tiles - 100
            a, sa = bn.bitnet_fp4_quant(torch.randn(M, K, device="cuda", generator=gen), fmt)
            av = bn.bitnet_fp4_dequant(a, sa, K, fmt, dtype=torch.float32).double()
            want, mag = av @ wv.t(), av.abs() @ wv.abs().t()
            tol = want.abs() * 2.0 ** -8 + mag * (K / 16 + 16) * 2.0 ** -22
            for behind in (0, 1):
                y = torch.empty(M, N + behind, dtype=torch.bfloat16, device="cuda")[:, :N]
                bn.bitnet_fp4_gemm(a, sa, w, ws, K, fmt, y=y)
                assert bn.bitnet_get_device_error() == bn.BITNET_OK, (K, tiles)
                assert bool(((y.double() - want).abs() <= tol).all()), (K, tiles)
