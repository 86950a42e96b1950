"""Products whose tensor scales multiply to less, or more, than fp32 holds while the result is an ordinary number."""
import numpy as np
import pytest

import fp4_ref as ref
import ternary_weight_bit_w2a8_b200 as bn

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ternary_weight_bit_w2a8_b200 import build
    build.build()
    yield
    torch.cuda.synchronize()
    assert bn.bitnet_get_device_error() == 0


# one token and a cluster to a tile; one CTA to a tile; pairs, several to a tile (long k) and one, and tiles of two
# halves; rows of y on 16-byte boundaries and off them
SHAPES = [(1, 600, 2560), (40, 300, 300), (70, 200, 5120), (130, 1000, 256), (2048, 2568, 512), (2048, 2569, 512)]


# format, ga, gw, and the first of the six scale bytes used
CASES = [(ref.MX, 2.0 ** -70 * 1.3, 2.0 ** -72, 146),    # 2^-142: 8 bits of it left
         (ref.MX, 2.0 ** -80, 2.0 ** -81 * 1.7, 154),    # 2^-160: none
         (ref.MX, 2.0 ** -20 * 1.1, 2.0 ** -130, 146),   # a subnormal scale
         (ref.MX, 2.0 ** 64 * 1.7, 2.0 ** 64, 110),      # beyond the top
         (ref.NV, 2.0 ** -70 * 1.3, 2.0 ** -71, 112),
         (ref.NV, 2.0 ** -10 * 1.1, 2.0 ** -130, 112),
         (ref.NV, 2.0 ** 64 * 1.7, 2.0 ** 64, 1)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt,ga,gw,first", CASES)
def test_product_of_scales_beyond_fp32(fmt, M, N, K, ga, gw, first):
    rng = np.random.default_rng(M + N + K)
    ca, sa = ref.random_matrix(M, K, fmt, rng)
    cw, sw = ref.random_matrix(N, K, fmt, rng)
    sa, sw = (rng.integers(first, first + 6, s.shape).astype(np.uint8) for s in (sa, sw))
    (a, a_s), (w, w_s) = ([torch.from_numpy(t).cuda() for t in ref.pack(c, s, fmt)] for c, s in ((ca, sa), (cw, sw)))
    gat, gwt = (torch.tensor([g], dtype=torch.float32, device="cuda") for g in (ga, gw))
    y = bn.bitnet_fp4_gemm(a, a_s, w, w_s, K, fmt, ga=gat, gw=gwt, dtype=torch.bfloat16)
    want, mag = ref.product(ref.values(ca, sa, fmt), ref.values(cw, sw, fmt), float(gat.item()) * float(gwt.item()))
    got = y.double().cpu().numpy()
    # ordinary bf16 numbers: far from 2^-126 and from the top
    assert 2.0 ** -121 < np.median(np.abs(want)) and np.abs(want).max() < 2.0 ** 127
    # one rounding more than a product whose scales fit; and a step of subnormal bf16 numbers
    tol = ref.product_tolerance(want, mag, K, torch.finfo(torch.bfloat16).eps) + mag * 2.0 ** -22 + 2.0 ** -133
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


@pytest.mark.parametrize("M", [3, 100])
def test_layer_of_tiny_tensors(M):
    """NV layers of values around 1e-21 and 1e-17, with the scales that the library itself takes for them (together
    some 2^-145): the result is around 2^-120."""
    gen = torch.Generator().manual_seed(M)
    K = 7000
    x = torch.randn(M, K, generator=gen) * 1e-21
    W = torch.randn(90, K, generator=gen) * 1e-17
    ga, gw = bn.bitnet_fp4_tensor_scale(x.cuda()), bn.bitnet_fp4_tensor_scale(W.cuda())
    w, ws = bn.bitnet_fp4_quant(W.cuda(), ref.NV, g=gw)
    y = bn.bitnet_fp4_linear(x.cuda(), w, ws, ref.NV, ga=ga, gw=gw, dtype=torch.bfloat16).double().cpu().numpy()
    av, wv = (ref.values(*ref.quantise(t.numpy(), ref.NV, g.item()), ref.NV) for t, g in ((x, ga), (W, gw)))
    want, mag = ref.product(av, wv, float(ga.item()) * float(gw.item()))
    tol = ref.product_tolerance(want, mag, K, torch.finfo(torch.bfloat16).eps) + mag * 2.0 ** -22 + 2.0 ** -133
    assert np.all(np.abs(y - want) <= tol)


@pytest.mark.parametrize("M", [1, 40, 70, 300])
@pytest.mark.parametrize("ga,gw", [(0.0, 1e30), (1e30, 0.0), (0.0, 0.0), (0.0, 1e-40)])
def test_a_scale_of_zero(M, ga, gw):
    w, ws = bn.bitnet_fp4_quant(torch.randn(200, 640, device="cuda"), ref.MX)
    a, sa = bn.bitnet_fp4_quant(torch.randn(M, 640, device="cuda"), ref.MX)
    g = [torch.tensor([v], dtype=torch.float32, device="cuda") for v in (ga, gw)]
    assert not bn.bitnet_fp4_gemm(a, sa, w, ws, 640, ref.MX, ga=g[0], gw=g[1]).any()
