"""Every variant of the 4-bit kernels against 64 bits, between guard bands: every tile width of the product for more
tokens, every split of the one for few, and quantisation and reading back in patches of 64 rows."""
import numpy as np
import pytest

import fp4_plans as plans
import fp4_ref as ref
import ternary_weight_bit_w2a8_b200 as bn
from guarded import Guarded

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

FORMATS = [ref.MX, ref.NV]
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ternary_weight_bit_w2a8_b200 import build
    build.build()
    yield
    torch.cuda.synchronize()
    assert bn.bitnet_get_device_error() == 0


def random_matrix(rows, K, fmt, gen):
    """Codes and scales around 1 in the library's layout, and the values they stand for in 64 bits, by the layout's
    definition.  What lies past K is code 0; rows past the matrix have any scale, NaN among them."""
    Kp, B = ref.pad_up(K, 128), ref.BLOCK[fmt]
    code = torch.randint(0, 16, (rows, Kp), dtype=torch.uint8, device="cuda", generator=gen)
    code[:, K:] = 0
    lo = 124 if fmt == ref.MX else 32
    nb, bands = Kp // B, -(-rows // 128)
    sb = torch.randint(lo, lo + (6 if fmt == ref.MX else 48), (128 * bands, nb), dtype=torch.uint8, device="cuda",
                       generator=gen)
    sb[rows:] = 255 if fmt == ref.MX else 127
    # tile [band, 4 blocks]: byte 16 * (r % 32) + 4 * (r / 32) + c
    tiles = sb.view(bands, 4, 32, nb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    grid = torch.tensor(np.concatenate([ref.GRID, -ref.GRID]), device="cuda")
    scale = torch.from_numpy(ref.scale_values(np.arange(256), fmt)).cuda()
    v = grid[code.int()] * scale[sb[:rows].int()].repeat_interleave(B, dim=1)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), tiles, v


def check(y, av, wv, scale, K):
    want, mag = av @ wv.t() * scale, av.abs() @ wv.abs().t() * scale
    err, half = (y.double() - want).abs(), torch.finfo(y.dtype).eps / 2
    # (ref.product_tolerance) half a step of y, K / 16 additions and a few more off by 2^-22 of the magnitudes at most
    tol = half * want.abs() * (1 + 2.0 ** -20) + mag * (K / 16 + 17) * 2.0 ** -22 + torch.finfo(y.dtype).tiny
    bad = err > tol
    assert not bool(bad.any()), (bad.nonzero()[:5].tolist(), y[bad][:5].tolist(), want[bad][:5].tolist())
    # Together much nearer: a rounding's error is spread over half a step either way, so its root mean square is 0.58
    # of half a step at most; the fp32 sums may add half of that again.
    assert float(err.square().mean().sqrt()) <= 0.7 * half * float(want.square().mean().sqrt())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,first,behind", plans.PAIRS)
def test_every_pair_kernel(fmt, M, N, K, first, behind):
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, a_s, av = random_matrix(M, K, fmt, gen)
    w, w_s, wv = random_matrix(N, K, fmt, gen)
    gw = torch.tensor([2.0 ** -4 / K ** 0.5], dtype=torch.float32, device="cuda")
    for dtype in (torch.bfloat16, torch.float16):
        out = Guarded(torch, (M, first + N + behind), dtype, fill=7.0)
        y = out.t[:, first:first + N]
        bn.bitnet_fp4_gemm(a, a_s, w, w_s, K, fmt, gw=gw, y=y)
        out.check("y")
        assert bool((out.t[:, :first] == 7.0).all()) and bool((out.t[:, first + N:] == 7.0).all())
        check(y, av, wv, float(gw.item()), K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", plans.FEW)
def test_every_split_of_few_tokens(fmt, M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, a_s, av = random_matrix(M, K, fmt, gen)
    w, w_s, wv = random_matrix(N, K, fmt, gen)
    gw = torch.tensor([2.0 ** -4 / K ** 0.5], dtype=torch.float32, device="cuda")
    for dtype, behind in ((torch.bfloat16, 0), (torch.float16, 3)):
        out = Guarded(torch, (M, N + behind), dtype, fill=7.0)
        bn.bitnet_fp4_gemm(a, a_s, w, w_s, K, fmt, gw=gw, y=out.t[:, :N])
        out.check("y")
        assert bool((out.t[:, N:] == 7.0).all())
        check(out.t[:, :N], av, wv, float(gw.item()), K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("M,N,K", [s for s in plans.FEW if s[0] <= 16])
def test_every_split_quantised_in_the_launch(fmt, dt, M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    w, w_s, wv = random_matrix(N, K, fmt, gen)
    for pad in (0, 1, -K % 16):  # rows of x as they come, off every boundary, on 32-byte ones
        x = torch.randn(M, K + pad, device="cuda", generator=gen).to(TYPES[dt])[:, :K]
        c, sb = ref.quantise(x.float().cpu().numpy(), fmt)
        av = torch.from_numpy(ref.values(c, sb, fmt)).cuda()
        gw = torch.tensor([2.0 ** -4 / K ** 0.5], dtype=torch.float32, device="cuda")
        out = Guarded(torch, (M, N), torch.bfloat16, fill=7.0)
        bn.bitnet_fp4_linear(x, w, w_s, fmt, gw=gw, y=out.t)
        out.check("y")
        check(out.t, av, wv, float(gw.item()), K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,K,behind", plans.PATCHES)
def test_quant_in_patches_of_64_rows(fmt, dt, rows, K, behind):
    rng = np.random.default_rng(rows + K + behind)
    x = (rng.standard_normal((rows, K), dtype=np.float32) * np.exp2(rng.integers(-9, 4, (rows, 1)))).astype(np.float32)
    x[:, : K // 3] *= rng.random((rows, K // 3)) < 0.7
    x[rows - 70, 3], x[rows - 1, K - 1], x[64, 100] = np.nan, np.inf, -np.inf
    t = torch.full((rows, K + behind), float("nan"), dtype=TYPES[dt])  # what lies between the rows is not read
    t[:, :K] = torch.from_numpy(x)
    xd = t.cuda()[:, :K]
    codes = Guarded(torch, (rows, bn.bitnet_fp4_code_bytes(1, K)), torch.uint8)
    scales = Guarded(torch, (bn.bitnet_fp4_scale_bytes(rows, K, fmt),), torch.uint8)
    bn.bitnet_fp4_quant(xd, fmt, codes=codes.t, scales=scales.t)
    codes.check("codes")
    scales.check("scales")
    p, s = ref.pack(*ref.quantise(t[:, :K].float().numpy(), fmt), fmt)
    assert np.array_equal(scales.t.cpu().numpy(), s)  # the rows past the matrix too: 0
    nz = lambda b: np.stack([np.where(b & 7, b & 15, 0), np.where(b & 0x70, b >> 4, 0)])  # noqa: E731 (a zero's sign is free)
    assert np.array_equal(nz(codes.t.cpu().numpy()), nz(p))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,K,behind", plans.PATCHES)
def test_dequant_in_patches_of_64_rows(fmt, dt, rows, K, behind):
    gen = torch.Generator(device="cuda").manual_seed(rows + K + behind)
    p, s, v = random_matrix(rows, K, fmt, gen)
    g = torch.tensor([0.3], dtype=torch.float32, device="cuda")
    want = (v[:, :K].float() * g).to(TYPES[dt])
    out = Guarded(torch, (rows, K + behind), TYPES[dt], fill=5.0)
    bn.bitnet_fp4_dequant(p, s, K, fmt, g=g, y=out.t[:, :K])
    out.check("y")
    assert torch.equal(out.t[:, :K], want)
    assert bool((out.t[:, K:] == 5.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [5, 40, 100])
def test_layer_of_tokens_that_are_not_finite(fmt, M):
    """A token with a NaN or an infinity gives NaN, and the others what they give without it."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, 700, device="cuda", generator=gen).to(torch.bfloat16)
    w, w_s = bn.bitnet_fp4_quant(torch.randn(300, 700, device="cuda", generator=gen), fmt)
    clean = bn.bitnet_fp4_linear(x, w, w_s, fmt)
    x[1, 699], x[4, 0] = float("nan"), float("-inf")
    y = bn.bitnet_fp4_linear(x, w, w_s, fmt)
    assert bool(y[[1, 4]].isnan().all())
    rest = [m for m in range(M) if m not in (1, 4)]
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("dt", list(TYPES))
def test_tensor_scale_of_every_cluster(dt):
    """One to eight CTAs of a cluster, and more without one, each holding the largest value once."""
    per_cta = (8 if dt == "fp32" else 16) * 32 * 4 * 8  # values that a CTA's eight warps take at once
    for ctas in (1, 2, 3, 5, 7, 8, 9, 12):
        n = ctas * per_cta - 5
        x = torch.full((1, n), 0.5, dtype=TYPES[dt], device="cuda")
        for at in range(0, n, per_cta):
            x[0, at + 3] = -(2.0 + at / per_cta)
            got = bn.bitnet_fp4_tensor_scale(x)
            x[0, at + 3] = 0.5
            want = np.float32(2.0 + at / per_cta) / np.float32(2688)
            assert got.item() == want, (ctas, at)
