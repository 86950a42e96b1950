"""Microscaled 4-bit floating point on the GPU: quantisation bit by bit, reading
back, products and the linear layer against 64 bits."""
import numpy as np
import pytest

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


def activations(rows, K, dtype, seed):
    """fp32 numpy values that the type holds, with zero blocks, outliers and rows of very different size."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-9, 4, (rows, 1)))
    x *= np.where(rng.random((rows, K)) < 0.02, 20.0, 1.0)
    x[:, : K // 3] *= rng.random((rows, K // 3)) < 0.7
    if K > 70:
        x[rows // 2, 32:70] = 0
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    return t, t.float().numpy()


def device_matrix(codes, sb, fmt):
    p, s = ref.pack(codes, sb, fmt)
    return torch.from_numpy(p).cuda(), torch.from_numpy(s).cuda()


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,K,pad", [(1, 1, 0), (1, 2560, 0), (5, 16, 0), (3, 130, 1), (33, 257, 3), (129, 383, 8),
                                        (300, 640, 0), (127, 1031, 2)])
def test_quant_bit_exact(fmt, dt, rows, K, pad):
    t, x = activations(rows, K, TYPES[dt], rows * 1000 + K)
    wide = torch.full((rows, K + pad), float("nan"), dtype=TYPES[dt])  # what lies between the rows is not read
    wide[:, :K] = t
    xd = wide.cuda()[:, :K]
    for g in (None, 0.37 if fmt == ref.MX else 0.0113):
        gd = None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")
        gv = None if g is None else gd.item()
        codes = Guarded(torch, (rows, bn.bitnet_fp4_code_bytes(1, K)), torch.uint8)
        scales = Guarded(torch, (bn.bitnet_fp4_scale_bytes(rows, K, fmt),), torch.uint8)
        bn.bitnet_fp4_quant(xd, fmt, g=gd, codes=codes.t, scales=scales.t)
        codes.check("codes")
        scales.check("scales")
        c, sb = ref.quantise(x, fmt, gv)
        p, s = ref.pack(c, sb, fmt)
        got = codes.t.cpu().numpy()
        # the sign of a zero is not part of the definition
        nz = lambda b: np.stack([np.where(b & 7, b & 15, 0), np.where(b & 0x70, b >> 4, 0)])  # noqa: E731
        assert np.array_equal(scales.t.cpu().numpy(), s)
        assert np.array_equal(nz(got), nz(p))


@pytest.mark.parametrize("fmt", FORMATS)
def test_quant_ties_and_borders(fmt):
    """Every midpoint of two elements times every block scale, and its fp32 neighbours: z / s is compared exactly."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    B = ref.BLOCK[fmt]
    scales = np.ldexp(1.0, np.arange(-126, 124, 7)) if fmt == ref.MX else ref.E4M3[1:]
    rows = []
    for s in scales:
        m = (mids * s).astype(np.float32)
        v = np.concatenate([m, np.nextafter(m, np.float32(np.inf)), np.nextafter(m, np.float32(0)), -m])
        for part in np.array_split(v, 4):  # with the block's largest value beside them
            row = np.zeros(B, dtype=np.float32)
            row[0] = 6 * s
            row[1:1 + len(part)] = part
            rows.append(row)
    x = np.stack(rows)
    c, sb = ref.quantise(x, fmt)
    codes, sc = bn.bitnet_fp4_quant(torch.from_numpy(x).cuda(), fmt)
    p, s = ref.pack(c, sb, fmt)
    assert np.array_equal(sc.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), p)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quant_non_finite_and_tiny(fmt):
    x = np.ones((4, 256), dtype=np.float32)
    x[0, 3] = np.nan
    x[1, 40] = np.inf
    x[2, 255] = -np.inf
    x[3, :64] = 1e-44       # subnormal
    x[3, 64:128] = 3e38     # near the top
    x[3, 128:192] = 2.0 ** -126
    c, sb = ref.quantise(x, fmt)
    codes, sc = bn.bitnet_fp4_quant(torch.from_numpy(x).cuda(), fmt)
    p, s = ref.pack(c, sb, fmt)
    assert np.array_equal(sc.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), p)
    y = bn.bitnet_fp4_dequant(codes, sc, 256, fmt, dtype=torch.float32).cpu().numpy()
    B = ref.BLOCK[fmt]
    assert np.isnan(y[0, :B]).all() and np.isfinite(y[0, B:]).all()
    assert np.isnan(y[1, 40 // B * B:(40 // B + 1) * B]).all() and np.isnan(y[2, -B:]).all()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,K,pad", [(1, 1, 0), (3, 77, 1), (9, 2560, 0), (33, 2560, 1), (64, 2048, 0), (500, 1031, 0),
                                        (2048, 2560, 8)])
def test_tensor_scale(dt, rows, K, pad):
    t, x = activations(rows, K, TYPES[dt], K)
    t[rows // 2, K // 2] = float("inf")
    t[0, 0] = float("nan") if rows * K > 1 else 3.0
    x = t.float().numpy()
    wide = torch.full((rows, K + pad), 6e4, dtype=TYPES[dt])
    wide[:, :K] = t
    top = np.abs(np.where(np.isfinite(x), x, 0)).max()
    want = np.maximum(top.astype(np.float32) / np.float32(2688), np.float32(2.0 ** -126))
    assert bn.bitnet_fp4_tensor_scale(wide.cuda()[:, :K]).item() == want
    z = torch.zeros(rows, K, dtype=TYPES[dt], device="cuda")
    assert bn.bitnet_fp4_tensor_scale(z).item() == 2.0 ** -126


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,K,pad", [(1, 1, 0), (3, 130, 1), (129, 383, 8), (260, 512, 0)])
def test_dequant(fmt, dt, rows, K, pad):
    rng = np.random.default_rng(K)
    codes, sb = ref.random_matrix(rows, K, fmt, rng)
    p, s = device_matrix(codes, sb, fmt)
    g = torch.tensor([0.3], dtype=torch.float32, device="cuda")
    v = ref.values(codes, sb, fmt)[:, :K].astype(np.float32)
    for gd in (None, g):
        want = torch.from_numpy(v * (np.float32(1) if gd is None else np.float32(g.item()))).to(TYPES[dt])
        out = Guarded(torch, (rows, K + pad), TYPES[dt], fill=5.0)
        bn.bitnet_fp4_dequant(p, s, K, fmt, g=gd, y=out.t[:, :K])
        out.check("y")
        assert torch.equal(out.t[:, :K].cpu(), want)
        assert bool((out.t[:, K:] == 5.0).all())


# ------------------------------------------------------------------ product
def check_product(y, codes_a, sa, codes_w, sw, fmt, K, scale):
    av, wv = ref.values(codes_a, sa, fmt), ref.values(codes_w, sw, fmt)
    want, mag = ref.product(av, wv, scale)
    eps = torch.finfo(y.dtype).eps
    got = y.float().cpu().numpy().astype(np.float64)
    tol = ref.product_tolerance(want, mag, K, eps) + torch.finfo(y.dtype).tiny
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 2560, 2560), (2, 129, 64), (3, 300, 1000), (8, 1000, 6912), (16, 257, 300),
          (17, 640, 512), (31, 96, 4100), (64, 513, 2560), (65, 100, 130), (100, 777, 1024), (128, 1000, 260),
          (129, 333, 700), (200, 1000, 2560), (257, 129, 5120), (513, 1100, 384), (1000, 640, 65), (1, 5, 20000),
          (600, 600, 600), (300, 20000, 256), (2100, 5000, 512), (520, 9700, 1000), (1030, 11111, 192),
          (510, 7001, 3000), (2048, 2560, 2000), (700, 4700, 256),
          (130, 300, 5000), (70, 1501, 4801), (300, 700, 4100), (448, 800, 9000), (65, 200, 16000)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(fmt, M, N, K):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    ca, sa = ref.random_matrix(M, K, fmt, rng)
    cw, sw = ref.random_matrix(N, K, fmt, rng)
    a, a_s = device_matrix(ca, sa, fmt)
    w, w_s = device_matrix(cw, sw, fmt)
    dtype = torch.bfloat16 if (M + N) % 2 else torch.float16
    g = 2.0 ** -6 / np.sqrt(K)
    ga = torch.tensor([0.75], dtype=torch.float32, device="cuda")
    gw = torch.tensor([g], dtype=torch.float32, device="cuda")
    for first, pad in [(0, [0, 8, 3][K % 3]), (1, [2, 3][N % 2])]:  # and rows off every boundary
        out = Guarded(torch, (M, first + N + pad), dtype, fill=7.0)
        y = out.t[:, first:first + N]
        bn.bitnet_fp4_gemm(a, a_s, w, w_s, K, fmt, ga=ga, gw=gw, y=y)
        out.check("y")
        assert bool((out.t[:, :first] == 7.0).all()) and bool((out.t[:, first + N:] == 7.0).all())
        check_product(y, ca, sa, cw, sw, fmt, K, 0.75 * float(gw.item()))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(3, 300, 1000), (65, 200, 16000), (130, 300, 5000), (513, 6643, 1113), (2047, 5000, 300)])
def test_product_bits_do_not_depend_on_rows_of_y(fmt, M, N, K):
    """The same sums whatever boundaries the rows of y start on."""
    rng = np.random.default_rng(K)
    a, a_s = device_matrix(*ref.random_matrix(M, K, fmt, rng), fmt)
    w, w_s = device_matrix(*ref.random_matrix(N, K, fmt, rng), fmt)
    ldy = -(-N // 8) * 8 + 8
    want = bn.bitnet_fp4_gemm(a, a_s, w, w_s, K, fmt, y=torch.empty(M, ldy, dtype=torch.float16, device="cuda")[:, :N])
    for first, pad in [(1, 0), (2, 0), (4, 1)]:
        y = torch.empty(M, ldy + pad, dtype=torch.float16, device="cuda")[:, first:first + N]
        assert torch.equal(bn.bitnet_fp4_gemm(a, a_s, w, w_s, K, fmt, y=y), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_product_of_nan_scales(fmt, M):
    """A NaN block makes its row NaN and no other."""
    rng = np.random.default_rng(M)
    N, K = 140, 500
    ca, sa = ref.random_matrix(M, K, fmt, rng)
    cw, sw = ref.random_matrix(N, K, fmt, rng)
    sw[130, 3] = 255 if fmt == ref.MX else 127
    a, a_s = device_matrix(ca, sa, fmt)
    w, w_s = device_matrix(cw, sw, fmt)
    y = bn.bitnet_fp4_gemm(a, a_s, w, w_s, K, fmt, dtype=torch.bfloat16).float().cpu().numpy()
    assert np.isnan(y[:, 130]).all()
    assert np.isfinite(np.delete(y, 130, axis=1)).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_of_nothing(fmt):
    w, w_s = bn.bitnet_fp4_quant(torch.ones(5, 64, device="cuda"), fmt)
    a = torch.empty(3, 0, dtype=torch.uint8, device="cuda")
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    y = bn.bitnet_fp4_gemm(a, e, torch.empty(5, 0, dtype=torch.uint8, device="cuda"), e, 0, fmt)
    assert y.shape == (3, 5) and not y.any()
    assert bn.bitnet_fp4_gemm(torch.empty(0, 64, dtype=torch.uint8, device="cuda"), e, w, w_s, 64, fmt).shape == (0, 5)


# ------------------------------------------------------------------ linear
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("M,N,K,pad", [(1, 300, 2560, 0), (1, 129, 1000, 1), (2, 64, 130, 8), (4, 500, 6912, 0),
                                       (9, 300, 515, 0), (16, 1000, 2560, 8), (17, 96, 640, 1), (130, 300, 2560, 0),
                                       (300, 257, 700, 3)])
def test_linear_is_quant_and_product(fmt, dt, M, N, K, pad):
    """The whole layer: bit by bit the two calls, and near the exact product of the quantised values."""
    t, x = activations(M, K, TYPES[dt], M + K)
    wide = torch.zeros(M, K + pad, dtype=TYPES[dt])
    wide[:, :K] = t
    xd = wide.cuda()[:, :K]
    W = torch.randn(N, K, generator=torch.Generator().manual_seed(N)) * 0.02
    ga = gw = None
    if fmt == ref.NV:
        ga, gw = bn.bitnet_fp4_tensor_scale(xd), bn.bitnet_fp4_tensor_scale(W.cuda())
    w, w_s = bn.bitnet_fp4_quant(W.cuda(), fmt, g=gw)
    y = bn.bitnet_fp4_linear(xd, w, w_s, fmt, ga=ga, gw=gw, dtype=torch.bfloat16)
    a, a_s = bn.bitnet_fp4_quant(xd, fmt, g=ga)
    y2 = bn.bitnet_fp4_gemm(a, a_s, w, w_s, K, fmt, ga=ga, gw=gw, dtype=torch.bfloat16)
    assert torch.equal(y, y2)
    gav, gwv = (1.0, 1.0) if ga is None else (ga.item(), gw.item())
    ca, sa = ref.quantise(x, fmt, None if ga is None else gav)
    cw, sw = ref.quantise(W.numpy(), fmt, None if gw is None else gwv)
    check_product(y, ca, sa, cw, sw, fmt, K, gav * gwv)


def test_layers_in_a_graph_on_another_stream():
    """Two layers with an activation between them, captured once and replayed on new inputs; and the same on a side
    stream: equal to the calls one by one."""
    fmt, M, D, H = ref.NV, 5, 640, 1500
    gen = torch.Generator().manual_seed(1)
    ws = []
    for n, k in ((H, D), (D, H)):
        W = (torch.randn(n, k, generator=gen) * 0.03).cuda()
        g = bn.bitnet_fp4_tensor_scale(W)
        ws.append((*bn.bitnet_fp4_quant(W, fmt, g=g), g))
    x = torch.randn(M, D, generator=gen).to(torch.bfloat16).cuda()

    def block(t):
        ga = bn.bitnet_fp4_tensor_scale(t)
        h = bn.bitnet_fp4_linear(t, ws[0][0], ws[0][1], fmt, ga=ga, gw=ws[0][2])
        h = torch.relu(h) ** 2
        gh = bn.bitnet_fp4_tensor_scale(h)
        return bn.bitnet_fp4_linear(h, ws[1][0], ws[1][1], fmt, ga=gh, gw=ws[1][2])

    want = block(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block(x)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(graph):
        out = block(xs)
    for seed in (2, 3):
        x2 = torch.randn(M, D, generator=gen.manual_seed(seed)).to(torch.bfloat16).cuda()
        xs.copy_(x2)
        graph.replay()
        assert torch.equal(out, block(x2))
    # an explicit stream argument
    y = bn.bitnet_fp4_linear(x, ws[0][0], ws[0][1], fmt, gw=ws[0][2], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, bn.bitnet_fp4_linear(x, ws[0][0], ws[0][1], fmt, gw=ws[0][2]))


def quantised_weight(N, K, fmt, seed):
    W = (torch.randn(N, K, generator=torch.Generator().manual_seed(seed)) * 0.02).cuda()
    return bn.bitnet_fp4_quant(W, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_calls_that_overlap(fmt):
    """Products of both kernels and fused layers on two streams at once, and two graphs replayed at once: the bits of
    the calls one by one, again and again."""
    gen = torch.Generator().manual_seed(7)
    shapes = [(1, 2560, 6912), (12, 1000, 2560), (150, 3000, 1280), (1, 300, 700)]
    work = []
    for i, (M, N, K) in enumerate(shapes):
        x = torch.randn(M, K, generator=gen).to(torch.bfloat16).cuda()
        w, s = quantised_weight(N, K, fmt, i)
        work.append((x, w, s, bn.bitnet_fp4_linear(x, w, s, fmt)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for rep in range(20):
        for j, st in enumerate(streams):
            x, w, s, want = work[(rep + j) % len(work)]
            with torch.cuda.stream(st):
                outs.append((bn.bitnet_fp4_linear(x, w, s, fmt), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)
    graphs = []
    for j in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys = [bn.bitnet_fp4_linear(x, w, s, fmt) for x, w, s, _ in work[2 * j:2 * j + 2]]
        graphs.append((g, ys))
    for rep in range(5):
        for (g, ys), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for j, (g, ys) in enumerate(graphs):
        assert all(torch.equal(y, work[2 * j + i][3]) for i, y in enumerate(ys))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_weights_written_just_before(fmt, M):
    """A layer right behind the kernels that write its weights and its tokens, again and again into the same buffers:
    nothing of the values before is read."""
    N, K = 1300, 2560
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(bn.bitnet_fp4_scale_bytes(N, K, fmt), dtype=torch.uint8, device="cuda")
    Ws = [(torch.randn(N, K, generator=torch.Generator().manual_seed(i)) * 0.02).cuda() for i in range(3)]
    xs = [torch.randn(M, K, generator=torch.Generator().manual_seed(9 + i)).to(torch.bfloat16).cuda() for i in range(3)]
    want = []
    for W, x in zip(Ws, xs):
        w, s = bn.bitnet_fp4_quant(W, fmt)
        torch.cuda.synchronize()
        want.append(bn.bitnet_fp4_linear(x, w, s, fmt))
        torch.cuda.synchronize()
    x = torch.empty_like(xs[0])
    got = []
    for rep in range(30):
        x.copy_(xs[rep % 3])
        bn.bitnet_fp4_quant(Ws[rep % 3], fmt, codes=codes, scales=scales)
        got.append(bn.bitnet_fp4_linear(x, codes, scales, fmt))
    for rep, y in enumerate(got):
        assert torch.equal(y, want[rep % 3]), rep


def test_binding_refuses_what_does_not_fit():
    w, s = quantised_weight(64, 256, ref.MX, 0)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    ok = bn.bitnet_fp4_linear(x, w, s, ref.MX)
    assert ok.shape == (4, 64)
    bad = [lambda: bn.bitnet_fp4_linear(x[:, :200], w, s, ref.NV),            # NV needs twice the scales
           lambda: bn.bitnet_fp4_linear(x.to(torch.int8), w, s, ref.MX),
           lambda: bn.bitnet_fp4_linear(x.t(), w, s, ref.MX),
           lambda: bn.bitnet_fp4_linear(x, w.cpu(), s, ref.MX),
           lambda: bn.bitnet_fp4_linear(x, w[:, :64], s, ref.MX),
           lambda: bn.bitnet_fp4_linear(x, w, s[:-1], ref.MX),
           lambda: bn.bitnet_fp4_linear(x, w, s, 2),
           lambda: bn.bitnet_fp4_linear(x, w, s, ref.MX, ga=torch.ones(1)),
           lambda: bn.bitnet_fp4_linear(x, w, s, ref.MX, y=torch.empty(4, 63, device="cuda")),
           lambda: bn.bitnet_fp4_quant(x, ref.MX, codes=w),
           lambda: bn.bitnet_fp4_quant(x[0], ref.MX),
           lambda: bn.bitnet_fp4_dequant(w, s, 300, ref.MX)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    for dtype in (torch.float32,):  # types that the C entry refuses
        with pytest.raises(bn.BitnetError):
            bn.bitnet_fp4_linear(x, w, s, ref.MX, dtype=dtype)
    with pytest.raises(bn.BitnetError):  # rows that overlap
        bn.bitnet_fp4_quant(x[:1].expand(4, 256), ref.MX)
    with pytest.raises(bn.BitnetError):  # 17 tokens need a workspace
        bn.bitnet_fp4_linear(torch.zeros(17, 256, dtype=torch.bfloat16, device="cuda"), w, s, ref.MX,
                             ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_offsets_beyond_32_bits():
    """Codes of 4.5 GB, an activation matrix of 2.2 and a product of 2.8 thousand million elements: their last rows."""
    fmt, gen = ref.NV, torch.Generator(device="cuda").manual_seed(1)
    N, K = 70000, 131072
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.randint(52, 60, (bn.bitnet_fp4_scale_bytes(N, K, fmt),), dtype=torch.uint8, device="cuda", generator=gen)
    last = N // 128 * 128
    wv = bn.bitnet_fp4_dequant(w[last:], s[bn.bitnet_fp4_scale_bytes(last, K, fmt):], K, fmt, dtype=torch.float32).double()
    gw = torch.tensor([2.0 ** -12], device="cuda")
    for M in (1, 70):
        x = torch.randn(M, K, device="cuda", generator=gen)
        a, a_s = bn.bitnet_fp4_quant(x, fmt)
        av = bn.bitnet_fp4_dequant(a, a_s, K, fmt, dtype=torch.float32).double()
        y = bn.bitnet_fp4_gemm(a, a_s, w, s, K, fmt, gw=gw)[:, last:].double()
        want, mag = av @ wv.t() * 2.0 ** -12, av.abs() @ wv.abs().t() * 2.0 ** -12
        assert bool(((y - want).abs() <= want.abs() * 2.0 ** -8 + mag * (K / 16 + 16) * 2.0 ** -22).all())
    del w, s, wv
    rows, K = 33000, 65600
    x = torch.randn(rows, K, device="cuda", generator=gen).to(torch.bfloat16)
    codes, scales = bn.bitnet_fp4_quant(x, fmt)
    c, sb = ref.quantise(x[-8:].float().cpu().numpy(), fmt)
    p, _ = ref.pack(c, sb, fmt)
    got = codes[-8:].cpu().numpy()
    assert np.array_equal(got & 0x77, p & 0x77)
    y = bn.bitnet_fp4_dequant(codes, scales, K, fmt)
    assert np.array_equal(y[-8:].float().cpu().numpy(),
                          torch.from_numpy(ref.values(c, sb, fmt)[:, :K]).to(torch.bfloat16).float().numpy())
    del x, codes, scales, y
    M, N, K = 70000, 40000, 128
    a, a_s = bn.bitnet_fp4_quant(torch.randn(M, K, device="cuda", generator=gen), fmt)
    w, w_s = bn.bitnet_fp4_quant(torch.randn(N, K, device="cuda", generator=gen), fmt)
    y = bn.bitnet_fp4_gemm(a, a_s, w, w_s, K, fmt)
    av = bn.bitnet_fp4_dequant(a, a_s, K, fmt, dtype=torch.float32).double()
    wv = bn.bitnet_fp4_dequant(w, w_s, K, fmt, dtype=torch.float32).double()
    want, mag = av[-40:] @ wv.t(), av[-40:].abs() @ wv.abs().t()
    assert bool(((y[-40:].double() - want).abs() <= want.abs() * 2.0 ** -8 + mag * (K / 16 + 16) * 2.0 ** -22).all())
