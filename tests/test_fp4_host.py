"""The 4-bit floating point entry points without a GPU: sizes, refusals, and
the reference that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import fp4_ref as ref
import ternary_weight_bit_w2a8_b200 as bn


@pytest.fixture(scope="module")
def lib():
    from ternary_weight_bit_w2a8_b200 import build
    build.build()
    return bn.lib()


A = ctypes.c_void_p(0x10000)
WS = ctypes.c_void_p(0x20000)
MIS1 = ctypes.c_void_p(0x10001)
MIS8 = ctypes.c_void_p(0x10008)
NULL = None
S = None
INV, ALIGN, WSERR, OK = bn.BITNET_ERR_INVALID_ARG, bn.BITNET_ERR_ALIGNMENT, bn.BITNET_ERR_WORKSPACE, bn.BITNET_OK


def test_sizes(lib):
    for rows, K in [(1, 1), (1, 128), (3, 129), (128, 2560), (129, 2560), (1000, 6912)]:
        Kp = ref.pad_up(K, 128)
        assert bn.bitnet_fp4_code_bytes(rows, K) == rows * Kp // 2
        for fmt in (ref.MX, ref.NV):
            assert bn.bitnet_fp4_scale_bytes(rows, K, fmt) == ref.pad_up(rows, 128) * Kp // ref.BLOCK[fmt]
            ws = bn.bitnet_fp4_workspace_bytes(rows, 64, K, fmt)
            assert bn.bitnet_fp4_workspace_bytes(16, 64, K, fmt) == 0
            if rows > 16:  # the linear layer's codes and scales
                assert ws >= rows * Kp // 2 + ref.pad_up(rows, 128) * Kp // ref.BLOCK[fmt]
            assert ws == bn.bitnet_fp4_workspace_bytes(rows, 64, K, fmt)
    assert bn.bitnet_fp4_code_bytes(0, 64) == 0 and bn.bitnet_fp4_scale_bytes(5, 0, ref.MX) == 0
    assert lib.bitnet_fp4_code_bytes(-1, 4) == -1
    assert lib.bitnet_fp4_code_bytes(1, (1 << 21) + 1) == -1
    assert lib.bitnet_fp4_scale_bytes(4, 4, 2) == -1
    assert lib.bitnet_fp4_workspace_bytes(4, -4, 4, 0) == -1


# Fake pointers: every call fails a check on the host before any device work,
# and none is made where a GPU is present.
@pytest.fixture
def no_gpu(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake-pointer host checks run only where no GPU is present")
    return lib


def test_quant_refusals(no_gpu):
    f = no_gpu.bitnet_fp4_quant
    ok = [A, 0, 4, 64, 64, 0, NULL, A, A, S]

    def call(**change):
        a = list(ok)
        for k, v in change.items():
            a[["x", "dt", "rows", "K", "ld", "fmt", "g", "codes", "scales"].index(k)] = v
        return f(*a)
    assert call(dt=3) == INV and call(dt=-1) == INV and call(fmt=2) == INV
    assert call(rows=-1) == INV and call(K=(1 << 21) + 1, ld=1 << 22) == INV and call(ld=63) == INV
    assert call(x=NULL) == INV and call(codes=NULL) == INV and call(scales=NULL) == INV
    assert call(x=MIS1) == ALIGN and call(codes=MIS8) == ALIGN and call(scales=MIS8) == ALIGN and call(g=MIS1) == ALIGN
    assert call(rows=0, x=NULL, codes=NULL, scales=NULL) == OK
    assert call(K=0, x=NULL, codes=NULL, scales=NULL) == OK
    assert call() == bn.BITNET_ERR_CUDA


def test_dequant_refusals(no_gpu):
    f = no_gpu.bitnet_fp4_dequant
    assert f(A, A, 4, 64, 0, NULL, A, 3, 64, S) == INV
    assert f(A, A, 4, 64, 5, NULL, A, 0, 64, S) == INV
    assert f(A, A, 4, 64, 0, NULL, A, 0, 63, S) == INV
    assert f(A, A, 4, 64, 0, NULL, NULL, 0, 64, S) == INV
    assert f(MIS8, A, 4, 64, 0, NULL, A, 0, 64, S) == ALIGN
    assert f(A, A, 4, 64, 0, NULL, MIS1, 0, 64, S) == ALIGN
    assert f(NULL, NULL, 0, 64, 0, NULL, NULL, 0, 64, S) == OK


def test_tensor_scale_refusals(no_gpu):
    f = no_gpu.bitnet_fp4_tensor_scale
    assert f(A, 0, 4, 64, 64, NULL, S) == INV
    assert f(A, 7, 4, 64, 64, A, S) == INV
    assert f(A, 0, 4, 64, 60, A, S) == INV
    assert f(NULL, 0, 4, 64, 64, A, S) == INV
    assert f(MIS1, 0, 4, 64, 64, A, S) == ALIGN
    assert f(A, 0, 4, 64, 64, MIS1, S) == ALIGN


def test_product_refusals(no_gpu):
    f = no_gpu.bitnet_fp4_gemm
    names = ["a", "sa", "ga", "w", "sw", "gw", "fmt", "y", "dt", "M", "N", "K", "ldy"]
    ok = [A, A, NULL, A, A, NULL, 0, A, 0, 3, 8, 64, 8]

    def call(**change):
        a = list(ok)
        for k, v in change.items():
            a[names.index(k)] = v
        return f(*a, S)
    assert call(fmt=2) == INV and call(dt=2) == INV and call(dt=9) == INV
    assert call(M=-1) == INV and call(K=1 << 22) == INV and call(ldy=7) == INV
    assert call(a=NULL) == INV and call(sw=NULL) == INV and call(y=NULL) == INV
    assert call(a=MIS8) == ALIGN and call(sa=MIS8) == ALIGN and call(w=MIS8) == ALIGN and call(sw=MIS8) == ALIGN
    assert call(y=MIS1) == ALIGN and call(ga=MIS1) == ALIGN
    assert call(M=0, a=NULL, sa=NULL, y=NULL) == OK and call(N=0, ldy=0, y=NULL) == OK
    assert call() == bn.BITNET_ERR_CUDA


def test_linear_refusals(no_gpu):
    f = no_gpu.bitnet_fp4_linear
    names = ["x", "xdt", "ldx", "ga", "w", "sw", "gw", "fmt", "y", "ydt", "M", "N", "K", "ldy", "ws", "wsb"]
    M, N, K = 200, 8, 1000
    need = bn.bitnet_fp4_workspace_bytes(M, N, K, 1)
    ok = [A, 0, K, NULL, A, A, NULL, 1, A, 0, M, N, K, N, WS, need]

    def call(**change):
        a = list(ok)
        for k, v in change.items():
            a[names.index(k)] = v
        return f(*a, S)
    assert call(fmt=2) == INV and call(ydt=2) == INV and call(xdt=3) == INV and call(ldx=K - 1) == INV
    assert call(x=NULL) == INV and call(w=NULL) == INV and call(y=NULL) == INV
    assert call(w=MIS8) == ALIGN and call(x=MIS1) == ALIGN and call(y=MIS1) == ALIGN
    assert call(ws=NULL, wsb=0) == WSERR and call(wsb=64) == WSERR and call(ws=MIS8) == ALIGN
    assert call(M=0, x=NULL, y=NULL) == OK


def test_binding_refusals():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (bn.bitnet_fp4_tensor_scale, lambda t: bn.bitnet_fp4_quant(t, bn.BITNET_FP4_MX)):
        with pytest.raises(ValueError):
            f(x)  # not a CUDA tensor


# ------------------------------------------------------------------ the reference
def test_reference_rounding():
    v = np.array([0.25, 0.2500001, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 100])
    assert ref.GRID[ref.nearest_even(v, ref.GRID)].tolist() == [0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6]
    assert ref.E4M3[126] == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[56] == 1.0


def test_reference_blocks():
    x = np.zeros((2, 40), dtype=np.float32)
    x[0, :3] = [7, -3.5, 1]       # MX: top 7 -> scale 1, 7 saturates at 6, 3.5 ties to 4
    x[1, 32] = np.nan
    c, sb = ref.quantise(x, ref.MX)
    assert c[0, :4].tolist() == [7, 14, 2, 0] and sb[0].tolist() == [127, 0, 0, 0]
    assert sb[1].tolist() == [0, 255, 0, 0] and not c[1].any()
    p, t = ref.pack(c, sb, ref.MX)
    assert p.shape == (2, 64) and p[0, 0] == 7 | (14 << 4) and t.size == 512
    assert t[0] == 127 and t[16 + 1] == 255
    c, sb = ref.quantise(x[:1], ref.NV)   # 7 / 6 = 1.1667 -> e4m3 1.125
    assert ref.E4M3[sb[0, 0]] == 1.125 and c[0, :3].tolist() == [7, 13, 2]
