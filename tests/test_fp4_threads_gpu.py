"""The 4-bit calls from several threads at once: each launch is made without the interpreter lock."""
import threading

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
    yield
    torch.cuda.synchronize()
    assert bn.bitnet_get_device_error() == 0


# few tokens, quantised in the launch and before it; the kernel for more; a reused workspace
SHAPES = [(1, 700, 2560), (12, 1300, 640), (40, 900, 1500), (200, 1000, 700)]


@pytest.mark.parametrize("own_streams", [False, True])
def test_layers_from_many_threads(own_streams):
    """Eight threads, each with its own weights, workspace and inputs, on one stream or on one each: the bits of the
    same calls one by one, and refusals raised in the thread that made them."""
    gen = torch.Generator().manual_seed(5)
    work = []
    for i in range(8):
        M, N, K = SHAPES[i % len(SHAPES)]
        fmt = (bn.BITNET_FP4_MX, bn.BITNET_FP4_NV)[i // len(SHAPES)]
        W, x = (torch.randn(r, K, generator=gen).cuda() for r in (N, M))
        gw = bn.bitnet_fp4_tensor_scale(W)
        w, ws = bn.bitnet_fp4_quant(W, fmt, g=gw)
        ga = bn.bitnet_fp4_tensor_scale(x)
        space = torch.empty(max(256, bn.bitnet_fp4_workspace_bytes(M, N, K, fmt)), dtype=torch.uint8, device="cuda")
        want = bn.bitnet_fp4_linear(x, w, ws, fmt, ga=ga, gw=gw)
        back = bn.bitnet_fp4_dequant(w, ws, K, fmt, g=gw)
        work.append((W, x, w, ws, fmt, K, gw, space, want, back))
    torch.cuda.synchronize()
    outs, failures = [[] for _ in work], []
    start = threading.Barrier(len(work))

    def run(i):
        W, x, w, ws, fmt, K, gw, space, want, back = work[i]
        stream = torch.cuda.Stream() if own_streams else torch.cuda.current_stream()
        try:
            with torch.cuda.stream(stream):
                start.wait(timeout=60)
                for rep in range(25):
                    g = bn.bitnet_fp4_tensor_scale(W)
                    c, s = bn.bitnet_fp4_quant(W, fmt, g=g)
                    ga = bn.bitnet_fp4_tensor_scale(x)
                    y = bn.bitnet_fp4_linear(x, c, s, fmt, ga=ga, gw=g, ws=space if rep % 2 else None)
                    outs[i].append((y, bn.bitnet_fp4_dequant(c, s, K, fmt, g=g)))
                    with pytest.raises(ValueError):
                        bn.bitnet_fp4_linear(x, c, s[:-1], fmt)
            stream.synchronize()
        except BaseException as e:  # noqa: BLE001 (handed to the test's own thread)
            failures.append((i, e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not failures, failures[0]
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        assert len(got) == 25
        assert all(torch.equal(y, work[i][8]) and torch.equal(b, work[i][9]) for y, b in got), i
