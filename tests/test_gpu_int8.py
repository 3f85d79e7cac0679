"""The 8-bit integer Linear against exact integer sums.

int8_linear: acc is exact; fp32(acc), times xs, and one fma with ws and the
bias round three times, so |y - ref| <= (2^-24 + 2^-24 + 2^-24)(1 + 2^-22)
|acc xs ws| + 2^-24 |b| in fp32, plus 2^-8 |ref| (1 + 2^-8) for bf16 output.
w8a8_linear's codes and scales are those of quantize_ex, bit for bit, so its
result is int8_linear's on them, bit for bit."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def wlq():
    import weight_only_quantized_rtn_b200 as m
    return m


def make(seed, M, N, K, bias=True, full=False):
    g = torch.Generator().manual_seed(seed)
    lo, hi = (-128, 128) if full else (-127, 128)
    xq = torch.randint(lo, hi, (M, K), generator=g, dtype=torch.int8)
    wq = torch.randint(lo, hi, (N, K), generator=g, dtype=torch.int8)
    xs, ws = torch.rand(M, generator=g) * 0.02 + 1e-4, torch.rand(N, generator=g) * 0.001 + 1e-5
    b = torch.randn(N, generator=g).bfloat16() if bias else None
    return xq, xs, wq, ws, b


def reference(xq, xs, wq, ws, b):
    """(exact y, the part without the bias) in fp64: the integer sums are below 2^53."""
    acc = (xq.cuda().double() @ wq.cuda().double().t()).cpu().numpy()
    p = acc * xs.double().numpy()[:, None] * ws.double().numpy()
    return (p if b is None else p + b.double().numpy()), p


def check(y, want, p, b):
    got = y.double().cpu().numpy()
    tol = 3 * 2.0 ** -24 * (1 + 2.0 ** -22) * np.abs(p) + (0 if b is None else 2.0 ** -24 * np.abs(b.double().numpy()))
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(want)
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%d wrong, first at %r: got %r want %r" % (bad.sum(), np.argwhere(bad)[0], got[bad][0], want[bad][0])


SHAPES = [
    (1, 8, 16), (1, 256, 256), (3, 129, 48), (16, 4096, 4096), (17, 320, 144), (48, 1000, 512), (64, 512, 4096), (100, 384, 1040),
    (128, 4096, 1024), (129, 136, 272), (200, 20000, 128), (256, 4096, 512), (300, 2056, 640), (1560, 4096, 256), (257, 16384, 384),
    (1000, 5000, 208), (2049, 2048, 128),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_int8_linear(M, N, K, dtype):
    m = wlq()
    for bias in (True, False):
        xq, xs, wq, ws, b = make(M + N + K, M, N, K, bias, full=not bias)
        want, p = reference(xq, xs, wq, ws, b)
        y = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
        m.int8_linear_into(y, xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), bias=None if b is None else b.cuda())
        m.check_status()
        check(y, want, p, b)


def test_sums_of_the_largest_codes_do_not_overflow():
    m = wlq()
    K = 131056
    for M, N in ((2, 8), (300, 9000)):
        xq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        wq = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        one = torch.ones(max(M, N), device="cuda")
        y = torch.empty((M, N), device="cuda")
        m.int8_linear_into(y, xq, one[:M], wq, one[:N])
        m.check_status()
        assert (y == 128 * 128 * K).all()  # 31 bits, a multiple of 2^14: exact in fp32


@pytest.mark.parametrize("M,K", [(1, 16), (5, 2048), (16, 4096), (33, 4112), (700, 8192), (40, 16384), (9, 32768), (3, 40000)])
def test_w8a8_has_the_bits_of_quantize_then_int8_linear(M, K):
    m = wlq()
    N = 264
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))).bfloat16().cuda()
    if M > 3:
        x[1] = 0            # an all-zero token
        x[2] *= 1e-38       # a subnormal scale
        x[3] = torch.arange(K).bfloat16().cuda() % 128 - 63.5  # halves
    _, _, wq, ws, b = make(1, 1, N, K)
    wq, ws, b = wq.cuda(), ws.cuda(), b.cuda()
    codes, scales = m.quantize_ex(x, 8, 0)
    want = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    m.int8_linear_into(want, codes, scales.reshape(-1), wq, ws, bias=b)
    y = m.w8a8_linear(x, wq, ws, bias=b)
    m.check_status()
    assert torch.equal(y, want)
    ws_ = torch.full((m.w8a8_workspace(M, K),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(m.w8a8_linear(x, wq, ws, bias=b, workspace=ws_), want)
    assert ws_[: M * K].view(torch.int8).reshape(M, K).equal(codes)


def test_the_layers_own_chain():
    """quantize -> w8a8 against the 64-bit Linear of the dequantised operands."""
    m = wlq()
    M, N, K = 70, 512, 1024
    g = torch.Generator().manual_seed(1)
    W, x = torch.randn(N, K, generator=g) * 0.02, torch.randn(M, K, generator=g).bfloat16()
    wq, ws = m.quantize(W.cuda(), 8, 0)
    y = m.w8a8_linear(x.cuda(), wq, ws.reshape(-1), out_dtype=torch.float32)
    xs = (x.double().abs().amax(1) / 127).float().double()
    xq = torch.round(x.double() / xs[:, None])
    want = (xq @ wq.cpu().double().t()) * xs[:, None] * ws.cpu().double().reshape(-1)
    check(y, want.numpy(), want.numpy(), None)


def test_non_finite_tokens_are_flagged():
    m = wlq()
    x = torch.randn(4, 64).bfloat16().cuda()
    x[2, 5] = float("inf")
    _, _, wq, ws, b = make(1, 1, 16, 64)
    y = m.w8a8_linear(x, wq.cuda(), ws.cuda(), bias=b.cuda())
    assert m.get_status() == m.ERR_NONFINITE
    assert torch.equal(y[2], b.cuda())
    m.check_status()


def test_unaligned_output_and_streams_and_graphs():
    m = wlq()
    for M, N, K in ((20, 130, 256), (600, 4100, 256)):  # rows of y that are not whole 16 bytes
        xq, xs, wq, ws, b = make(7, M, N, K)
        want, p = reference(xq, xs, wq, ws, b)
        buf = torch.full((M * N + 4,), float("nan"), device="cuda")
        y = buf[1:1 + M * N].view(M, N)
        a = [t.cuda() for t in (xq, xs, wq, ws)]
        m.int8_linear_into(y, *a, bias=b.cuda())
        check(y, want, p, b)
        assert torch.isnan(buf[0]) and torch.isnan(buf[1 + M * N:]).all()
    x = torch.randn(300, 512).bfloat16().cuda()
    _, _, wq, ws, b = [t if t is None else t.cuda() for t in make(3, 1, 1024, 512)]
    want = m.w8a8_linear(x, wq, ws)
    torch.cuda.synchronize()
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            outs.append(m.w8a8_linear(x, wq, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = m.w8a8_linear(x, wq, ws)
    x.copy_(x.flip(0))
    graph.replay()
    assert torch.equal(o, want.flip(0))
