"""GPU parity of the INT8 layers against their definitions in 64 bits.

Quantizer: codes and scales are the exact quotient's and one FP32 division, so
they are compared for equality.  Products: the integer sum is exact, so with
p = |sum sA sB|, y = sum sA sB + bias and u the half step of the output type
(2^-8 bf16, 2^-11 fp16):
  FP32 steps: RN(sum) and its product with sA are off by 2^-24 each, the FMA
  with sB and bias by 2^-24 of its result: at most 2^-24 (3 p + |y|);
  the output's rounding adds u (|y| + that), or half of fp16's smallest
  subnormal step, 2^-25.
"""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from block_scaled_fp4_05_b200 import fp4
from test_int8_abi import bounds_wanted

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
KERNELS = [fp4.GEMM_PREFILL, fp4.GEMM_DECODE, fp4.GEMM_AUTO]


@pytest.fixture(autouse=True)
def status_is_clean():
    yield
    torch.cuda.synchronize()
    assert fp4.fp4_get_device_status() == 0


# ---------------------------------------------------------------------------
# Quantizer
# ---------------------------------------------------------------------------
def quantize_definition(x):
    """Codes and scales of finite rows, from numpy in 64 bits."""
    v = x.double().cpu().numpy()
    amax = np.abs(v).max(1) if v.shape[1] else np.zeros(v.shape[0])
    safe = np.where(amax == 0, 1.0, amax)
    codes = np.rint(127.0 * v / safe[:, None])
    scales = np.where(amax == 0, np.float32(1), amax.astype(np.float32) / np.float32(127))
    return codes.astype(np.int8), scales.astype(np.float32)


def check_quantized(x, codes, scales, what=""):
    want_codes, want_scales = quantize_definition(x)
    assert np.array_equal(scales.cpu().numpy(), want_scales), what
    got = codes.cpu().numpy()
    bad = np.argwhere(got != want_codes)
    assert bad.size == 0, "%s: %d codes differ, first %s: %s for %s" % (
        what, len(bad), bad[0], got[tuple(bad[0])], want_codes[tuple(bad[0])])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (9, 8), (5, 255), (17, 256), (9, 257), (7, 513), (6, 1000),
                                       (9, 1025), (2, 2048), (3, 2049), (2, 4096), (3, 4099), (1, 8192), (2, 8193),
                                       (2, 16384), (2, 16391), (1, 32768), (2, 32771), (300, 64), (0, 64), (3, 0)])
def test_quantize_shapes(dtype, rows, cols):
    g = torch.Generator().manual_seed(rows * 1000 + cols)
    x = (torch.randn(rows, cols + 40, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))).to(dtype).cuda()
    x = x[:, : (cols + 40) // 8 * 8].contiguous()
    v = x[:, 8:8 + cols]                       # a strided view: what is beside it may not matter
    x[:, :8] = float("nan")
    x[:, 8 + cols:] = float("inf")
    whole = torch.full((rows + 2, (cols + 15) // 16 * 16 + 16), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((rows + 2,), -5.0, device="cuda")
    fp4.fp4_quantize_int8(v, whole[1:rows + 1, :cols], scales[1:rows + 1])
    check_quantized(v, whole[1:rows + 1, :cols], scales[1:rows + 1], (rows, cols))
    whole[1:rows + 1, :cols] = 77              # nothing else was written
    assert (whole == 77).all() and scales[0] == -5 and scales[-1] == -5


@pytest.mark.parametrize("dtype", [BF, HF])
def test_quantize_every_quotient_of_mantissas(dtype):
    # rows: every mantissa of the maximum; columns: every mantissa of x at
    # nine exponents.  Ties and their neighbours are all among them.
    bits, one = (7, 0x3F80) if dtype == BF else (10, 0x3C00)
    n = 1 << bits
    amax = torch.arange(one, one + n, dtype=torch.int16).view(dtype)
    xs = torch.cat([torch.arange(one - e * n, one - e * n + n, dtype=torch.int16).view(dtype) for e in range(9)])
    x = xs[None, :].repeat(n, 1)
    x = torch.where(x.float() <= amax[:, None].float(), x, -amax[:, None])
    x = torch.cat([amax[:, None], x, torch.zeros(n, 7, dtype=dtype)], 1).cuda()
    codes, scales = fp4.quantize_int8(x)
    check_quantized(x, codes, scales)
    assert (codes[:, 0] == 127).all()


def test_quantize_extreme_rows():
    # subnormal, smallest, largest and mixed magnitudes
    tiny = torch.tensor([2.0 ** -133, 2.0 ** -126, 2.0 ** -118, 2.0 ** -100, 3.0 * 2.0 ** -132])
    big = torch.tensor([3.3895314e38, 2.0 ** 127, 1.5 * 2.0 ** 120])
    rows = [torch.linspace(-1, 1, 64) * v for v in list(tiny) + list(big)]
    rows += [torch.cat([torch.full((32,), float(tiny[0])), torch.full((32,), float(big[0]))])]
    x = torch.stack(rows).to(BF).cuda()
    codes, scales = fp4.quantize_int8(x)
    check_quantized(x, codes, scales, "bf16")
    y = torch.stack([torch.linspace(-1, 1, 64) * v for v in (65504.0, 2.0 ** -24, 2.0 ** -14, 6e-8)]).to(HF).cuda()
    check_quantized(y, *fp4.quantize_int8(y), what="fp16")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("cols", [40, 256, 3001, 4096])
def test_quantize_zero_and_non_finite_rows(dtype, cols):
    x = torch.randn(6, cols, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[1] = 0
    x[2, cols - 1] = float("inf")
    x[3, 0] = float("-inf")
    x[4, cols // 2] = float("nan")
    x[5] = -0.0
    x = torch.nn.functional.pad(x, (0, -cols % 8)).cuda()[:, :cols]
    codes, scales = fp4.quantize_int8(x)
    keep = [0, 1, 5]
    check_quantized(x[keep], codes[keep], scales[keep])
    assert torch.isnan(scales[2:5]).all() and (codes[2:5] == 0).all()
    assert scales[1] == 1 and scales[5] == 1
    w = torch.randint(-127, 128, (16, cols), dtype=torch.int8)
    w = torch.nn.functional.pad(w, (0, -cols % 16)).cuda()[:, :cols]
    for kernel in KERNELS:                     # such a token's outputs are NaN, the others' are not
        d = fp4.gemm_int8(codes, scales, w, torch.ones(16, device="cuda"), kernel=kernel)
        assert torch.isnan(d[2:5].float()).all() and torch.isfinite(d[[0, 1, 5]].float()).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("cols", [64, 256, 1001, 4096, 5000])
def test_quantize_gathers_rows(dtype, cols):
    x = torch.randn(10, (cols + 7) // 8 * 8, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()[:, :cols]
    index = torch.tensor([3, 3, 9, 0, 3, 5, 0, 9, 1, 2, 4, 6, 7, 8, 3, 3, 3], dtype=torch.int32, device="cuda")
    codes, scales = fp4.quantize_int8(x, index)
    check_quantized(x[index.long()], codes, scales)
    index[::3] = torch.tensor([-1, 10, 2 ** 31 - 1, -2 ** 31, 11, -7], dtype=torch.int32, device="cuda")
    codes, scales = fp4.quantize_int8(x, index)
    assert (codes[::3] == 0).all() and (scales[::3] == 1).all()
    kept = torch.ones(17, dtype=torch.bool)
    kept[::3] = False
    check_quantized(x[index[kept.cuda()].long()], codes[kept.cuda()], scales[kept.cuda()])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("cols", [2049, 2600, 4090, 4096])
def test_quantize_gathers_many_rows(dtype, cols):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(400, (cols + 7) // 8 * 8, generator=g).to(dtype).cuda()[:, :cols]
    x[17], x[18, cols - 1], x[19, 1] = 0, float("inf"), float("nan")
    index = torch.randint(0, 400, (3101,), generator=g, dtype=torch.int32).cuda()
    index[:6] = torch.tensor([17, 18, 19, -1, 400, 2 ** 31 - 1], dtype=torch.int32)
    codes, scales = fp4.quantize_int8(x, index)
    assert (codes[:6] == 0).all()
    assert scales[0] == 1 and torch.isnan(scales[1:3]).all() and (scales[3:6] == 1).all()
    kept = ((index >= 0) & (index < 400) & (index != 18) & (index != 19)).nonzero()[:, 0]
    check_quantized(x[index[kept].long()], codes[kept], scales[kept])


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------
def random_codes(g, rows, cols, pad=16):
    """Codes whose rows end inside 77s."""
    w = torch.full((rows, (cols + 15) // 16 * 16 + pad), 77, dtype=torch.int8)
    w[:, :cols] = torch.randint(-128, 128, (rows, cols), generator=g, dtype=torch.int8)
    return w.cuda()[:, :cols]


def check_product(d, a, sa, b, sb, bias, what=""):
    p = (a.double() @ b.double().T) * sa.double()[:, None] * sb.double()[None, :]
    y = p if bias is None else p + bias.double()
    u = torch.finfo(d.dtype).eps / 2
    e32 = 2.0 ** -24 * (3 * p.abs() + y.abs())
    tol = u * y.abs() + (1 + u) * e32 + (2.0 ** -25 if d.dtype == HF else 0.0)
    off = (d.double() - y).abs()
    bad = torch.nonzero(~(off <= tol))
    assert bad.numel() == 0, "%s: %d of %d outside, first %s: %r for %r" % (
        what, len(bad), d.numel(), bad[0].tolist(), d[tuple(bad[0])].item(), y[tuple(bad[0])].item())


def operands(M, N, K, seed, bias, experts=None):
    g = torch.Generator().manual_seed(seed)
    a, sa = random_codes(g, M, K), (torch.rand(M, generator=g) * 2e-3 + 1e-4).cuda()
    n = N * (experts or 1)
    b, sb = random_codes(g, n, K, pad=32), (torch.rand(n, generator=g) * 2e-3 + 1e-4).cuda()
    c = torch.randn(n, generator=g).cuda() if bias else None
    return a, sa, b, sb, c


DENSE = [(1, 1, 1), (1, 8, 16), (3, 7, 5), (2, 130, 31), (16, 128, 128), (17, 130, 129), (33, 257, 300), (64, 200, 1024),
         (65, 264, 640), (129, 513, 1000), (256, 256, 128), (257, 520, 2051), (700, 1030, 384), (1, 4096, 4096),
         (5, 1000, 1151), (16, 4104, 1024), (100, 2048, 2048)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("MNK", DENSE)
def test_dense_shapes(dtype, MNK):
    M, N, K = MNK
    a, sa, b, sb, bias = operands(M, N, K, 7 + M, bias=M % 2 == 1)
    seen = []
    for kernel in KERNELS + [fp4.GEMM_AUTO | fp4.GEMM_B_STATIC, fp4.GEMM_DECODE | fp4.GEMM_B_STATIC]:
        whole = torch.full((M + 2, (N + 7) // 8 * 8 + 8), 3.0, dtype=dtype, device="cuda")
        d = whole[1:M + 1, :N]
        fp4.fp4_gemm_int8(a, sa, b, sb, d, bias, kernel)
        check_product(d, a, sa, b, sb, bias, (MNK, kernel))
        seen.append(d.clone())
        whole[1:M + 1, :N] = 3.0
        assert (whole == 3.0).all(), "wrote outside D"
    assert all(torch.equal(s, seen[0]) for s in seen)


# several tiles a CTA pair at either tile width, the grouped raster (A above
# 64 MB), all token tiles of the other kernel, large M on it
@pytest.mark.parametrize("MNK,kernel", [((2048, 5120, 512), fp4.GEMM_PREFILL), ((1024, 4600, 256), fp4.GEMM_PREFILL),
                                        ((8450, 300, 8192), fp4.GEMM_PREFILL), ((600, 1000, 512), fp4.GEMM_DECODE),
                                        ((16, 28672, 1024), fp4.GEMM_DECODE), ((128, 19000, 500), fp4.GEMM_DECODE),
                                        ((300, 40000, 256), fp4.GEMM_AUTO)])
def test_dense_many_tiles(MNK, kernel):
    M, N, K = MNK
    a, sa, b, sb, bias = operands(M, N, K, 3, bias=True)
    d = fp4.gemm_int8(a, sa, b, sb, bias, kernel=kernel)
    check_product(d, a, sa, b, sb, bias, MNK)


@pytest.mark.parametrize("kernel", KERNELS)
def test_dense_largest_sums(kernel):
    K = 131071                                  # 128 * 128 * K = 2^31 - 16384
    a = torch.full((2, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    b = torch.full((9, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    b[1] = 127
    sa, sb = torch.full((2,), 2.0 ** -20, device="cuda"), torch.ones(9, device="cuda")
    d = fp4.gemm_int8(a, sa, b, sb, kernel=kernel)
    y = torch.full((2, 9), 16384.0 * K * 2.0 ** -20, dtype=torch.float64, device="cuda")
    y[:, 1] = -128.0 * 127 * K * 2.0 ** -20
    assert ((d.double() - y).abs() <= (2.0 ** -8 + 2.0 ** -22) * y.abs()).all()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("bias", [False, True])
def test_dense_empty_sums(kernel, bias):
    a, b = torch.empty(5, 0, dtype=torch.int8, device="cuda"), torch.empty(9, 0, dtype=torch.int8, device="cuda")
    c = torch.arange(9, dtype=torch.float32, device="cuda") if bias else None
    d = fp4.gemm_int8(a, torch.ones(5, device="cuda"), b, torch.ones(9, device="cuda"), c, kernel=kernel)
    assert torch.equal(d.float(), c.expand(5, 9) if bias else torch.zeros(5, 9, device="cuda"))
    for M, N in ((0, 9), (5, 0), (0, 0)):
        fp4.gemm_int8(torch.zeros(M, 16, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"),
                      torch.zeros(N, 16, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"), kernel=kernel)


# ---------------------------------------------------------------------------
# By expert
# ---------------------------------------------------------------------------
def check_grouped(offsets, T, N, K, dtype, kernel, bias, seed=5, static=False):
    E = len(offsets) - 1
    a, sa, b, sb, c = operands(T, N, K, seed, bias, experts=E)
    b, sb, c = b.unflatten(0, (E, N)), sb.view(E, N), c.view(E, N) if bias else None
    whole = torch.full((T + 2, (N + 7) // 8 * 8 + 8), 3.0, dtype=dtype, device="cuda")
    d = whole[1:T + 1, :N]
    fp4.fp4_gemm_int8_grouped(a, sa, b, sb, torch.tensor(offsets, dtype=torch.int32, device="cuda"), d, c,
                              kernel | (fp4.GEMM_B_STATIC if static else 0))
    for e, (lo, hi) in enumerate(bounds_wanted(offsets, T)):
        if lo < hi:
            check_product(d[lo:hi], a[lo:hi], sa[lo:hi], b[e], sb[e], c[e] if bias else None, (e, lo, hi, kernel))
            d[lo:hi] = 3.0
    assert (whole == 3.0).all(), "wrote outside the groups"


def ends(*counts, first=0):
    return [first] + (first + np.cumsum(counts)).tolist()


GROUPS = [
    (ends(16), 16, 128, 128), (ends(0, 0, 1, 0), 1, 40, 64), (ends(0), 4, 40, 64),
    (ends(3, 0, 20, 1, 0, 9), 40, 264, 300),                          # rows behind the last group
    (ends(5, 1, 2, first=7), 20, 136, 1000),                          # rows before the first
    (ends(255, 0, 256, 257, 1, 31), 800, 520, 257),
    (ends(300, 2, 140, 0, 0, 33, 65, 1), 541, 1000, 512),
    (ends(*([1] * 33)), 33, 72, 96), (ends(*([0, 7] * 40)), 280, 130, 160),
    (ends(*([2, 0, 1, 5] * 128)), 1024, 24, 48),                      # 512 experts
    (ends(900, 1500, 20), 2420, 5003, 130),                           # several tiles a CTA pair
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped(case, kernel, dtype):
    offsets, T, N, K = GROUPS[case]
    check_grouped(offsets, T, N, K, dtype, kernel, bias=case % 2 == 0, static=case % 3 == 0)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("offsets", [[0, 30, 10, 50], [-5, 20, 400, 100], [90, 40, 40, 100], [2 ** 31 - 1, 0, 5, -2 ** 31],
                                     [0, 0, 0, 0], [100, 100, 100, 100], [-1, -2 ** 31, 7, 2 ** 31 - 1]])
def test_grouped_offsets_out_of_order_or_range(kernel, offsets):
    check_grouped(offsets, 100, 72, 160, BF, kernel, bias=True)


@pytest.mark.parametrize("kernel", KERNELS)
def test_grouped_weights_with_gaps_between_experts(kernel):
    g = torch.Generator().manual_seed(9)
    E, N, K, T = 3, 50, 70, 30
    store = torch.randint(-128, 128, (E, N + 5, 96), generator=g, dtype=torch.int8).cuda()
    b = store[:, 2:2 + N, 16:16 + K]
    a, sa, sb = random_codes(g, T, K), torch.rand(T, generator=g).cuda(), torch.rand(E, N, generator=g).cuda()
    d = fp4.gemm_int8_grouped(a, sa, b, sb, torch.tensor([0, 11, 11, 30], dtype=torch.int32, device="cuda"), kernel=kernel)
    check_product(d[:11], a[:11], sa[:11], b[0], sb[0], None)
    check_product(d[11:], a[11:], sa[11:], b[2], sb[2], None)


@pytest.mark.parametrize("kernel", KERNELS)
def test_grouped_empty_sums_and_no_rows(kernel):
    b = torch.empty(2, 9, 0, dtype=torch.int8, device="cuda")
    c = torch.arange(18, dtype=torch.float32, device="cuda").view(2, 9)
    off = torch.tensor([1, 3, 4], dtype=torch.int32, device="cuda")
    d = torch.full((6, 16), 7.0, dtype=BF, device="cuda")
    fp4.fp4_gemm_int8_grouped(torch.empty(6, 0, dtype=torch.int8, device="cuda"), torch.ones(6, device="cuda"), b,
                              torch.ones(2, 9, device="cuda"), off, d[:, :9], c, kernel)
    want = torch.full((6, 16), 7.0, device="cuda")
    want[1:3, :9], want[3, :9] = c[0], c[1]
    assert torch.equal(d.float(), want)
    fp4.gemm_int8_grouped(torch.empty(0, 16, dtype=torch.int8, device="cuda"), torch.ones(0, device="cuda"),
                          torch.zeros(2, 9, 16, dtype=torch.int8, device="cuda"), torch.ones(2, 9, device="cuda"), off,
                          kernel=kernel)


# ---------------------------------------------------------------------------
# Together, on streams and in graphs
# ---------------------------------------------------------------------------
def weights(g, experts, N, K):
    w = (torch.randn(experts * N, K, generator=g) * 0.02).to(BF).cuda()
    codes, scales = fp4.quantize_int8(w)
    check_quantized(w, codes, scales)
    return codes.unflatten(0, (experts, N)), scales.view(experts, N)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M", [1, 9, 40, 300])
def test_linear(dtype, M):
    g = torch.Generator().manual_seed(11)
    N, K = 392, 840
    w, sw = weights(g, 1, N, K)
    x, bias = torch.randn(M, K, generator=g).to(dtype).cuda(), torch.randn(N, generator=g).cuda()
    y = fp4.linear_int8(x, w[0], sw[0], bias)
    codes, scales = fp4.quantize_int8(x)
    check_quantized(x, codes, scales)
    check_product(y, codes, scales, w[0], sw[0], bias)
    # against the product that was never quantized: each code is off by at most half a step of its row
    exact = x.double() @ (w[0].double() * sw[0].double()[:, None]).T + bias.double()
    step = 0.5 * scales.double()[:, None] * (w[0].double().abs() * sw[0].double()[:, None]).sum(1)[None, :]
    u = torch.finfo(dtype).eps / 2
    assert ((y.double() - exact).abs() <= step * 1.01 + 1.01 * u * (exact.abs() + step) + 2.0 ** -20).all()


def moe(x, index, off, up, sup, down, sdown):
    a, sa = fp4.quantize_int8(x, index)
    h = fp4.gemm_int8_grouped(a, sa, up, sup, off, kernel=fp4.GEMM_AUTO | fp4.GEMM_B_STATIC)
    b, sb = fp4.quantize_int8(h)
    return a, sa, h, b, sb, fp4.gemm_int8_grouped(b, sb, down, sdown, off, kernel=fp4.GEMM_AUTO | fp4.GEMM_B_STATIC)


def check_moe(x, index, off, up, sup, down, sdown, got):
    a, sa, h, b, sb, y = got
    check_quantized(x[index.long()], a, sa)
    check_quantized(h, b, sb)
    o = off.tolist()
    for e in range(len(o) - 1):
        s = slice(o[e], o[e + 1])
        if o[e] < o[e + 1]:
            check_product(h[s], a[s], sa[s], up[e], sup[e], None)
            check_product(y[s], b[s], sb[s], down[e], sdown[e], None)


def routing(g, tokens, experts):
    """Two experts a token: source rows in the experts' order, and the group bounds."""
    picks = torch.stack([torch.randperm(experts, generator=g)[:2] for _ in range(tokens)]).flatten()
    order = torch.argsort(picks, stable=True)
    counts = torch.bincount(picks, minlength=experts)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    return (order // 2).to(torch.int32).cuda(), off.to(torch.int32).cuda()


@pytest.mark.parametrize("tokens", [1, 30, 700])
def test_expert_layer_and_its_graph(tokens):
    g = torch.Generator().manual_seed(12)
    E, H, F = 6, 256, 328
    up, sup = weights(g, E, F, H)
    down, sdown = weights(g, E, H, F)
    x = torch.randn(tokens, H, generator=g).to(BF).cuda()
    index, off = routing(g, tokens, E)
    check_moe(x, index, off, up, sup, down, sdown, moe(x, index, off, up, sup, down, sdown))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe(x, index, off, up, sup, down, sdown)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moe(x, index, off, up, sup, down, sdown)
    for _ in range(3):                          # other tokens, other routing, the same graph
        x.copy_(torch.randn(tokens, H, generator=g).to(BF))
        i2, o2 = routing(g, tokens, E)
        index.copy_(i2)
        off.copy_(o2)
        graph.replay()
        torch.cuda.synchronize()
        check_moe(x, index, off, up, sup, down, sdown, got)


def test_two_streams_at_once():
    g = torch.Generator().manual_seed(13)
    runs = []
    for i, (M, N, K) in enumerate([(16, 6000, 2048), (16, 6000, 2048), (600, 1500, 512), (600, 1500, 512)]):
        a, sa, b, sb, _ = operands(M, N, K, 20 + i, False)
        runs.append((a, sa, b, sb, torch.empty(M, (N + 7) // 8 * 8, dtype=BF, device="cuda")[:, :N], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, sa, b, sb, d, s in runs:
            fp4.fp4_gemm_int8(a, sa, b, sb, d, stream=s)
    torch.cuda.synchronize()
    for a, sa, b, sb, d, _ in runs:
        check_product(d, a, sa, b, sb, None)


def test_threads_with_streams_of_their_own():
    g = torch.Generator().manual_seed(17)
    jobs = []
    for M, N, K in [(1, 300, 504), (20, 2056, 1496), (200, 900, 2048), (700, 600, 328)]:
        w, sw = weights(g, 1, N, K)
        x = torch.randn(M, (K + 7) // 8 * 8, generator=g).to(BF).cuda()[:, :K]
        jobs.append((x, w[0], sw[0], fp4.linear_int8(x, w[0], sw[0]), torch.cuda.Stream()))
    torch.cuda.synchronize()
    wrong = []

    def work(x, w, sw, want, stream):
        try:
            for i in range(40):   # the stream as an object and as its handle
                y = fp4.linear_int8(x, w, sw, stream=stream if i % 2 else stream.cuda_stream)
                stream.synchronize()
                if not torch.equal(y, want):
                    wrong.append((tuple(x.shape), i))
        except Exception as e:   # (an assertion of a thread is not seen by the test)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=job) for job in jobs * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_chain_without_waits():
    # each product's output is the next one's input, nothing waits in between
    g = torch.Generator().manual_seed(14)
    w, sw = weights(g, 1, 512, 512)
    x = torch.randn(20, 512, generator=g).to(BF).cuda()
    want = x
    for _ in range(12):
        want = fp4.linear_int8(want, w[0], sw[0])
        want = (want.float() * 2.2).to(BF)
        torch.cuda.synchronize()
    for _ in range(5):
        y = x
        for _ in range(12):
            y = fp4.linear_int8(y, w[0], sw[0])
            y = (y.float() * 2.2).to(BF)
        assert torch.equal(y, want)


@pytest.mark.parametrize("M,N,K", [(16, 1024, 65536), (1, 400, 40000), (600, 1024, 65536)])
def test_linear_right_after_its_weight_is_quantized(M, N, K):
    # the weight's quantizer still runs when the layer is called, and the
    # weight's memory holds another weight's codes until then
    g = torch.Generator().manual_seed(16)
    ws = [torch.randn(N, K, generator=g).to(BF).cuda() for _ in range(2)]
    x = torch.randn(M, K, generator=g).to(BF).cuda()
    want = []
    for w in ws:
        q = fp4.quantize_int8(w)
        torch.cuda.synchronize()
        want.append(fp4.linear_int8(x, *q))
        torch.cuda.synchronize()
    codes, scales = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    for i in range(10):
        fp4.fp4_quantize_int8(ws[i % 2], codes, scales)
        assert torch.equal(fp4.linear_int8(x, codes, scales), want[i % 2])


def test_bound_calls():
    a, sa, b, sb, bias = operands(20, 100, 200, 15, True)
    d = torch.zeros(20, 104, dtype=BF, device="cuda")[:, :100]
    fp4.bind_gemm_int8(a, sa, b, sb, d, bias)()
    check_product(d, a, sa, b, sb, bias)
    d.zero_()
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    fp4.bind_gemm_int8_grouped(a, sa, b[None], sb[None], off, d, bias[None])()
    check_product(d, a, sa, b, sb, bias)
    x = torch.randn(4, 96, device="cuda").to(BF)
    codes, scales = torch.empty(4, 96, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    fp4.bind_quantize_int8(x, codes, scales)()
    check_quantized(x, codes, scales)


def test_binding_refusals():
    a, sa, b, sb, bias = operands(4, 16, 64, 16, True)
    d = torch.zeros(4, 16, dtype=BF, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    bad = [
        lambda: fp4.fp4_gemm_int8(a, sa, b[:, :32], sb, d), lambda: fp4.fp4_gemm_int8(a.short(), sa, b, sb, d),
        lambda: fp4.fp4_gemm_int8(a, sa, b, sb, d.float()), lambda: fp4.fp4_gemm_int8(a, sa.double(), b, sb, d),
        lambda: fp4.fp4_gemm_int8(a, sa[:3], b, sb, d), lambda: fp4.fp4_gemm_int8(a, sa, b, sb, d, bias[:8]),
        lambda: fp4.fp4_gemm_int8(a, sa, b, sb, d.T), lambda: fp4.fp4_gemm_int8(a.cpu(), sa, b, sb, d),
        lambda: fp4.fp4_gemm_int8(a, sa, b, sb, torch.zeros(4, 20, dtype=BF, device="cuda")[:, :16]),   # ldd % 8
        lambda: fp4.fp4_gemm_int8_grouped(a, sa, b, sb, off, d),
        lambda: fp4.fp4_gemm_int8_grouped(a, sa, b[None], sb[None], off.long(), d),
        lambda: fp4.fp4_gemm_int8_grouped(a, sa, b[None], sb[None], off[:1], d),
        lambda: fp4.fp4_gemm_int8_grouped(a, sa, b[None].expand(2, 16, 64), sb[None].repeat(2, 1), off[[0, 0, 1]], d),
        lambda: fp4.quantize_int8(x.float()), lambda: fp4.quantize_int8(x, off.long()),
        lambda: fp4.fp4_quantize_int8(x, torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), sa),
        lambda: fp4.fp4_quantize_int8(x, torch.zeros(5, 64, dtype=torch.int8, device="cuda"), torch.zeros(5, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, fp4.Fp4Error)):
            call()
            pytest.fail("call %d was accepted" % i)
    assert (d == 0).all()


def test_offsets_past_32_bits():
    # three rows (or experts) that lie more than 2^31 elements apart
    far = 2 ** 31 + 64
    g = torch.Generator().manual_seed(17)
    x = torch.empty(3, far, dtype=BF, device="cuda")[:, :520]
    x.copy_(torch.randn(3, 520, generator=g).to(BF))
    store = torch.empty(3, far, dtype=torch.int8, device="cuda")
    codes, scales = store[:, :520], torch.empty(3, device="cuda")
    fp4.fp4_quantize_int8(x, codes, scales)
    check_quantized(x, codes, scales)
    gathered, gs = fp4.quantize_int8(x, torch.tensor([2, 0, 2, 1], dtype=torch.int32, device="cuda"))
    check_quantized(x[[2, 0, 2, 1]], gathered, gs)
    del x
    b, sb = random_codes(g, 40, 520), torch.rand(40, generator=g).cuda()
    d = torch.empty(3, far, dtype=BF, device="cuda")[:, :40]
    for kernel in KERNELS:
        d.zero_()
        fp4.fp4_gemm_int8(codes, scales, b, sb, d, kernel=kernel)                  # far rows of A and D
        check_product(d, codes, scales, b, sb, None)
        y = fp4.gemm_int8(b, sb, codes, scales, kernel=kernel)                     # far rows of B
        check_product(y, b, sb, codes, scales, None)
    experts = store.as_strided((3, 5, 96), (far, 96, 1))
    experts.copy_(torch.randint(-128, 128, (3, 5, 96), generator=g, dtype=torch.int8))
    a, sa, se = random_codes(g, 9, 96), torch.rand(9, generator=g).cuda(), torch.rand(3, 5, generator=g).cuda()
    off = torch.tensor([0, 2, 5, 9], dtype=torch.int32, device="cuda")
    for kernel in KERNELS:
        y = fp4.gemm_int8_grouped(a, sa, experts, se, off, kernel=kernel)
        for e, (lo, hi) in enumerate(((0, 2), (2, 5), (5, 9))):
            check_product(y[lo:hi], a[lo:hi], sa[lo:hi], experts[e], se[e], None)


@pytest.mark.parametrize("kernel", KERNELS)
def test_expert_stride_is_no_multiple_of_the_rows(kernel):
    g = torch.Generator().manual_seed(18)
    store = torch.randint(-128, 128, (4000,), generator=g, dtype=torch.int8).cuda()
    b = store[16:].as_strided((4, 11, 20), (11 * 48 + 16, 48, 1), store.storage_offset() + 16)
    a, sa, sb = random_codes(g, 14, 20), torch.rand(14, generator=g).cuda(), torch.rand(4, 11, generator=g).cuda()
    y = fp4.gemm_int8_grouped(a, sa, b, sb, torch.tensor([0, 3, 7, 8, 14], dtype=torch.int32, device="cuda"), kernel=kernel)
    for e, (lo, hi) in enumerate(((0, 3), (3, 7), (7, 8), (8, 14))):
        check_product(y[lo:hi], a[lo:hi], sa[lo:hi], b[e], sb[e], None)


FIRST_CALL = """
import sys
import threading
sys.path.insert(0, %r)
import torch
from block_scaled_fp4_05_b200 import fp4
x = torch.randn(%d, 256, device="cuda").bfloat16()
w = torch.randint(-127, 128, (300, 256), dtype=torch.int8, device="cuda")
sw = torch.rand(300, device="cuda")
off = torch.tensor([0, %d], dtype=torch.int32, device="cuda")
d, e = (torch.zeros(%d, 304, dtype=torch.bfloat16, device="cuda")[:, :300] for _ in range(2))
codes, scales = torch.empty(%d, 256, dtype=torch.int8, device="cuda"), torch.empty(%d, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    fp4.fp4_quantize_int8(x, codes, scales)
    fp4.fp4_gemm_int8(codes, scales, w, sw, d)
    fp4.fp4_gemm_int8_grouped(codes, scales, w[None], sw[None], off, e)
graph.replay()
torch.cuda.synchronize()
y = (codes.double() @ w.double().T * scales.double()[:, None] * sw.double()).float()
assert torch.equal(d, e) and ((d.float() - y).abs() <= (2.0 ** -8 + 2.0 ** -20) * y.abs() + 1e-6).all()
assert fp4.fp4_get_device_status() == 0
"""


@pytest.mark.parametrize("M", [9, 600])
def test_first_calls_of_a_process_are_captured(M):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL % (root, M, M, M, M, M)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ---------------------------------------------------------------------------
# Drawn sizes, by the forms that the choice takes for them
# ---------------------------------------------------------------------------
def drawn(seed, lo, hi):
    return int(round(np.exp(np.random.default_rng(seed).uniform(np.log(lo), np.log(hi)))))


@pytest.mark.parametrize("seed", range(24))
def test_dense_drawn(seed):
    M, N, K = drawn(3 * seed, 1, 1500), drawn(3 * seed + 1, 1, 3000), drawn(3 * seed + 2, 1, 3000)
    a, sa, b, sb, bias = operands(M, N, K, seed, bias=seed % 2 == 0)
    dtype = (BF, HF)[seed % 3 == 0]
    got = [fp4.gemm_int8(a, sa, b, sb, bias, out_dtype=dtype, kernel=k) for k in KERNELS]
    check_product(got[0], a, sa, b, sb, bias, (M, N, K))
    assert all(torch.equal(g, got[0]) for g in got)


@pytest.mark.parametrize("seed", range(24))
def test_grouped_drawn(seed):
    rng = np.random.default_rng(1000 + seed)
    E, rows, skew = int(rng.choice([1, 2, 5, 8, 31, 32, 33, 64, 100])), drawn(seed, 1, 2500), rng.choice([0.0, 1.0, 3.0])
    N, K = drawn(500 + seed, 1, 900 if E > 8 else 2500), drawn(700 + seed, 1, 900)
    p = np.exp(skew * rng.standard_normal(E))
    counts = np.bincount(rng.choice(E, rows, p=p / p.sum()), minlength=E)
    first, tail = int(rng.integers(0, 3)), int(rng.choice([0, 0, 7, 300]))
    for kernel in KERNELS:
        check_grouped(ends(*counts.tolist(), first=first), first + rows + tail, N, K, (BF, HF)[seed % 2], kernel,
                      bias=seed % 3 == 0, seed=seed)


@pytest.mark.parametrize("kernel", KERNELS)
def test_grouped_captured_once_serves_any_routing(kernel):
    # the tile lists are formed when the graph runs: from no rows to all of them in one expert
    T, E, N, K = 700, 9, 300, 200
    a, sa, b, sb, _ = operands(T, N, K, 21, False, experts=E)
    b, sb = b.unflatten(0, (E, N)), sb.view(E, N)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    d = torch.zeros(T, 304, dtype=BF, device="cuda")[:, :N]
    fp4.fp4_gemm_int8_grouped(a, sa, b, sb, off, d, kernel=kernel)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp4.fp4_gemm_int8_grouped(a, sa, b, sb, off, d, kernel=kernel)
    for o in ([0] * 10, [0] + [700] * 9, [0] * 9 + [700], ends(100, 0, 1, 255, 33, 0, 3, 200, 108), ends(*([1] * 9))):
        off.copy_(torch.tensor(o, dtype=torch.int32))
        d.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        for e in range(E):
            if o[e] < o[e + 1]:
                s = slice(o[e], o[e + 1])
                check_product(d[s], a[s], sa[s], b[e], sb[e], None, (o, e))
                d[s] = 5.0
        assert (d == 5.0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 15), (5, 16), (31, 17), (7, 511), (130, 512), (130, 513), (1000, 1536),
                                 (33, 8191), (4, 40960), (9000, 70), (4097, 2049)])
def test_few_tokens_small_weights(dtype, M, N, K):
    # dot products and tensor cores on both sides of the choice between them
    a, sa, b, sb, bias = operands(M, N, K, 31 * M + N, bias=N % 2 == 0)
    b_end = torch.randint(-128, 128, (N, K), generator=torch.Generator().manual_seed(N), dtype=torch.int8).cuda()
    ld = (K + 15) // 16 * 16
    tight = torch.empty((N - 1) * ld + K, dtype=torch.int8, device="cuda").as_strided((N, K), (ld, 1))   # ends with its last code
    tight.copy_(b_end)
    for w in (b, tight):
        got = []
        for kernel in KERNELS + [fp4.GEMM_AUTO | fp4.GEMM_B_STATIC]:
            whole = torch.full((M + 2, (N + 7) // 8 * 8 + 8), 3.0, dtype=dtype, device="cuda")
            d = whole[1:M + 1, :N]
            fp4.fp4_gemm_int8(a, sa, w, sb, d, bias, kernel)
            got.append(d.clone())
            d.fill_(3.0)
            assert (whole == 3.0).all()
        check_product(got[0], a, sa, w, sb, bias, (M, N, K))
        assert all(torch.equal(g, got[0]) for g in got)


# ---------------------------------------------------------------------------
# Operands that the call right before writes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M", [1, 4, 8, 20])
def test_product_right_after_its_weight_is_rewritten(M):
    # no B_STATIC: the weight's quantizer may be the kernel before, and the
    # weight's memory has been read with other codes in it by the call before that
    g = torch.Generator().manual_seed(40 + M)
    N, K = 480, 2000
    ws = [torch.randn(N, K, generator=g).to(BF).cuda() for _ in range(2)]
    a, sa = random_codes(g, M, K), torch.rand(M, generator=g).cuda()
    want = []
    for w in ws:
        q = fp4.quantize_int8(w)
        torch.cuda.synchronize()
        want.append(fp4.gemm_int8(a, sa, *q))
        check_product(want[-1], a, sa, *q, None)
        torch.cuda.synchronize()
    codes, scales = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    got = []
    for i in range(60):
        fp4.fp4_quantize_int8(ws[i % 2], codes, scales)
        got.append(fp4.gemm_int8(a, sa, codes, scales))
    torch.cuda.synchronize()
    assert all(torch.equal(d, want[i % 2]) for i, d in enumerate(got))


@pytest.mark.parametrize("M,N", [(1, 1000), (8, 4096), (300, 2056)])
def test_quantizer_right_after_its_input_is_rewritten(M, N):
    g = torch.Generator().manual_seed(50 + M)
    K = 512
    b, sb = random_codes(g, N, K), torch.rand(N, generator=g).cuda()
    inputs = [(random_codes(g, M, K), torch.rand(M, generator=g).cuda()) for _ in range(2)]
    want = []
    for a, sa in inputs:
        d = fp4.gemm_int8(a, sa, b, sb)
        torch.cuda.synchronize()
        want.append(fp4.quantize_int8(d))
        check_quantized(d, *want[-1])
    d = torch.zeros(M, (N + 7) // 8 * 8, dtype=BF, device="cuda")[:, :N]
    got = []
    for i in range(60):
        fp4.fp4_gemm_int8(*inputs[i % 2], b, sb, d)
        got.append(fp4.quantize_int8(d))
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[i % 2][0]) and torch.equal(g[1], want[i % 2][1]) for i, g in enumerate(got))


@pytest.mark.parametrize("experts", [0, 40])
def test_few_token_launches_of_several_turns_right_behind_each_other(experts):
    # more tiles than clusters run at once, each launch's weights written by the call before it
    g = torch.Generator().manual_seed(60 + experts)
    M, K = 48, 640
    N = 2056 if experts else 60000
    a, sa = random_codes(g, M, K), torch.rand(M, generator=g).cuda()
    ws = [torch.randn((experts or 1) * N, K, generator=g).to(BF).cuda() for _ in range(2)]
    off = torch.tensor(np.linspace(0, M, experts + 1).astype(int), dtype=torch.int32, device="cuda") if experts else None
    codes, scales = torch.empty_like(ws[0], dtype=torch.int8), torch.empty(len(ws[0]), device="cuda")

    def product():
        if experts:
            return fp4.gemm_int8_grouped(a, sa, codes.unflatten(0, (experts, N)), scales.view(experts, N), off,
                                         kernel=fp4.GEMM_DECODE)
        return fp4.gemm_int8(a, sa, codes, scales, kernel=fp4.GEMM_DECODE)

    want = []
    for w in ws:
        fp4.fp4_quantize_int8(w, codes, scales)
        torch.cuda.synchronize()
        d = product()
        for e in range(experts or 1):
            rows = slice(*off[e:e + 2].tolist()) if experts else slice(None)
            check_product(d[rows], a[rows], sa[rows], codes[e * N:(e + 1) * N], scales[e * N:(e + 1) * N], None)
        want.append(d)
    got = []
    for i in range(12):
        fp4.fp4_quantize_int8(ws[i % 2], codes, scales)
        got += [product(), product()]
    torch.cuda.synchronize()
    assert all(torch.equal(d, want[i // 2 % 2]) for i, d in enumerate(got))


# ---------------------------------------------------------------------------
# Every form that the choice can take: tile widths and splits by name
# ---------------------------------------------------------------------------
PAIR = [(fp4.GEMM_PREFILL, bt, 1) for bt in range(32, 257, 32)]
FEW = [(fp4.GEMM_DECODE, nt, split) for nt in (16, 32, 64, 128) for split in (1, 2, 4, 8)]


def cta_pairs():
    return torch.cuda.get_device_properties(0).multi_processor_count // 2


def dense_by_form(form, M, N, K, dtype, seed, static=False, want=None):
    kernel, tile, split = form
    a, sa, b, sb, bias = operands(M, N, K, seed, True)
    whole = torch.full((M + 2, (N + 7) // 8 * 8 + 8), 3.0, dtype=dtype, device="cuda")
    d = whole[1:M + 1, :N]
    fp4.fp4_selftest_gemm_int8(kernel | (fp4.GEMM_B_STATIC if static else 0), tile, split, a, sa, b, sb, d, bias=bias)
    got = d.clone()
    check_product(got, a, sa, b, sb, bias, (form, M, N, K))
    assert torch.equal(got, fp4.gemm_int8(a, sa, b, sb, bias, out_dtype=dtype)), "other bits than the form that is chosen"
    d.fill_(3.0)
    assert (whole == 3.0).all(), "wrote outside D"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("form", PAIR, ids=str)
def test_pair_form(form, dtype):
    bt, pairs = form[1], cta_pairs()
    # a remainder of tokens and channels, less than a wave, K longer than the ring
    dense_by_form(form, bt + bt // 2 + 5, 300, 2500, dtype, bt)
    dense_by_form(form, bt - 3, 264, 130, dtype, bt + 1, static=True)
    # a wave and a few tiles more, which are computed as halves; the last token tile is narrow
    dense_by_form(form, 3 * bt + bt // 2 + 3, (pairs // 4 + 2) * 256 - 20, 420, dtype, bt + 2)
    # whole tiles only, a last wave too long for halves
    dense_by_form(form, 4 * bt, ((pairs + pairs // 2) // 4 + 1) * 256, 384, dtype, bt + 3, static=True)
    # several tiles a pair, a short K: both accumulators in turn
    dense_by_form(form, 5 * bt + 1, (pairs // 2) * 256 + 8, 100, dtype, bt + 4)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("form", FEW, ids=str)
def test_few_token_form(form, dtype):
    nt, split = form[1:]
    dense_by_form(form, 2 * nt + nt // 2 + 1, 434, 1300, dtype, nt + split)                # a CTA's shares of K differ
    dense_by_form(form, nt, 130, 128 * split - 5, dtype, nt + split + 1, static=True)      # one stage a CTA
    dense_by_form(form, nt - 3, 384, 128 * 13 * split + 40, dtype, nt + split + 2)         # more stages than the ring has
    # more tiles than run at once, so clusters take them in turn
    dense_by_form(form, 3 * nt - 1, 25650, 1050, dtype, nt + split + 3, static=True)


def grouped_by_form(form, counts, N, K, dtype, seed, first=0, tail=0):
    kernel, tile, split = form
    offsets = ends(*counts, first=first)
    E, T = len(counts), offsets[-1] + tail
    a, sa, b, sb, c = operands(T, N, K, seed, True, experts=E)
    b, sb, c = b.unflatten(0, (E, N)), sb.view(E, N), c.view(E, N)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    whole = torch.full((T + 2, (N + 7) // 8 * 8 + 8), 3.0, dtype=dtype, device="cuda")
    d, other = whole[1:T + 1, :N], torch.full((T, (N + 7) // 8 * 8), 3.0, dtype=dtype, device="cuda")[:, :N]
    fp4.fp4_selftest_gemm_int8(kernel, tile, split, a, sa, b, sb, d, off, c)
    fp4.fp4_gemm_int8_grouped(a, sa, b, sb, off, other, c)
    assert torch.equal(d, other), "other bits than the form that is chosen"
    for e in range(E):
        lo, hi = offsets[e:e + 2]
        if lo < hi:
            check_product(d[lo:hi], a[lo:hi], sa[lo:hi], b[e], sb[e], c[e], (form, e, lo, hi))
            d[lo:hi] = 3.0
    assert (whole == 3.0).all(), "wrote outside the groups"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("form", PAIR, ids=str)
def test_pair_form_by_expert(form, dtype):
    bt, pairs = form[1], cta_pairs()
    grouped_by_form(form, [bt - 1, 0, bt, bt + 1, 1, 33, 0, 2 * bt + 31], 520, 330, dtype, bt, first=3, tail=40)
    # eight token tiles of a wave and a bit: the last ones as halves, some of them narrow
    grouped_by_form(form, [3 * bt - 31, 40, 3 * bt + 1], (pairs // 8 + 1) * 256 - 20, 300, dtype, bt + 1)
    grouped_by_form(form, [7] * 70 + [0] * 20 + [bt // 2 + 1] * 9, 264, 1700, dtype, bt + 2)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("form", FEW, ids=str)
def test_few_token_form_by_expert(form, dtype):
    nt, split = form[1:]
    grouped_by_form(form, [nt - 1, 0, nt, nt + 1, 1, 3, 0, 2 * nt + 5], 520, 1300, dtype, nt + split, first=3, tail=40)
    grouped_by_form(form, [3] * 50 + [0] * 20 + [nt // 2 + 1] * 9 + [0], 1300, 1034, dtype, nt + split + 1)


# ---------------------------------------------------------------------------
# A wait that gives up
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("both", [False, True])
def test_a_timeout_of_an_int8_kernel_is_reported_and_cleared(both):
    assert fp4.fp4_get_device_status() == 0
    fp4.fp4_selftest_bounded_wait_int8()
    if both:
        fp4.fp4_selftest_bounded_wait()
    assert fp4.fp4_get_device_status() == 5          # FP4_ERR_TIMEOUT, then cleared
    assert fp4.fp4_get_device_status() == 0
    a, sa, b, sb, bias = operands(300, 520, 640, 70, True)
    check_product(fp4.gemm_int8(a, sa, b, sb, bias), a, sa, b, sb, bias)   # the context is usable


# ---------------------------------------------------------------------------
# Tensors as they come: widths and views whose rows are not aligned
# ---------------------------------------------------------------------------
def as_they_come(g, dtype):
    yield from (torch.randn(r, c, generator=g).to(dtype).cuda() for r, c in
                [(5, 1), (3, 7), (1, 61), (40, 1001), (2, 4099), (3, 33001), (2, 12)])
    x = torch.randn(9, 640, generator=g).to(dtype).cuda()
    yield from (x[:, 1:], x[:, 3:500], x[1:, 4:12], x[::2, 7:8])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_quantize_tensors_as_they_come(dtype):
    g = torch.Generator().manual_seed(71)
    side = torch.cuda.Stream()
    for x in as_they_come(g, dtype):
        check_quantized(x, *fp4.quantize_int8(x), what=tuple(x.shape))
        index = torch.randint(0, len(x), (13,), generator=g, dtype=torch.int32).cuda()
        codes, scales = fp4.quantize_int8(x, index)
        check_quantized(x[index.long()], codes, scales, tuple(x.shape))
        torch.cuda.synchronize()
        codes, scales = fp4.quantize_int8(x, stream=side)
        side.synchronize()
        check_quantized(x, codes, scales, tuple(x.shape))
    for x in (torch.empty(0, 7, dtype=dtype, device="cuda"), torch.empty(3, 0, dtype=dtype, device="cuda")):
        codes, scales = fp4.quantize_int8(x)
        assert codes.shape == x.shape and (scales == 1).all()


def test_linear_of_an_odd_width_and_its_graph():
    g = torch.Generator().manual_seed(72)
    N, K = 391, 1003
    w, bias = (torch.randn(N, K, generator=g) * 0.02).to(BF).cuda(), torch.randn(N, generator=g).cuda()
    W, sW = fp4.quantize_int8(w)
    check_quantized(w, W, sW)
    for M in (1, 9, 130):
        x = torch.randn(M, K, generator=g).to(BF).cuda()
        fp4.linear_int8(x, W, sW, bias)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = fp4.linear_int8(x, W, sW, bias)
        for _ in range(2):
            x.copy_(torch.randn(M, K, generator=g).to(BF))
            graph.replay()
            codes, scales = fp4.quantize_int8(x)
            check_product(y, codes, scales, W, sW, bias)


def test_calls_into_given_memory_say_what_is_misaligned():
    x = torch.zeros(4, 61, dtype=BF, device="cuda")
    codes, scales = torch.zeros(4, 64, dtype=torch.int8, device="cuda")[:, :61], torch.zeros(4, device="cuda")
    for call in (lambda: fp4.fp4_quantize_int8(x, codes, scales),
                 lambda: fp4.gemm_int8(codes.contiguous(), scales, codes, scales),
                 lambda: fp4.gemm_int8_grouped(codes.contiguous(), scales, codes[None], scales[None],
                                               torch.tensor([0, 4], dtype=torch.int32, device="cuda"))):
        with pytest.raises(fp4.Fp4Error, match="multiples of 16 bytes") as e:
            call()
        assert e.value.status == 3
    with pytest.raises(fp4.Fp4Error):                # no other error is taken for that one
        fp4.quantize_int8(torch.zeros(1, 64, dtype=BF, device="cuda").expand(4, 64))


# ---------------------------------------------------------------------------
# FP32's range between the scales
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M,N,K", [(4, 40, 200), (40, 136, 200), (300, 264, 200)])
def test_products_of_huge_and_tiny_tokens(M, N, K):
    # 127^2 K = 3225800 = 2^21.62: times 2^106 it fits FP32, times 2^107 it does not
    a, b = torch.full((M, K + 8), 127, dtype=torch.int8, device="cuda")[:, :K], torch.full((N, K + 8), 127, dtype=torch.int8,
                                                                                         device="cuda")[:, :K]
    sums = 127.0 * 127 * K
    sa, sb = torch.full((M,), 2.0 ** 106, device="cuda"), torch.full((N,), 2.0 ** -100, device="cuda")
    sa[1::4], sa[2::4], sa[3::4] = 2.0 ** 107, 2.0 ** -126, 2.0 ** -149    # (2^-149: the smallest there is)
    sb[1::2] = 2.0 ** 100
    seen = []
    for kernel in KERNELS:
        d = fp4.gemm_int8(a, sa, b, sb, kernel=kernel).double()
        # exact in FP32 where they fit: only the output's rounding, or its range
        fits = (sums * sa.double()) < 2.0 ** 128
        want = sums * sa.double()[:, None] * sb.double()[None, :]
        assert torch.isinf(d[~fits]).all() and (d[~fits] > 0).all()
        inside = fits[:, None] & (want < 3.3895e38) & (want >= 2.0 ** -126)
        off = (d - want).abs()
        assert (off[inside] <= 2.0 ** -8 * want[inside]).all()
        small = fits[:, None] & (want < 2.0 ** -126)
        assert (off[small] <= 2.0 ** -134 + 2.0 ** -150).all()             # half a step of BF16's subnormals, and of FP32's
        assert torch.isinf(d[fits[:, None] & (want > 3.4e38)]).all()
        seen.append(d)
    assert all(torch.equal(d, seen[0]) for d in seen)


# ---------------------------------------------------------------------------
# Beside the FP4 GEMM
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", [fp4.NVFP4, fp4.MXFP4])
@pytest.mark.parametrize("split", [2, 8])
def test_clusters_beside_the_fp4_pair_gemm_on_another_stream(fmt, split):
    # clusters of one stage's work each, and CTA pairs that take all tensor memory
    g = torch.Generator().manual_seed(73)
    M, N, K = 20, 1000, 128 * split - 24
    a, sa, b, sb, bias = operands(M, N, K, 74, True)
    d = torch.zeros(M, 1000, dtype=BF, device="cuda")
    R, KF = 512, 1024
    codes = [torch.randint(0, 256, (R, KF // 2), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    one = 127 if fmt == fp4.MXFP4 else 0x38                   # 1.0 in E8M0 and in E4M3
    scales = [torch.full((fp4.fp4_scale_bytes(fmt, R, KF),), one, dtype=torch.uint8, device="cuda") for _ in range(2)]
    alpha = torch.ones(1, device="cuda") if fmt == fp4.NVFP4 else None
    outs = [torch.zeros(R, R, dtype=BF, device="cuda") for _ in range(2)]
    fp4.gemm(fmt, codes[0], scales[0], codes[1], scales[1], KF, alpha, fp4.GEMM_PREFILL, outs[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(200):
        fp4.gemm(fmt, codes[0], scales[0], codes[1], scales[1], KF, alpha, fp4.GEMM_PREFILL, outs[1], stream=streams[0])
        fp4.fp4_selftest_gemm_int8(fp4.GEMM_DECODE, 16, split, a, sa, b, sb, d, bias=bias, stream=streams[1])
    torch.cuda.synchronize()
    check_product(d, a, sa, b, sb, bias)
    assert torch.equal(outs[0], outs[1])


def test_kernel_numbers_that_leave_32_bits_are_refused():
    a, sa, b, sb, _ = operands(4, 16, 64, 75, False)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for kernel in (1 << 32, (1 << 32) | fp4.GEMM_DECODE, -(1 << 32), 1 << 70, -1):
        with pytest.raises((ValueError, OverflowError, fp4.Fp4Error)):
            fp4.gemm_int8(a, sa, b, sb, kernel=kernel)
        with pytest.raises((ValueError, OverflowError, fp4.Fp4Error)):
            fp4.gemm_int8_grouped(a, sa, b[None], sb[None], off, kernel=kernel)
