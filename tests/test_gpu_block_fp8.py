"""The e4m3 product with a scale per block of 128 against plain forms (needs a GB300): codes and
scales bit for bit, products against 64-bit sums of the same codes."""
import numpy as np
import pytest
import torch

from block_cases import (F32, check, half_ulp, product_reference, quantized_matrices, quantized_rows)

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def out_bound(ref, mag, K, dtype):
    """Block sums of 128 products and KB scaled additions, each rounded to fp32 (twice the half ulp:
    the tensor cores' sums may truncate)."""
    return half_ulp(dtype) * ref.abs() + 2 * (128 + -(-K // 128) + 4) * F32 * mag


def rows(M, K, seed, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[::7] *= 30.0
    if M > 2:
        x[1] = 0.0
        x[2, :: 3] = 0.0
    return x.to(dtype)


@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 144), (33, 2048), (9, 4112), (257, 640)])
def test_row_codes_are_exact(cuda_lib, M, K):
    x = rows(M, K, M * K)
    codes, scales = cuda_lib.quantize_rows_block_fp8(x.cuda())
    rc, rs = quantized_rows(x.float().numpy())
    assert np.array_equal(codes.cpu().numpy(), rc)
    KB = rs.shape[1]
    got = scales.cpu().numpy()
    assert np.array_equal(got[:, :KB], rs) and not got[:, KB:].any()


def test_rows_with_ties_infinities_and_nan(cuda_lib):
    x = torch.zeros(6, 256)
    x[0, :8] = torch.tensor([448.0, 17.0, 18.0, 19.0, 25.0, 26.0, -27.0, 2.0 ** -10])   # midpoints of e4m3 steps
    x[1, 5] = float("inf")
    x[1, 6] = 500.0
    x[2, 130] = float("nan")
    x[2, 131] = -1e30
    x[3] = 2.0 ** -133                                                               # subnormal in fp32
    x[4, 0] = 3.3e38
    x[5, 255] = -3.0e-39
    x = x.bfloat16()
    codes, scales = cuda_lib.quantize_rows_block_fp8(x.cuda())
    rc, rs = quantized_rows(x.float().numpy())
    assert np.array_equal(codes.cpu().numpy() & 0x7f, rc & 0x7f)                      # a NaN's sign is open
    keep = (rc & 0x7f) != 0x7f
    assert np.array_equal(codes.cpu().numpy()[keep], rc[keep])
    assert np.array_equal(scales.cpu().numpy()[:, :2], rs)


@pytest.mark.parametrize("G,N,K,dtype", [(1, 128, 128, FP), (2, 200, 144, BF), (3, 64, 400, FP), (1, 7, 16, FP)])
def test_matrix_codes_and_transpose_are_exact(cuda_lib, G, N, K, dtype):
    g = torch.Generator().manual_seed(N + K)
    w = (torch.randn(G, N, K, generator=g) * 0.02).to(dtype)
    w[0, : min(N, 128), : min(K, 128)] = 0.0
    q = cuda_lib.quantize_block_fp8(w.cuda())
    rc, rs = quantized_matrices(w.float().numpy())
    assert np.array_equal(q.codes.cpu().numpy(), rc) and np.array_equal(q.scales.cpu().numpy(), rs)
    if N % 16 == 0:
        t = cuda_lib.transpose_block_fp8(q)
        assert torch.equal(t.codes, q.codes.transpose(1, 2)) and torch.equal(t.scales, q.scales.transpose(1, 2))
        back = cuda_lib.transpose_block_fp8(t)
        assert torch.equal(back.codes, q.codes) and torch.equal(back.scales, q.scales)


def offsets_of(counts, M):
    o = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    assert o[-1] <= M
    return torch.from_numpy(o)


# (M, N, K, rows of each matrix or None, dtype): single rows, empty groups at both ends, groups on
# and one past the tile heights, partial tiles of N and K on either side of the tile widths, rows
# of no matrix, one matrix for all rows, many matrices
PRODUCTS = [
    (1, 128, 128, None, BF), (1, 1, 16, None, FP), (3, 64, 144, None, FP), (16, 256, 256, None, BF),
    (129, 257, 272, None, FP), (300, 512, 512, None, BF), (130, 1000, 1040, None, FP), (700, 1536, 640, None, BF),
    (80, 192, 256, [0, 1, 0, 31, 32, 16, 0, 0], BF), (500, 384, 384, [0, 128, 129, 127, 1, 0, 33], FP),
    (64, 130, 160, [64, 0, 0], FP), (40, 264, 528, [0, 0, 40], BF), (50, 96, 2064, [17, 0, 20], BF),
    (600, 520, 400, [5, 300, 0, 250, 40], FP), (90, 64, 128, [1] * 90, BF), (33, 72, 112, [0] * 5, FP),
    (1500, 2048, 512, [700, 3, 400, 0, 390], BF), (257, 4096, 256, None, BF), (2050, 320, 1408, [2000, 1, 49], FP),
    # up to 16 rows, which the product quantizes itself: several blocks per warp, both tile widths
    (16, 300, 2064, [0, 5, 0, 1, 7, 0], FP), (13, 4096, 400, None, BF), (9, 264, 4112, [2, 0, 3], FP),
    (16, 9800, 272, None, FP), (11, 1000, 1152, [1] * 9, BF), (1, 72, 4096, None, FP),
    # enough tiles for the large ones: one CTA per tile (many matrices), and pairs of CTAs
    (2500, 1300, 400, [0, 128, 129, 127, 1, 0, 0, 255, 256, 257, 16, 17, 300, 64, 33, 500, 32, 31, 0, 200], FP),
    (5000, 1536, 256, [100] * 45 + [480], BF), (4100, 1300, 272, None, FP), (4224, 2048, 1040, None, BF),
    (9000, 520, 640, [3000, 0, 2177, 3600, 100], BF), (9000, 776, 144, [128, 129, 4000, 1, 4463], FP),
]


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: f"M{c[0]}_N{c[1]}_K{c[2]}_G{len(c[3]) if c[3] else 1}")
def test_product(cuda_lib, case):
    M, N, K, counts, dtype = case
    moe = cuda_lib
    G = len(counts) if counts else 1
    x = rows(M, K, 11 * M + K)
    g = torch.Generator().manual_seed(5 * N + K)
    w = torch.randn(G, N, K, generator=g) * 0.02 * (1 + torch.arange(G)[:, None, None])
    q = moe.quantize_block_fp8(w.cuda())
    offsets = offsets_of(counts, M) if counts else None
    ws = moe.block_fp8_workspace(M, q)
    xc, xs = quantized_rows(x.float().numpy())
    ref, mag = product_reference(xc, xs, q.codes.cpu().numpy(), q.scales.cpu().numpy(), offsets)
    out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    moe.block_fp8_matmul(x.cuda(), q, ws, offsets=None if offsets is None else offsets.cuda(), out=out)
    check(out, ref, out_bound(ref, mag, K, dtype), "out")
    if offsets is not None:
        assert bool((out[int(offsets[-1]):] == 0).all())
    assert moe.device_status(ws) == 0


def test_many_matrices_with_few_rows(cuda_lib):
    """A decode step's shape: 512 matrices, most of them without rows."""
    moe = cuda_lib
    M, N, K, G = 80, 256, 512, 512
    g = torch.Generator().manual_seed(2)
    which = torch.sort(torch.randint(0, G, (M - 6,), generator=g))[0]
    offsets = torch.searchsorted(which, torch.arange(G + 1)).int()
    codes = torch.randint(0, 120, (G, N, K), generator=g, dtype=torch.uint8)
    codes |= torch.randint(0, 2, (G, N, K), generator=g, dtype=torch.uint8) << 7
    scales = torch.rand(G, 2, 4, generator=g) + 0.5
    q = moe.BlockFP8Weights(codes.cuda(), scales.cuda())
    x = rows(M, K, 8)
    ws = moe.block_fp8_workspace(M, q)
    out = moe.block_fp8_matmul(x.cuda(), q, ws, offsets=offsets.cuda(), out_fp32=True)
    ref, mag = product_reference(*quantized_rows(x.float().numpy()), codes.numpy(), scales.numpy(), offsets)
    check(out, ref, out_bound(ref, mag, K, FP), "out")


def test_input_gradient_is_the_transposed_product(cuda_lib):
    """Against the formula on the transposed codes, and, for rows that e4m3 holds exactly, against
    central differences of the forward form in 64 bits."""
    moe = cuda_lib
    M, N, K = 150, 192, 272
    counts = [100, 0, 45]
    offsets = offsets_of(counts, M)
    g = torch.Generator().manual_seed(12)
    q = moe.quantize_block_fp8((torch.randn(3, N, K, generator=g) * 0.02).cuda())
    t = moe.transpose_block_fp8(q)
    dy = torch.randint(-8, 9, (M, N), generator=g).float()
    dy[:, ::128] = 448.0                      # each block's largest is 448: the codes hold the integers exactly
    ws = moe.block_fp8_workspace(M, t)
    dx = moe.block_fp8_matmul(dy.bfloat16().cuda(), t, ws, offsets=offsets.cuda(), out_fp32=True)
    ref, mag = product_reference(*quantized_rows(dy.numpy()), t.codes.cpu().numpy(), t.scales.cpu().numpy(), offsets)
    check(dx, ref, out_bound(ref, mag, N, FP), "dx")
    direction = torch.randn(M, K, generator=g).double()
    codes = q.codes.cpu().view(torch.float8_e4m3fn).double()
    s = q.scales.cpu().double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    total = 0.0
    for i in range(3):
        a, b = int(offsets[i]), int(offsets[i + 1])
        f = lambda e: float((dy[a:b].double() * ((e * direction[a:b]) @ (codes[i] * s[i]).t())).sum())  # noqa: E731
        total += (f(1e-3) - f(-1e-3)) / 2e-3
    got = float((dx.cpu().double() * direction).sum())
    assert abs(got - total) <= float((out_bound(ref, mag, N, FP) * direction.abs()).sum()) + 1e-9 * abs(total)


def test_empty_and_bad_offsets(cuda_lib):
    moe = cuda_lib
    q = moe.quantize_block_fp8(torch.randn(3, 96, 128, device="cuda"))
    ws = moe.block_fp8_workspace(64, q)
    assert moe.block_fp8_matmul(torch.empty(0, 128, dtype=BF, device="cuda"), q, ws,
                                offsets=torch.zeros(4, dtype=torch.int32, device="cuda")).shape == (0, 96)
    x = torch.randn(64, 128, device="cuda").bfloat16()
    for bad in ([0, 10, 5, 64], [1, 10, 20, 64], [0, 10, 20, 65], [-1, 0, 3, 4], [0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]):
        out = torch.full((64, 96), 7.0, device="cuda")
        moe.block_fp8_matmul(x, q, ws, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out)
        assert moe.device_status(ws) == -1 and bool((out == 0).all())


def test_other_streams_graphs_and_repeats(cuda_lib):
    moe = cuda_lib
    M, N, K = 200, 512, 384
    q = moe.quantize_block_fp8(torch.randn(4, N, K, device="cuda"))
    offsets = offsets_of([50, 0, 100, 30], M).cuda()
    x = rows(M, K, 1).cuda()
    ws = moe.block_fp8_workspace(1000, q)
    first = moe.block_fp8_matmul(x, q, ws, offsets=offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = torch.empty_like(first)
    moe.block_fp8_matmul(x, q, ws, offsets=offsets, out=second, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    third = torch.empty_like(first)
    with torch.cuda.graph(graph):
        moe.block_fp8_matmul(x, q, ws, offsets=offsets, out=third)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third)


def test_refusals(cuda_lib):
    moe = cuda_lib
    q = moe.quantize_block_fp8(torch.randn(2, 64, 128, device="cuda"))
    ws = moe.block_fp8_workspace(32, q)
    x = torch.randn(32, 128, device="cuda").bfloat16()
    off = torch.tensor([0, 16, 32], dtype=torch.int32, device="cuda")
    with pytest.raises(moe.MoeError) as e:            # two matrices need offsets
        moe.block_fp8_matmul(x, q, ws)
    assert e.value.status == -1
    with pytest.raises(ValueError):
        moe.block_fp8_matmul(x[:, :64].contiguous(), q, ws, offsets=off)
    with pytest.raises(ValueError):
        moe.block_fp8_matmul(x, q, ws, offsets=off[:2])
    with pytest.raises(TypeError):
        moe.block_fp8_matmul(x.float(), q, ws, offsets=off)
    with pytest.raises(TypeError):
        moe.block_fp8_matmul(x, q, ws, offsets=off, out=torch.empty(32, 64, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        moe.block_fp8_matmul(x, moe.BlockFP8Weights(q.codes, q.scales[:1]), ws, offsets=off)
    with pytest.raises(moe.MoeError) as e:
        moe.block_fp8_matmul(x, q, ws[:512], offsets=off)
    assert e.value.status == -3
    with pytest.raises(moe.MoeError) as e:
        moe.quantize_block_fp8(torch.randn(1, 64, 120, device="cuda"))
    assert e.value.status == -2
    with pytest.raises(moe.MoeError) as e:
        moe.transpose_block_fp8(moe.quantize_block_fp8(torch.randn(1, 72, 128, device="cuda")))
    assert e.value.status == -2
    with pytest.raises(moe.MoeError) as e:
        moe.quantize_rows_block_fp8(torch.randn(4, 8, device="cuda").bfloat16())
    assert e.value.status == -2
