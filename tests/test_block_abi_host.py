"""Host checks of the operators around the experts (no GPU): workspace sizes and refusals that come
before any CUDA call, and the plain forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from block_cases import quantized_matrices, quantized_rows, sort_reference

P = ctypes.c_void_p
OK, MIS, NULL = P(0x100000), P(0x100008), P(0)     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from quantized_moe_expert_nvfp4_gb300 import build
    build.build()
    import quantized_moe_expert_nvfp4_gb300 as moe
    return moe, moe.load()


def test_workspace_sizes(lib):
    moe, L = lib
    assert L.moe_sort_workspace_size(8, 512, 10) > 0 and L.moe_sort_workspace_size(0, 1, 1) > 0
    for bad in ((-1, 8, 2), (8, 0, 2), (8, 1025, 2), (8, 8, 0), (8, 8, 17), (1 << 30, 8, 2)):
        assert L.moe_sort_workspace_size(*bad) == 0, bad
    assert L.moe_block_fp8_workspace_size(80, 2048) >= 80 * 2048
    assert L.moe_block_fp8_workspace_size(2 ** 31 - 1, 131072) > 2 ** 47        # sizes past 32 bits
    for bad in ((-1, 128), (1, 8), (1, 24), (1, 131088), (2 ** 31, 128)):
        assert L.moe_block_fp8_workspace_size(*bad) == 0, bad
    assert L.moe_norm_workspace_size(8, 2048) > 0 and L.moe_norm_workspace_size(2 ** 31 - 1, 16384) > 0
    for bad in ((-1, 64), (8, 4), (8, 60), (8, 16392)):
        assert L.moe_norm_workspace_size(*bad) == 0, bad


def test_token_refusals(lib):
    moe, L = lib
    B = moe.block
    s = B.MoeTokens(16, 64, 8, 2, 0)
    need = L.moe_sort_workspace_size(16, 8, 2)
    sort = lambda **o: L.moe_sort_tokens(o.get("x", OK), o.get("ids", OK), o.get("s", s), o.get("xs", OK), OK,  # noqa: E731
                                         o.get("ss", OK), OK, o.get("ws", OK), o.get("n", need), None)
    assert sort(x=NULL) == -1 and sort(ids=MIS) == -1 and sort(xs=MIS) == -1 and sort(ss=NULL) == -1
    assert sort(ws=P(0x100010)) == -1 and sort(ws=NULL) == -1 and sort(n=need - 1) == -3
    for bad, status in ((B.MoeTokens(16, 60, 8, 2, 0), -2), (B.MoeTokens(16, 64, 8, 17, 0), -2),
                        (B.MoeTokens(-1, 64, 8, 2, 0), -2), (B.MoeTokens(16, 64, 8, 2, 2), -1), (B.MoeTokens(16, 16392, 8, 2, 0), -2)):
        assert sort(s=bad) == status
        assert L.moe_return_tokens(OK, OK, OK, NULL, bad, OK, None) == status
        assert L.moe_sort_tokens_backward(OK, OK, bad, OK, None) == status
        assert L.moe_return_tokens_backward(OK, OK, OK, OK, bad, OK, OK, None) == status
    assert L.moe_return_tokens(OK, OK, OK, MIS, s, OK, None) == -1
    assert L.moe_return_tokens(OK, OK, NULL, NULL, s, OK, None) == -1
    assert L.moe_sort_tokens_backward(OK, NULL, s, OK, None) == -1
    assert L.moe_return_tokens_backward(OK, OK, OK, OK, s, OK, MIS, None) == -1
    empty = B.MoeTokens(0, 64, 8, 2, 0)
    assert L.moe_return_tokens(NULL, NULL, NULL, NULL, empty, NULL, None) == 0     # nothing to enqueue


def test_product_refusals(lib):
    moe, L = lib
    B = moe.block
    w = B.MoeBlockFp8Weights(0x200000, 0x300000, 4, 64, 128)
    need = L.moe_block_fp8_workspace_size(32, 128)
    mm = lambda **o: L.moe_block_fp8_matmul(o.get("x", OK), o.get("M", 32), o.get("off", OK), o.get("w", w),  # noqa: E731
                                            o.get("out", OK), o.get("f", 0), o.get("ws", OK), o.get("n", need), None)
    assert mm(x=MIS) == -1 and mm(out=NULL) == -1 and mm(off=NULL) == -1 and mm(off=MIS) == -1 and mm(f=2) == -1
    assert mm(n=need - 1) == -3 and mm(M=-1) == -2 and mm(M=2 ** 31, n=2 ** 60) == -2
    for bad, status in ((B.MoeBlockFp8Weights(0, 0x300000, 4, 64, 128), -1), (B.MoeBlockFp8Weights(0x200000, 0x300008, 4, 64, 128), -1),
                        (B.MoeBlockFp8Weights(0x200000, 0x300000, 1026, 64, 128), -2),
                        (B.MoeBlockFp8Weights(0x200000, 0x300000, 4, 0, 128), -2),
                        (B.MoeBlockFp8Weights(0x200000, 0x300000, 4, 64, 120), -2)):
        assert mm(w=bad) == status
        assert L.moe_transpose_block_fp8(bad, OK, OK, None) == status
    assert L.moe_transpose_block_fp8(B.MoeBlockFp8Weights(0x200000, 0x300000, 4, 72, 128), OK, OK, None) == -2
    assert L.moe_transpose_block_fp8(w, MIS, OK, None) == -1
    assert L.moe_quantize_block_fp8(OK, 2, 1, 16, 32, OK, OK, None) == -1
    assert L.moe_quantize_block_fp8(OK, 1, 1, 16, 24, OK, OK, None) == -2
    assert L.moe_quantize_rows_block_fp8(MIS, 4, 32, OK, OK, None) == -1
    assert L.moe_quantize_rows_block_fp8(OK, 4, 40, OK, OK, None) == -2
    assert L.moe_quantize_rows_block_fp8(NULL, 0, 32, NULL, NULL, None) == 0


def test_norm_refusals(lib):
    moe, L = lib
    B = moe.block
    mk = lambda **o: B.MoeNorm(*[{**dict(T=4, H=64, r=0, b=0, gate=0, eps=1e-6, off=0.0, rs=1.0, bs=1.0), **o}[k]  # noqa: E731
                                 for k in ("T", "H", "r", "b", "gate", "eps", "off", "rs", "bs")])
    before = lambda s, x=OK, rstd=OK: L.moe_norm_before(x, OK, s, OK, rstd, None)  # noqa: E731
    assert before(mk(), x=NULL) == -1 and before(mk(), rstd=MIS) == -1
    for bad, status in ((mk(H=60), -2), (mk(T=-1), -2), (mk(H=0), -2), (mk(r=2), -1), (mk(b=-1), -1), (mk(gate=4), -1), (mk(gate=-1), -1),
                        (mk(eps=-1.0), -1), (mk(eps=float("nan")), -1), (mk(rs=float("inf")), -1), (mk(bs=float("nan")), -1)):
        assert before(bad) == status
    after = lambda s, gate=NULL, wn=NULL, n=NULL, rn=NULL: L.moe_norm_after(OK, OK, OK, gate, wn, s, OK, n, OK, rn, None)  # noqa: E731
    assert after(mk(), gate=OK) == -1 and after(mk(gate=1)) == -1 and after(mk(), wn=OK) == -1 and after(mk(), n=OK) == -1
    assert after(mk(), rn=OK) == -1 and after(mk(gate=3), gate=MIS) == -1
    need = L.moe_norm_workspace_size(4, 64)

    def grad(s=mk(), dn=NULL, out=NULL, gate=NULL, wn=NULL, rn=NULL, dg=NULL, dwn=NULL, n=need, dw=OK):
        return L.moe_norm_after_backward(OK, dn, OK, out, OK, gate, wn, OK, rn, s, OK, OK, dw, dg, dwn, OK, n, None)

    assert grad(wn=OK) == -1 and grad(wn=OK, dwn=OK) == -1 and grad(dn=OK) == -1 and grad(dwn=OK) == -1 and grad(rn=OK) == -1
    assert grad(s=mk(gate=1), gate=OK) == -1 and grad(s=mk(gate=1), dg=OK) == -1 and grad(gate=OK, dg=OK) == -1
    assert grad(dw=NULL) == -1 and grad(n=need - 1) == -3
    assert L.moe_norm_before_backward(OK, OK, OK, OK, MIS, mk(), OK, OK, OK, need, None) == -1
    assert L.moe_norm_before_backward(OK, OK, OK, OK, NULL, mk(), OK, OK, OK, need - 1, None) == -3


def test_plain_forms():
    """The block rule on values whose codes are known, and the sort's on a hand-worked batch."""
    x = np.zeros((2, 144), dtype=np.float32)
    x[0, :5] = [448, 17, 18.5, -0.001, 240]
    x[1, 128] = -7
    codes, scales = quantized_rows(x)
    v = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert v[0, :5].tolist() == [448, 16, 18, -(2.0 ** -9), 240] and v[1, 128] == -448
    assert scales[0].tolist() == [1, 1] and scales[1, 0] == 1 and scales[1, 1] == np.float32(7) / np.float32(448)
    w = np.zeros((1, 130, 16), dtype=np.float32)
    w[0, 129, 0] = 896.0
    codes, scales = quantized_matrices(w)
    assert codes.shape == (1, 130, 16) and codes[0, 129, 0] == 0x7e and scales.tolist() == [[[1.0], [2.0]]]
    offsets, order, pos = sort_reference(torch.tensor([[2, -1], [0, 2], [9, 0]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4] and order.tolist() == [2, 5, 0, 3, 1, 4]
    assert pos.tolist() == [[2, -5], [0, 3], [-6, 1]]
