"""Plain 64-bit forms of the operators around the experts, on the CPU, and their error bounds.

u is half an ulp: 2^-8 for a result rounded to bf16, 0 for one kept in fp32 (whose roundings the
other term covers); every bound is u |ref| plus a multiple of 2^-24 of the sum of the magnitudes
that the kernel adds in fp32."""
import numpy as np
import torch

F32 = 2.0 ** -24


def half_ulp(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 0.0


def f64(t):
    return t.detach().cpu().double()


def check(got, ref, bound, what):
    """|got - ref| <= bound elementwise; infinities and NaN have to be the reference's."""
    got, ref = f64(got), f64(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = (got == ref) | (got.isnan() & ref.isnan())
    off = torch.where(same, 0.0, (got - ref).abs())
    over = ~(off <= bound)
    assert not over.any(), f"{what}: {int(over.sum())} of {over.numel()} beyond the bound, worst {float((off / (bound + 1e-300)).max()):.3g} x"


# ---------------------------------------------------------------- tokens

def sort_reference(ids, E):
    """(offsets, sorted_slot, slot_pos) by Python's stable sort."""
    T, k = ids.shape
    flat = ids.reshape(-1).tolist()
    key = [e if 0 <= e < E else E for e in flat]
    order = sorted(range(T * k), key=lambda s: key[s])
    pos = [0] * (T * k)
    for p, s in enumerate(order):
        pos[s] = p if key[s] < E else -1 - p
    offsets = np.cumsum([0] + [key.count(e) for e in range(E)])
    return offsets, np.array(order, dtype=np.int64), np.array(pos, dtype=np.int64).reshape(T, k)


def taken(rows, slot_pos):
    routed = slot_pos >= 0
    return torch.where(routed[..., None], rows[slot_pos.clamp_min(0)], torch.zeros((), dtype=torch.float64))


# ---------------------------------------------------------------- e4m3 in blocks of 128

def e4m3_values(codes):
    return torch.from_numpy(codes).view(torch.float8_e4m3fn).double()


def quantized(blocks):
    """Codes and scales of fp32 blocks [..., n] with one scale each, by the block rule in numpy's fp32."""
    b = blocks.astype(np.float32)
    amax = np.abs(b).max(-1, keepdims=True)
    usable = (amax > 0) & np.isfinite(amax)
    with np.errstate(all="ignore"):
        inv = np.where(usable, np.float32(448) / np.where(usable, amax, 1), np.float32(1)).astype(np.float32)
        scale = np.where(usable, np.where(usable, amax, 1) / np.float32(448), np.float32(1)).astype(np.float32)
        q = np.clip(b * inv, -448, 448)
    return torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), scale[..., 0]


def pad128(a, axes):
    return np.pad(a, [(0, -a.shape[i] % 128 if i in axes else 0) for i in range(a.ndim)])


def quantized_rows(x):
    """x fp32 [M, K] -> codes [M, 128 KB], scales [M, KB]."""
    t = pad128(x, (1,)).reshape(x.shape[0], -1, 128)
    codes, scales = quantized(t)
    return codes.reshape(x.shape[0], -1), scales


def quantized_matrices(w):
    """w fp32 [G, N, K] -> codes [G, N, K], scales [G, NB, KB]."""
    G, N, K = w.shape
    t = pad128(w, (1, 2))
    NB, KB = t.shape[1] // 128, t.shape[2] // 128
    t = t.reshape(G, NB, 128, KB, 128).transpose(0, 1, 3, 2, 4)
    codes, scales = quantized(t.reshape(G, NB, KB, -1))
    codes = codes.reshape(G, NB, KB, 128, 128).transpose(0, 1, 3, 2, 4).reshape(G, NB * 128, KB * 128)
    return np.ascontiguousarray(codes[:, :N, :K]), scales


def product_reference(xc, xs, wc, ws, offsets):
    """(out, sum of magnitudes) [M, N] in 64 bits of codes [M, 128 KB], [G, N, K] and their scales."""
    G, N, K = wc.shape
    M = xc.shape[0]
    x = e4m3_values(xc)[:, :K] * torch.from_numpy(xs).double().repeat_interleave(128, 1)[:, :K]
    out, mag = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    for g in range(G):
        a, b = (0, M) if offsets is None else (int(offsets[g]), int(offsets[g + 1]))
        if b > a:
            s = torch.from_numpy(ws[g]).double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
            w = e4m3_values(wc[g]) * s
            out[a:b] = x[a:b] @ w.t()
            mag[a:b] = x[a:b].abs() @ w.abs().t()
    return out, mag


# ---------------------------------------------------------------- norms

def rstd_of(x, eps):
    return (x.square().mean(1) + eps).rsqrt()


def gate_factor(gate, T, H):
    if gate is None:
        return torch.ones(1, 1, dtype=torch.float64)
    g = f64(gate)
    return g[None] if g.shape == (H,) else g.reshape(T, 1) if g.numel() == T else g


def after_reference(y, x, w, gate, a, b, eps):
    """out and the magnitudes of its two terms."""
    T, H = x.shape
    branch = b * gate_factor(gate, T, H) * (y * rstd_of(y, eps)[:, None] * w)
    return a * x + branch, (a * x).abs() + branch.abs()


def norm_grad(dn, x, w, r):
    """dx, dw of n = x r w and the sums of their terms' magnitudes."""
    xh = x * r[:, None]
    d = dn * w
    dot, mag = (d * xh).mean(1, keepdim=True), (d * xh).abs().mean(1, keepdim=True)
    return (r[:, None] * (d - xh * dot), (dn * xh).sum(0),
            r[:, None].abs() * (d.abs() + xh.abs() * mag), (dn * xh).abs().sum(0))
