"""Measured cases of the operators around the routed experts, each in a plain form and through the library.

Three operators of one differentiable block whose experts are frozen 8-bit weights:

  tokens    tokens sorted by expert and returned with their weights, and the gradients of both
  product   matrix product in e4m3 with a scale for each block of 128, one matrix or one per expert
  norm      norms before and after the block with its gate and residual scale, and their gradients

`run` computes a case with elementary torch operations in 32 bits, or, where `own` is true, with the
library's calls; `exact` computes it once more in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one decode step of 8 rows: ten experts each out of 512
        dict(name="sort_decode", op="tokens", kind="sort", T=8, H=2048, E=512, k=10, fp32=False, skew=1.0, drop=0.0),
        # a prefill chunk with a few padding tokens and dropped slots
        dict(name="sort_prefill", op="tokens", kind="sort", T=4096, H=2048, E=512, k=10, fp32=False, skew=1.0, drop=0.03),
        # an odd batch in 32 bits, few experts
        dict(name="return_odd_f32", op="tokens", kind="return", T=1501, H=1000, E=40, k=6, fp32=True, skew=1.5, drop=0.05),
        # the backward pass of a long sequence: gradients of the expert rows and of the weights
        dict(name="return_grad_long", op="tokens", kind="return_grad", T=32768, H=2048, E=512, k=10, fp32=False, skew=1.0,
             drop=0.01),
        # gate and up of a decode step of 8 rows: 80 rows over 512 experts, most of them empty
        dict(name="experts_decode", op="product", M=80, N=1024, K=2048, G=512, skew=0.5, tail=0, fp32=False, grad=False),
        # gate and up of a prefill chunk of 4096 tokens: every expert's weights are read
        dict(name="experts_prefill", op="product", M=40960, N=1024, K=2048, G=512, skew=0.5, tail=0, fp32=False, grad=False),
        # one large matrix (a shared projection over a long batch)
        dict(name="dense_large", op="product", M=8192, N=4096, K=4096, G=1, skew=0.0, tail=0, fp32=False, grad=False),
        # input gradient through odd-sized experts, with dropped rows at the end
        dict(name="experts_grad_odd", op="product", M=1777, N=2000, K=1040, G=24, skew=1.0, tail=37, fp32=True, grad=True),
        # a decode step's residual update and the next block's input
        dict(name="after_decode", op="norm", kind="after", T=8, H=2048, fp32=False, gate="channel", next=True),
        # the same over a long sequence
        dict(name="after_long", op="norm", kind="after", T=32768, H=2048, fp32=False, gate="channel", next=True),
        # backward pass of a prefill chunk: sums over the tokens for both norms' weights and the gate
        dict(name="after_grad_prefill", op="norm", kind="after_grad", T=4096, H=2048, fp32=False, gate="channel", next=True),
        # backward pass of the norm before the block, odd sizes, residual stream in 32 bits
        dict(name="before_grad_odd", op="norm", kind="before_grad", T=2999, H=1000, fp32=True, gate="none", next=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tokens", "product", "norm"])
    if op == "tokens":
        E = _log(rng, 4, 512)
        return dict(op=op, kind=rng.choice(["sort", "sort_grad", "return", "return_grad"]), T=_log(rng, 1, 16384),
                    H=8 * _log(rng, 16, 320), E=E, k=rng.randint(1, min(E, 10)), fp32=rng.random() < 0.3,
                    skew=round(rng.uniform(0.0, 2.0), 2), drop=round(rng.choice([0.0, rng.uniform(0.0, 0.3)]), 3))
    if op == "product":
        G = rng.choice([1, _log(rng, 2, 128)])
        M = _log(rng, 1, 8192)
        return dict(op=op, M=M, N=8 * _log(rng, 8, 256), K=16 * _log(rng, 4, 160), G=G,
                    skew=round(rng.uniform(0.0, 1.0), 2), tail=rng.choice([0, M // 7]), fp32=rng.random() < 0.3,
                    grad=rng.random() < 0.4)
    kind = rng.choice(["before", "before_grad", "after", "after_grad"])
    after = kind.startswith("after")
    return dict(op=op, kind=kind, T=_log(rng, 1, 16384), H=8 * _log(rng, 16, 640), fp32=rng.random() < 0.3,
                gate=rng.choice(["none", "channel", "token", "element"]) if after else "none",
                next=after and rng.random() < 0.6)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _fill(out, g, scale=1.0):
    return out.normal_(0.0, scale, generator=g)


def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _routing(case, g):
    """Ids of a routed batch (-1: dropped) and its weights: skewed experts, padding tokens, single dropped slots."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = _randn(g, T, E) + case["skew"] * _randn(g, E)
    v, ids = torch.topk(logits, k, dim=1)
    w = torch.softmax(v, 1)
    if case["drop"]:
        gone = torch.rand(T, k, generator=g, device="cuda") < case["drop"]
        gone |= torch.rand(T, 1, generator=g, device="cuda") < case["drop"] / 2
        ids = torch.where(gone, -1, ids)
    return ids.to(torch.int32).contiguous(), w.contiguous()


def _positions(ids, E):
    """(slot_pos, key, order) of the stable sort by expert; a dropped slot's place p is written as -1 - p."""
    flat = ids.reshape(-1).long()
    routed = (flat >= 0) & (flat < E)
    key = torch.where(routed, flat, E)
    order = torch.sort(key, stable=True)[1]
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=order.device)
    return torch.where(routed, pos, -1 - pos).to(torch.int32), key, order


def _prepare_tokens(case, g):
    T, H, E, k, kind = case["T"], case["H"], case["E"], case["k"], case["kind"]
    dt = torch.float32 if case["fp32"] else torch.bfloat16
    ids, w = _routing(case, g)
    S = T * k
    if kind == "sort":
        return dict(x=_fill(_empty(T, H, dtype=dt), g), ids=ids, xs=_empty(S, H, dtype=dt), offsets=_empty(E + 1, dtype=torch.int32),
                    sorted_slot=_empty(S, dtype=torch.int32), slot_pos=_empty(T, k, dtype=torch.int32))
    slot_pos = _positions(ids, E)[0].view(T, k).contiguous()
    if kind == "sort_grad":
        return dict(dxs=_fill(_empty(S, H, dtype=dt), g), slot_pos=slot_pos, dx=_empty(T, H, dtype=dt))
    ys = _fill(_empty(S, H, dtype=dt), g, 0.3)
    if kind == "return":
        return dict(ys=ys, slot_pos=slot_pos, w=w, out=_empty(T, H, dtype=dt))
    return dict(ys=ys, slot_pos=slot_pos, w=w, dout=_fill(_empty(T, H, dtype=dt), g, 0.1), dys=_empty(S, H, dtype=dt),
                dw=_empty(T, k, dtype=torch.float32))


def _blocks(n):
    return (n + 127) // 128


def _quantized_weights(case, g):
    """Weights N(0, 0.02^2) in blocks of 128 x 128: e4m3 bytes [G, N, K] and scales [G, N/128, K/128].  A backward pass
    multiplies by the transposed matrix, of which its program keeps a second layout: the same codes and scales, transposed."""
    G, N, K = case["G"], case["N"], case["K"]
    if case["grad"]:
        N, K = K, N
    NB, KB = _blocks(N), _blocks(K)
    w = torch.zeros(G, NB * 128, KB * 128, device="cuda")
    w[:, :N, :K].normal_(0.0, 0.02, generator=g)
    t = w.view(G, NB, 128, KB, 128)
    amax = t.abs().amax(dim=(2, 4))
    t *= (448.0 / amax)[:, :, None, :, None]
    codes, scales = w.to(torch.float8_e4m3fn).view(torch.uint8)[:, :N, :K], amax / 448.0
    if case["grad"]:
        codes, scales = codes.transpose(1, 2), scales.transpose(1, 2)
    return codes.contiguous(), scales.contiguous()


def _prepare_product(case, g):
    M, N, K, G = case["M"], case["N"], case["K"], case["G"]
    codes, scales = _quantized_weights(case, g)
    x = _fill(_empty(M, K, dtype=torch.bfloat16), g)
    x[:: max(1, min(100, M))] *= 30.0  # a few rows of outliers
    offsets, longest = None, M
    if G > 1 or case["tail"]:
        share = torch.softmax(case["skew"] * _randn(g, G), 0)
        which = torch.multinomial(share, M - case["tail"], replacement=True, generator=g)
        counts = torch.zeros(G, dtype=torch.int64, device="cuda").index_add_(0, which, torch.ones_like(which))
        offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.cumsum(counts, 0)
        longest = int(counts.max())
    return dict(x=x, codes=codes, scales=scales, offsets=offsets, longest=longest,
                out=_empty(M, N, dtype=torch.float32 if case["fp32"] else torch.bfloat16))


def _prepare_norm(case, g):
    T, H, kind = case["T"], case["H"], case["kind"]
    rt = torch.float32 if case["fp32"] else torch.bfloat16  # type of the residual stream
    bf = torch.bfloat16
    x = _fill(_empty(T, H, dtype=rt), g, 2.0)
    w = 1.0 + _randn(g, H, scale=0.1)
    s = dict(x=x, w=w)
    if kind.startswith("before"):
        if kind == "before":
            s.update(n=_empty(T, H, dtype=bf), rstd=_empty(T, dtype=torch.float32))
        else:
            s.update(dn=_fill(_empty(T, H, dtype=bf), g, 0.1), dres=_fill(_empty(T, H, dtype=rt), g, 0.1),
                     rstd=torch.rsqrt(x.float().square().mean(1) + EPS), dx=_empty(T, H, dtype=rt),
                     dw=_empty(H, dtype=torch.float32))
        return s
    gate = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[case["gate"]]
    if gate is not None:
        gate = _randn(g, *gate, scale=0.3).to(bf if case["gate"] == "element" else torch.float32)
    y = _fill(_empty(T, H, dtype=bf), g, 0.5)
    wn = 1.0 + _randn(g, H, scale=0.1) if case["next"] else None
    s.update(y=y, gate=gate, w_next=wn, a=0.9, b=1.25)
    if kind == "after":
        s.update(out=_empty(T, H, dtype=rt), n=_empty(T, H, dtype=bf) if case["next"] else None,
                 rstd=_empty(T, dtype=torch.float32), rstd_next=_empty(T, dtype=torch.float32) if case["next"] else None)
        return s
    s.update(dout=_fill(_empty(T, H, dtype=rt), g, 0.1), rstd=torch.rsqrt(y.float().square().mean(1) + EPS))
    if case["next"]:  # x stands for the saved output of the forward call, from which the next norm was taken
        s.update(dn=_fill(_empty(T, H, dtype=bf), g, 0.1), rstd_next=torch.rsqrt(x.float().square().mean(1) + EPS))
    s.update(dy=_empty(T, H, dtype=bf), dx=_empty(T, H, dtype=rt), dw=_empty(H, dtype=torch.float32),
             dgate=None if gate is None else torch.empty_like(gate),
             dw_next=_empty(H, dtype=torch.float32) if case["next"] else None)
    return s


def prepare(case, seed):
    g = _gen(seed)
    make = {"tokens": _prepare_tokens, "product": _prepare_product, "norm": _prepare_norm}[case["op"]]
    return dict(make(case, g), case=case)


# ---------------------------------------------------------------- plain forms

def _plain_sort(s):
    x, ids, E = s["x"], s["ids"], s["case"]["E"]
    slot_pos, key, order = _positions(ids, E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = torch.cumsum(counts[:E], 0)
    xs = torch.where((key[order] < E)[:, None], x[order // ids.shape[1]], torch.zeros((), dtype=x.dtype, device=x.device))
    return dict(xs=xs, offsets=offsets, sorted_slot=order.to(torch.int32), slot_pos=slot_pos.view(ids.shape))


def _taken(rows, slot_pos):
    """The rows of each token's slots [T, k, H] in 32 bits, zero for dropped slots."""
    routed = slot_pos >= 0
    return torch.where(routed[..., None], rows[slot_pos.clamp_min(0).long()].float(), 0.0)


def _plain_sort_grad(s):
    return dict(dx=_taken(s["dxs"], s["slot_pos"]).sum(1).to(s["dxs"].dtype))


def _plain_return(s):
    return dict(out=(s["w"][..., None] * _taken(s["ys"], s["slot_pos"])).sum(1).to(s["ys"].dtype))


def _plain_return_grad(s):
    pos, dout = s["slot_pos"], s["dout"].float()
    w = torch.where(pos >= 0, s["w"], 0.0)
    dys = torch.empty_like(s["ys"])
    dys[torch.where(pos >= 0, pos, -1 - pos).reshape(-1).long()] = (w[..., None] * dout[:, None]).view(dys.shape).to(dys.dtype)
    return dict(dys=dys, dw=(_taken(s["ys"], pos) * dout[:, None]).sum(-1))


def _pad128(t, dims):
    pads = []
    for d in reversed(range(t.dim())):
        pads += [0, -t.shape[d] % 128 if d in dims else 0]
    return torch.nn.functional.pad(t, pads)


def _plain_quantized_rows(x):
    """Rows through e4m3 with a scale for each 128 columns, as the 32-bit values that they stand for."""
    K = x.shape[1]
    t = _pad128(x.float(), (1,)).view(x.shape[0], -1, 128)
    amax = t.abs().amax(2, keepdim=True)
    some, top = amax > 0, torch.full_like(amax, 448.0)
    inv = torch.where(some, top / amax, 1.0)  # tensors on both sides: each division is rounded once
    scale = torch.where(some, amax / top, 1.0)
    return ((t * inv).to(torch.float8_e4m3fn).float() * scale).view(x.shape[0], -1)[:, :K]


def _plain_product(s):
    x, codes, scales, offsets = s["x"], s["codes"], s["scales"], s["offsets"]
    G, N, K = codes.shape
    v = _plain_quantized_rows(x)
    full = scales.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    w = codes.view(torch.float8_e4m3fn).float() * full
    if offsets is None:
        return dict(out=(v @ w[0].t()).to(s["out"].dtype))
    start = offsets[:-1].long()
    at = torch.arange(s["longest"], device=x.device)
    rows = start[:, None] + at
    inside = rows < offsets[1:, None]
    rows = rows.clamp_max(x.shape[0] - 1)
    y = torch.bmm(torch.where(inside[..., None], v[rows], 0.0), w.transpose(1, 2))
    out = torch.zeros(x.shape[0] + 1, N, device=x.device)
    out[torch.where(inside, rows, x.shape[0])] = y
    return dict(out=out[:-1].to(s["out"].dtype))


def _gate_of(gate, kind):
    return 1.0 if gate is None else gate.float()[:, None] if kind == "token" else gate.float()


def _plain_norm_backward(dn, x, w, rstd):
    """(dx, dw) of n = x * rstd * w, in 32 bits."""
    xh = x.float() * rstd[:, None]
    d = dn * w
    return rstd[:, None] * (d - xh * (d * xh).mean(1, keepdim=True)), (dn * xh).sum(0)


def _plain_before(s):
    x = s["x"].float()
    rstd = torch.rsqrt(x.square().mean(1) + EPS)
    return dict(n=(x * rstd[:, None] * s["w"]).to(torch.bfloat16), rstd=rstd)


def _plain_before_grad(s):
    dx, dw = _plain_norm_backward(s["dn"].float(), s["x"], s["w"], s["rstd"])
    return dict(dx=(dx + s["dres"].float()).to(s["x"].dtype), dw=dw)


def _plain_after(s):
    x, y = s["x"].float(), s["y"].float()
    rstd = torch.rsqrt(y.square().mean(1) + EPS)
    out = s["a"] * x + s["b"] * _gate_of(s["gate"], s["case"]["gate"]) * (y * rstd[:, None] * s["w"])
    r = dict(out=out.to(s["x"].dtype), rstd=rstd)
    if s["w_next"] is not None:
        out = r["out"].float()  # the stored residual stream is what the next norm reads
        r["rstd_next"] = torch.rsqrt(out.square().mean(1) + EPS)
        r["n"] = (out * r["rstd_next"][:, None] * s["w_next"]).to(torch.bfloat16)
    return r


def _plain_after_grad(s):
    kind = s["case"]["gate"]
    d = s["dout"].float()
    r = {}
    if s["w_next"] is not None:
        more, r["dw_next"] = _plain_norm_backward(s["dn"].float(), s["x"], s["w_next"], s["rstd_next"])
        d = d + more
    r["dx"] = (s["a"] * d).to(s["x"].dtype)
    d = s["b"] * d
    if s["gate"] is not None:
        dgate = d * (s["y"].float() * s["rstd"][:, None] * s["w"])
        r["dgate"] = dgate.sum(0) if kind == "channel" else dgate.sum(1) if kind == "token" else dgate.to(s["gate"].dtype)
    dy, r["dw"] = _plain_norm_backward(d * _gate_of(s["gate"], kind), s["y"], s["w"], s["rstd"])
    r["dy"] = dy.to(s["y"].dtype)
    return r


def _plain(s):
    c = s["case"]
    if c["op"] == "product":
        return _plain_product(s)
    return {"sort": _plain_sort, "sort_grad": _plain_sort_grad, "return": _plain_return, "return_grad": _plain_return_grad,
            "before": _plain_before, "before_grad": _plain_before_grad, "after": _plain_after,
            "after_grad": _plain_after_grad}[c["kind"]](s)


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import quantized_moe_expert_nvfp4_gb300 as moe
    c = s["case"]
    if c["op"] == "product":
        if "weights" not in s:  # a program makes these once, at load time
            s["weights"] = moe.BlockFP8Weights(s["codes"], s["scales"])
            s["ws"] = moe.block_fp8_workspace(c["M"], s["weights"])
        return dict(out=moe.block_fp8_matmul(s["x"], s["weights"], s["ws"], offsets=s["offsets"], out=s["out"]))
    kind = c["kind"]
    if kind == "sort":
        if "ws" not in s:
            s["ws"] = moe.sort_workspace(c["T"], c["E"], c["k"])
        xs, offsets, sorted_slot, slot_pos = moe.sort_tokens(s["x"], s["ids"], c["E"], s["ws"], xs=s["xs"], offsets=s["offsets"],
                                                             sorted_slot=s["sorted_slot"], slot_pos=s["slot_pos"])
        return dict(xs=xs, offsets=offsets, sorted_slot=sorted_slot, slot_pos=slot_pos)
    if kind == "sort_grad":
        return dict(dx=moe.sort_tokens_backward(s["dxs"], s["slot_pos"], dx=s["dx"]))
    if kind == "return":
        return dict(out=moe.return_tokens(s["ys"], s["slot_pos"], s["w"], out=s["out"]))
    if kind == "return_grad":
        dys, dw = moe.return_tokens_backward(s["dout"], s["ys"], s["slot_pos"], s["w"], dys=s["dys"], dw=s["dw"])
        return dict(dys=dys, dw=dw)
    if kind == "before":
        n, rstd = moe.norm_before(s["x"], s["w"], eps=EPS, n=s["n"], rstd=s["rstd"])
        return dict(n=n, rstd=rstd)
    if kind == "after":
        out, n, rstd, rstd_next = moe.norm_after(s["y"], s["x"], s["w"], gate=s["gate"], w_next=s["w_next"], residual_scale=s["a"],
                                                 branch_scale=s["b"], eps=EPS, out=s["out"], n=s["n"], rstd=s["rstd"],
                                                 rstd_next=s["rstd_next"])
        r = dict(out=out, rstd=rstd)
        return dict(r, n=n, rstd_next=rstd_next) if n is not None else r
    if "ws" not in s:
        s["ws"] = moe.norm_workspace(c["T"], c["H"])
    if kind == "before_grad":
        dx, dw = moe.norm_before_backward(s["dn"], s["x"], s["w"], s["rstd"], s["ws"], dresidual=s["dres"], dx=s["dx"], dw=s["dw"])
        return dict(dx=dx, dw=dw)
    dy, dx, dw, dgate, dw_next = moe.norm_after_backward(
        s["dout"], s["y"], s["w"], s["rstd"], s["ws"], gate=s["gate"], dn=s.get("dn"), out=s["x"] if c["next"] else None,
        w_next=s["w_next"], rstd_next=s.get("rstd_next"), residual_scale=s["a"], branch_scale=s["b"], dy=s["dy"], dx=s["dx"],
        dw=s["dw"], dgate=s["dgate"], dw_next=s["dw_next"])
    r = dict(dy=dy, dx=dx, dw=dw)
    if dgate is not None:
        r["dgate"] = dgate
    if dw_next is not None:
        r["dw_next"] = dw_next
    return r


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_tokens(case, s):
    k, E, kind = case["k"], case["E"], case["kind"]
    if kind == "sort":
        ids = s["ids"].cpu().numpy().reshape(-1)
        groups = [[] for _ in range(E + 1)]
        for slot, e in enumerate(ids.tolist()):
            groups[e if 0 <= e < E else E].append(slot)
        order = [slot for g in groups for slot in g]
        kept = len(order) - len(groups[E])
        offsets, at = [0], 0
        for g in groups[:E]:
            at += len(g)
            offsets.append(at)
        slot_pos = [0] * len(order)
        for p, slot in enumerate(order):
            slot_pos[slot] = p if p < kept else -1 - p
        where = torch.tensor(order, device="cuda")
        xs = s["x"].double().index_select(0, where // k)
        xs[kept:] = 0.0
        as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        return dict(xs=xs, offsets=as_int(offsets), sorted_slot=as_int(order), slot_pos=as_int(slot_pos).view(-1, k))
    pos = s["slot_pos"].long()
    T = pos.shape[0]
    if kind in ("sort_grad", "return"):
        rows = s["dxs"] if kind == "sort_grad" else s["ys"]
        total = torch.zeros(T, rows.shape[1], dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(pos[:, j] >= 0)[:, 0]
            v = rows.index_select(0, pos[t, j]).double()
            total.index_add_(0, t, v if kind == "sort_grad" else v * s["w"][t, j].double()[:, None])
        return {"dx" if kind == "sort_grad" else "out": total}
    dys = torch.zeros(s["ys"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        p, d = pos[t, j], s["dout"].index_select(0, t).double()
        dys[p] = s["w"][t, j].double()[:, None] * d
        dw[t, j] = torch.einsum("th,th->t", d, s["ys"].index_select(0, p).double())
    return dict(dys=dys, dw=dw)


def _exact_e4m3(v):
    """Nearest e4m3 value, ties to the even one, saturating at 448 (v in 64 bits)."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def _exact_product(case, s):
    M, N, K, G = case["M"], case["N"], case["K"], case["G"]
    table = torch.empty(256, dtype=torch.float64, device="cuda")
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        table[c] = -v if c & 128 else v
    v = torch.empty(M, K, dtype=torch.float64, device="cuda")
    for kb in range(_blocks(K)):
        part = s["x"][:, 128 * kb:128 * kb + 128].float()
        amax = part.abs().max(1, keepdim=True)[0]
        amax = torch.where(amax == 0, 448.0, amax)
        top = torch.full_like(amax, 448.0)
        scaled = part * (top / amax)  # the definition takes the codes from this 32-bit product
        v[:, 128 * kb:128 * kb + 128] = _exact_e4m3(scaled.double()) * (amax / top).double()
    out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    bounds = [0, M] if s["offsets"] is None else s["offsets"].tolist()
    n_of, k_of = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    for g in range(G):
        a, b = bounds[g], bounds[g + 1]
        if b > a:
            w = table[s["codes"][g].long()] * s["scales"][g].double()[n_of][:, k_of]
            out[a:b] = v[a:b] @ w.t()
    return dict(out=out)


def _exact_norm(case, s):
    kind, f = case["kind"], lambda t: None if t is None else t.double()  # noqa: E731
    H = case["H"]
    x, w = f(s["x"]), f(s["w"])
    inv = lambda t: ((t * t).sum(1) / H + EPS).pow(-0.5)  # noqa: E731

    def back(dn, t, weight, r):
        g = dn * weight
        dot = (g * t).sum(1)
        return r[:, None] * g - t * (r.pow(3) * dot / H)[:, None], torch.einsum("th,th,t->h", dn, t, r)

    if kind == "before":
        r = inv(x)
        return dict(n=x * r[:, None] * w, rstd=r)
    if kind == "before_grad":
        dx, dw = back(f(s["dn"]), x, w, f(s["rstd"]))
        return dict(dx=dx + f(s["dres"]), dw=dw)
    y, gate, wn = f(s["y"]), f(s["gate"]), f(s["w_next"])
    if gate is None:
        gate = torch.ones((), dtype=torch.float64, device="cuda")
    elif case["gate"] == "token":
        gate = gate.unsqueeze(1)
    if kind == "after":
        r = inv(y)
        out = s["a"] * x + (s["b"] * gate) * (w * (y * r[:, None]))
        res = dict(out=out, rstd=r)
        if wn is not None:
            stored = out.to(s["x"].dtype).double()  # the next norm is that of the stored residual stream
            res.update(rstd_next=inv(stored), n=stored * inv(stored)[:, None] * wn)
        return res
    d, res = f(s["dout"]), {}
    if wn is not None:
        more, res["dw_next"] = back(f(s["dn"]), x, wn, f(s["rstd_next"]))
        d = d + more
    res["dx"] = s["a"] * d
    r = f(s["rstd"])
    if case["gate"] != "none":
        at = s["b"] * d * (y * r[:, None] * w)
        res["dgate"] = at.sum(0) if case["gate"] == "channel" else at.sum(1) if case["gate"] == "token" else at
    res["dy"], res["dw"] = back(s["b"] * d * gate, y, w, r)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return {"tokens": _exact_tokens, "product": _exact_product, "norm": _exact_norm}[case["op"]](case, s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "tokens":
        T, H, k, E, kind = case["T"], case["H"], case["k"], case["E"], case["kind"]
        e, S = 4 if case["fp32"] else 2, case["T"] * case["k"]
        rows, tok = S * H * e, T * H * e
        if kind == "sort":
            return dict(bytes=tok + rows + 4 * (3 * S + E + 1), flops=0)
        if kind == "sort_grad":
            return dict(bytes=rows + tok + 4 * S, flops=S * H)
        if kind == "return":
            return dict(bytes=rows + tok + 8 * S, flops=2 * S * H)
        return dict(bytes=2 * rows + tok + 12 * S, flops=3 * S * H)
    if case["op"] == "product":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        used, live = min(G, M), M - case["tail"]
        if G > M // 4:  # the expected number of groups that get a row
            used = G * (1.0 - (1.0 - 1.0 / G) ** live)
        per = N * K + 4 * _blocks(N) * _blocks(K)
        return dict(bytes=2 * live * K + used * per + (4 if case["fp32"] else 2) * M * N, flops=2 * live * N * K)
    T, H = case["T"], case["H"]
    r, kind = (4 if case["fp32"] else 2), case["kind"]
    gate = {"none": 0, "channel": 4 * H, "token": 4 * T, "element": 2 * T * H}[case["gate"]]
    if kind == "before":
        return dict(bytes=T * H * (r + 2) + 4 * (H + T), flops=4 * T * H)
    if kind == "before_grad":
        return dict(bytes=T * H * (3 * r + 2) + 4 * (2 * H + T), flops=9 * T * H)
    if kind == "after":
        return dict(bytes=T * H * (2 * r + 2 + 2 * case["next"]) + gate + 4 * (H + T) * (1 + case["next"]),
                    flops=T * H * (7 + 4 * case["next"]))
    return dict(bytes=T * H * (2 * r + 4 + (r + 2) * case["next"]) + 2 * gate + 4 * (2 * H + T) * (1 + case["next"]),
                flops=T * H * (12 + 9 * case["next"]))
