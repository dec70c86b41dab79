"""The norms before and after a block against plain 64-bit forms (needs a GB300)."""
import pytest
import torch

from block_cases import F32, after_reference, check, f64, gate_factor, half_ulp, norm_grad, rstd_of

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
EPS = 1e-6

# (T, H, residual type, branch type, gate, next norm, weight offset)
CASES = [
    (1, 8, BF, BF, "none", True, 0.0), (1, 2048, BF, BF, "channel", True, 0.0), (8, 2048, BF, FP, "token", True, 1.0),
    (33, 1000, FP, BF, "element", False, 0.0), (700, 264, FP, FP, "channel", True, 1.0), (5, 4096, BF, BF, "element", True, 0.0),
    (64, 4104, FP, BF, "channel", True, 0.0), (19, 16384, BF, FP, "token", True, 0.0), (3, 8200, FP, FP, "none", False, 1.0),
    (2000, 96, BF, BF, "token", False, 0.0), (1301, 520, BF, BF, "channel", False, 0.0),
    (701, 1288, BF, BF, "channel", True, 0.0), (650, 2080, FP, FP, "token", True, 1.0), (37, 2504, BF, FP, "channel", True, 0.0),
    (161, 3200, BF, BF, "element", True, 0.0), (21, 4608, FP, FP, "element", True, 0.0), (170, 776, FP, BF, "element", True, 1.0),
    (9, 6152, BF, BF, "channel", True, 0.0), (6, 9208, FP, FP, "element", True, 0.0), (5, 9224, BF, BF, "element", True, 1.0),
    (2500, 1096, FP, BF, "none", False, 0.0), (2501, 1288, BF, BF, "none", True, 0.0),
]
IDS = lambda c: f"T{c[0]}_H{c[1]}_{c[4]}{'_next' if c[5] else ''}"  # noqa: E731


def make(case, seed=1):
    T, H, rt, yt, kind, nxt, off = case
    g = torch.Generator().manual_seed(seed + T + H)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=(2 * r(T, H)).to(rt), y=(0.5 * r(T, H)).to(yt), w=1 - off + 0.2 * r(H), wn=1 - off + 0.2 * r(H),
             dout=r(T, H).to(rt), dn=r(T, H).to(BF))
    d["gate"] = {"none": None, "channel": 0.5 * r(H), "token": 0.5 * r(T, 1), "element": (0.5 * r(T, H)).to(BF)}[kind]
    if T > 4:
        d["y"][2] = 0.0
        d["x"][3] = 0.0
    return d


def cuda(t):
    return None if t is None else t.cuda()


def row_slack(H):
    """Relative error of rstd and of a row sum: H fp32 products summed by threads and shuffles."""
    return (H / 256 + 24) * F32


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(cuda_lib, case):
    T, H, rt, yt, kind, nxt, off = case
    moe = cuda_lib
    d = make(case)
    a, b = 0.75, 1.5
    slack = row_slack(H)
    n, rstd = moe.norm_before(d["x"].cuda(), d["w"].cuda(), eps=EPS, weight_offset=off)
    x, w = f64(d["x"]), f64(d["w"]) + off
    r = rstd_of(x, EPS)
    check(rstd, r, slack * r, "rstd")
    ref = x * r[:, None] * w
    check(n, ref, (2.0 ** -8 + slack) * ref.abs() + 4 * F32 * (x * r[:, None]).abs() * (f64(d["w"]).abs() + off), "n")
    out, n2, ry, rn = moe.norm_after(d["y"].cuda(), d["x"].cuda(), d["w"].cuda(), gate=cuda(d["gate"]),
                                     w_next=d["wn"].cuda() if nxt else None, residual_scale=a, branch_scale=b, eps=EPS,
                                     weight_offset=off)
    y = f64(d["y"])
    check(ry, rstd_of(y, EPS), slack * rstd_of(y, EPS), "rstd of y")
    ref, mag = after_reference(y, x, w, d["gate"], a, b, EPS)
    extra = 4 * F32 * (b * gate_factor(d["gate"], T, H) * y * rstd_of(y, EPS)[:, None]).abs() * (f64(d["w"]).abs() + off)
    check(out, ref, half_ulp(rt) * ref.abs() + (slack + 4 * F32) * mag + extra, "out")
    if not nxt:
        assert n2 is None and rn is None
        return
    separate, r_sep = moe.norm_before(out, d["wn"].cuda(), eps=EPS, weight_offset=off)
    assert torch.equal(n2, separate) and torch.equal(rn, r_sep)     # the fused norm is that of the stored stream
    o = f64(out)
    check(rn, rstd_of(o, EPS), slack * rstd_of(o, EPS), "rstd of out")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradients(cuda_lib, case):
    T, H, rt, yt, kind, nxt, off = case
    moe = cuda_lib
    d = make(case)
    a, b = 0.75, 1.5
    slack, cols = row_slack(H) + 8 * F32, (T / 100 + 64) * F32
    x, y, dout, dn = (f64(d[k]) for k in ("x", "y", "dout", "dn"))
    w, wn = f64(d["w"]) + off, f64(d["wn"]) + off
    ws = moe.norm_workspace(T, H)
    rx = rstd_of(x, EPS).float()
    dx, dw = moe.norm_before_backward(d["dn"].cuda(), d["x"].cuda(), d["w"].cuda(), rx.cuda(), ws, dresidual=d["dout"].cuda(),
                                      weight_offset=off)
    ref, refw, mag, magw = norm_grad(dn, x, w, rx.double())
    check(dx, ref + dout, half_ulp(rt) * (ref + dout).abs() + slack * (mag + dout.abs()), "dx of before")
    check(dw, refw, cols * magw, "dw of before")
    plain, _ = moe.norm_before_backward(d["dn"].cuda(), d["x"].cuda(), d["w"].cuda(), rx.cuda(), ws, weight_offset=off)
    check(plain, ref, half_ulp(rt) * ref.abs() + slack * mag, "dx of before without a residual")

    ry = rstd_of(y, EPS).float()
    more = dict(dn=d["dn"].cuda(), out=d["x"].cuda(), w_next=d["wn"].cuda(), rstd_next=rx.cuda()) if nxt else {}
    dy, dx, dw, dgate, dwn = moe.norm_after_backward(d["dout"].cuda(), d["y"].cuda(), d["w"].cuda(), ry.cuda(), ws,
                                                     gate=cuda(d["gate"]), residual_scale=a, branch_scale=b,
                                                     weight_offset=off, **more)
    t, tm = dout, dout.abs()
    if nxt:
        gn, refn, magn, magwn = norm_grad(dn, x, wn, rx.double())
        t, tm = t + gn, tm + magn
        check(dwn, refn, cols * magwn, "dw of the next norm")
    else:
        assert dwn is None
    check(dx, a * t, half_ulp(rt) * (a * t).abs() + slack * a * tm, "dx of after")
    gf = gate_factor(d["gate"], T, H)
    v = y * ry.double()[:, None] * w
    ref, _, mag, _ = norm_grad(b * t * gf, y, w, ry.double())
    magt = norm_grad(b * tm * gf.abs(), y.abs(), w.abs(), ry.double())
    check(dy, ref, half_ulp(yt) * ref.abs() + 2 * slack * (mag + magt[2]), "dy")
    check(dw, (b * t * gf * y * ry.double()[:, None]).sum(0), (cols + 2 * slack) * magt[3], "dw of after")
    if kind == "none":
        assert dgate is None
        return
    per, perm = b * t * v, b * tm * v.abs()
    if kind == "element":
        check(dgate, per, 2.0 ** -8 * per.abs() + 2 * slack * perm, "dgate")
    elif kind == "channel":
        check(dgate, per.sum(0), (cols + 2 * slack) * perm.sum(0), "dgate")
    else:
        check(dgate, per.sum(1, keepdim=True), 3 * slack * perm.sum(1, keepdim=True), "dgate")


@pytest.mark.parametrize("kind", ["channel", "token", "element"])
def test_gradients_against_differences(cuda_lib, kind):
    """<gradients, direction> of a loss on both outputs against a central difference of the 64-bit form."""
    moe = cuda_lib
    T, H = 13, 72
    d = make((T, H, FP, FP, kind, True, 0.0), seed=5)
    a, b = 0.9, 1.1
    g = torch.Generator().manual_seed(3)
    c1, c2 = d["dout"], d["dn"]
    names = ["x", "y", "w", "wn", "gate"]
    direction = {k: torch.randn(d[k].shape, generator=g).double() for k in names}

    def loss(e):
        v = {k: f64(d[k]) + e * direction[k] for k in names}
        out, _ = after_reference(v["y"], v["x"], v["w"], v["gate"], a, b, EPS)
        return float((f64(c1) * out).sum() + (f64(c2) * out * rstd_of(out, EPS)[:, None] * v["wn"]).sum())

    h = 1e-5
    want = (loss(h) - loss(-h)) / (2 * h)
    gate = d["gate"].cuda()
    out, n, ry, rn = moe.norm_after(d["y"].cuda(), d["x"].cuda(), d["w"].cuda(), gate=gate, w_next=d["wn"].cuda(),
                                    residual_scale=a, branch_scale=b, eps=EPS)
    ws = moe.norm_workspace(T, H)
    dy, dx, dw, dgate, dwn = moe.norm_after_backward(c1.cuda(), d["y"].cuda(), d["w"].cuda(), ry, ws, gate=gate, dn=c2.cuda(),
                                                     out=out, w_next=d["wn"].cuda(), rstd_next=rn, residual_scale=a,
                                                     branch_scale=b)
    grads = dict(x=dx, y=dy, w=dw, wn=dwn, gate=dgate)
    terms = {k: f64(grads[k]) * direction[k] for k in names}
    got = sum(float(t.sum()) for t in terms.values())
    # fp32 gradients, but for an element gate's, which is bf16
    bound = sum((2.0 ** -8 if k == "gate" and kind == "element" else 2e-5) * float(t.abs().sum()) for k, t in terms.items())
    assert abs(got - want) <= bound + 1e-7 * abs(want)


def test_rows_that_are_zero_or_not_finite(cuda_lib):
    moe = cuda_lib
    H = 256
    x = torch.randn(5, H)
    x[1] = 0.0
    x[2, 3] = float("nan")
    x[3, 4] = float("inf")
    w = torch.ones(H)
    n, rstd = moe.norm_before(x.cuda(), w.cuda())
    n, rstd = n.cpu().float(), rstd.cpu()
    assert bool((n[1] == 0).all()) and float(rstd[1]) == pytest.approx(1e3, rel=1e-5)
    assert bool(n[2].isnan().all()) and float(rstd[3]) == 0.0 and bool(n[3, 4].isnan()) and bool((n[3, :4] == 0).all())
    assert bool(n[[0, 4]].isfinite().all())            # the other rows are untouched
    out, _, _, _ = moe.norm_after(x.cuda(), torch.ones(5, H, device="cuda"), w.cuda(), residual_scale=2.0)
    assert bool((out[1] == 2.0).all()) and bool(out[[0, 4]].isfinite().all())


def test_no_tokens(cuda_lib):
    moe = cuda_lib
    H = 64
    e, w = torch.empty(0, H, device="cuda"), torch.ones(H, device="cuda")
    r = torch.empty(0, device="cuda")
    ws = moe.norm_workspace(0, H)
    assert moe.norm_before(e, w)[0].shape == (0, H) and moe.norm_after(e, e, w, w_next=w)[1].shape == (0, H)
    _, dw = moe.norm_before_backward(e.bfloat16(), e, w, r, ws)
    assert bool((dw == 0).all())
    _, _, dw, dg, dwn = moe.norm_after_backward(e, e, w, r, ws, gate=w, dn=e.bfloat16(), out=e, w_next=w, rstd_next=r)
    assert bool((dw == 0).all()) and bool((dg == 0).all()) and bool((dwn == 0).all())


def test_in_place_streams_graphs_and_repeats(cuda_lib):
    moe = cuda_lib
    case = (900, 512, BF, BF, "channel", True, 0.0)
    d = {k: cuda(v) for k, v in make(case).items()}
    ws = moe.norm_workspace(2000, 512)

    def step(stream=None):
        out, n, ry, rn = moe.norm_after(d["y"], d["x"], d["w"], gate=d["gate"], w_next=d["wn"], stream=stream)
        return (out, n, ry, rn, *moe.norm_after_backward(d["dout"], d["y"], d["w"], ry, ws, gate=d["gate"], dn=d["dn"],
                                                         out=out, w_next=d["wn"], rstd_next=rn, stream=stream))

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for p, q, r in zip(first, second, third):
        assert torch.equal(p, q) and torch.equal(p, r)
    x = d["x"].clone()
    moe.norm_after(d["y"], x, d["w"], gate=d["gate"], out=x)
    assert torch.equal(x, first[0])


def test_refusals(cuda_lib):
    moe = cuda_lib
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    r, ws = torch.ones(4, device="cuda"), moe.norm_workspace(4, 64)
    with pytest.raises(TypeError):
        moe.norm_before(x.half(), w)
    with pytest.raises(TypeError):
        moe.norm_before(x, w.bfloat16())
    with pytest.raises(ValueError):
        moe.norm_before(x, w[:32])
    with pytest.raises(ValueError):
        moe.norm_after(x, x, w, gate=torch.ones(5, device="cuda"))
    with pytest.raises(TypeError):
        moe.norm_after(x, x, w, gate=torch.ones(4, 64, device="cuda"))
    with pytest.raises(ValueError):
        moe.norm_after(x, x, w, n=torch.empty(4, 64, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        moe.norm_after_backward(x, x, w, r, ws, w_next=w)
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(weight_offset=float("inf"))):
        with pytest.raises(moe.MoeError) as e:
            moe.norm_before(x, w, **bad)
        assert e.value.status == -1
    with pytest.raises(moe.MoeError) as e:
        moe.norm_before(torch.randn(4, 60, device="cuda"), torch.ones(60, device="cuda"))
    assert e.value.status == -2
    with pytest.raises(moe.MoeError) as e:
        moe.norm_before(torch.randn(1, 16392, device="cuda"), torch.ones(16392, device="cuda"))
    assert e.value.status == -2
    with pytest.raises(moe.MoeError) as e:
        moe.norm_before_backward(x.bfloat16(), x, w, r, ws[:256])
    assert e.value.status == -3
