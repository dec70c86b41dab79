"""Tokens sorted by expert and back against plain 64-bit forms (needs a GB300)."""
import numpy as np
import pytest
import torch

from block_cases import F32, check, f64, half_ulp, sort_reference, taken

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32

# (T, H, E, k, dropped share, dtype): one token; both sort paths; partial warps and chunks; more
# experts than slots; one expert; every row length modulo the launch's thread counts
CASES = [
    (1, 8, 1, 1, 0.0, BF), (1, 2048, 512, 10, 0.0, BF), (8, 2048, 512, 10, 0.1, BF), (7, 24, 3, 3, 0.3, FP),
    (64, 1000, 40, 6, 0.2, FP), (204, 256, 16, 10, 0.05, BF), (205, 256, 16, 10, 0.05, BF), (300, 136, 1024, 16, 0.02, BF),
    (2500, 264, 33, 4, 0.0, FP), (1024, 64, 1, 1, 0.5, BF), (3000, 4104, 8, 2, 0.01, BF), (37, 16384, 5, 5, 0.1, FP),
    (3001, 2312, 8, 3, 0.1, BF), (700, 2056, 20, 9, 0.05, BF), (1300, 520, 9, 5, 0.1, FP), (2501, 1040, 7, 1, 0.2, BF),
    (6, 2600, 4, 1, 0.0, FP), (650, 2304, 11, 6, 0.1, BF),
]
IDS = lambda c: f"T{c[0]}_H{c[1]}_E{c[2]}_k{c[3]}_{'f32' if c[5] == FP else 'bf16'}"  # noqa: E731


def make(case, seed=3):
    T, H, E, k, drop, dt = case
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    if T > 2 and drop:
        ids[T // 2] = -1          # a padding token: none of its slots is routed
        ids[1, 0] = -2 ** 31
    w = torch.rand(T, k, generator=g) + 0.01
    x = torch.randn(T, H, generator=g).to(dt)
    ys = torch.randn(T * k, H, generator=g).to(dt)
    return ids, w, x, ys


def run_sort(moe, case, ids, x):
    T, H, E, k = case[:4]
    ws = moe.sort_workspace(T, E, k)
    got = moe.sort_tokens(x.cuda(), ids.cuda(), E, ws)
    return got, ws


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_sort_is_exact(cuda_lib, case):
    T, H, E, k, drop, dt = case
    ids, _, x, _ = make(case)
    (xs, offsets, sorted_slot, slot_pos), ws = run_sort(cuda_lib, case, ids, x)
    ro, rs, rp = sort_reference(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(sorted_slot.cpu().numpy(), rs)
    assert np.array_equal(slot_pos.cpu().numpy(), rp)
    want = x[torch.from_numpy(rs) // k]
    want[int(ro[E]):] = 0
    assert torch.equal(xs.cpu().view(torch.int16 if dt == BF else torch.int32), want.view(torch.int16 if dt == BF else torch.int32))
    assert cuda_lib.device_status(ws) == 0


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_return_and_gradients(cuda_lib, case):
    T, H, E, k, drop, dt = case
    moe = cuda_lib
    ids, w, x, ys = make(case)
    _, _, rp = sort_reference(ids, E)
    pos = torch.from_numpy(rp)
    dropped_rows = (-1 - pos[pos < 0]).long()
    ys[dropped_rows] = float("nan")                    # rows and weights of dropped slots are not read
    w = torch.where(pos < 0, torch.nan, w)
    d_pos, d_w, d_ys = pos.int().cuda(), w.cuda(), ys.cuda()
    t = taken(f64(ys), pos)
    wz = torch.where(pos < 0, 0.0, f64(w))
    ref, mag = (wz[..., None] * t).sum(1), (wz[..., None] * t).abs().sum(1)
    u = half_ulp(dt)
    check(moe.return_tokens(d_ys, d_pos, d_w), ref, u * ref.abs() + (k + 2) * F32 * mag, "out")
    shared = x.cuda()
    s64 = f64(x)
    check(moe.return_tokens(d_ys, d_pos, d_w, shared=shared), ref + s64,
          u * (ref + s64).abs() + (k + 3) * F32 * (mag + s64.abs()), "out with shared rows")
    ref, mag = t.sum(1), t.abs().sum(1)
    check(moe.sort_tokens_backward(d_ys, d_pos), ref, u * ref.abs() + k * F32 * mag, "dx")
    dys, dw = moe.return_tokens_backward(x.cuda(), d_ys, d_pos, d_w)
    want = torch.zeros(T * k, H, dtype=torch.float64)
    place = torch.where(pos >= 0, pos, -1 - pos).reshape(-1)
    want[place] = (wz[..., None] * f64(x)[:, None]).reshape(T * k, H)
    check(dys, want, (u + 2 * F32) * want.abs(), "dys")
    prod = t * f64(x)[:, None]
    check(dw, prod.sum(-1), (H + 8) * F32 * prod.abs().sum(-1), "dw")
    assert bool((dw[pos.cuda() < 0] == 0).all()) and bool((dys[dropped_rows.cuda()] == 0).all())


def test_gradient_against_differences(cuda_lib):
    """<gradients, direction> against a central difference of the 64-bit forward form, through both calls."""
    moe = cuda_lib
    T, H, E, k = 23, 64, 6, 3
    case = (T, H, E, k, 0.15, FP)
    ids, w, x, _ = make(case, seed=9)
    _, _, rp = sort_reference(ids, E)
    pos = torch.from_numpy(rp)
    g = torch.Generator().manual_seed(4)
    c = torch.randn(T, H, generator=g)                 # loss = <c, return(2 sort(x) + sort(x)^2)>
    dx_dir, dw_dir = torch.randn(T, H, generator=g).double(), torch.randn(T, k, generator=g).double()

    def loss(e):
        xs = (f64(x) + e * dx_dir)[:, None].expand(T, k, H)
        y = torch.where(pos[..., None] >= 0, 2 * xs + xs ** 2, 0.0)
        return float((f64(c) * ((f64(w) + e * dw_dir)[..., None] * y).sum(1)).sum())

    h = 1e-4
    want = (loss(h) - loss(-h)) / (2 * h)
    ws = moe.sort_workspace(T, E, k)
    xs, _, _, sp = moe.sort_tokens(x.cuda(), ids.cuda(), E, ws)
    ys = 2 * xs + xs ** 2
    dys, dw = moe.return_tokens_backward(c.cuda(), ys, sp, w.cuda())
    dx = moe.sort_tokens_backward(dys * (2 + 2 * xs), sp)
    got = float((f64(dx) * dx_dir).sum() + (f64(dw) * dw_dir).sum())
    scale = float((f64(dx) * dx_dir).abs().sum() + (f64(dw) * dw_dir).abs().sum())
    assert abs(got - want) <= 1e-6 * scale


def test_empty_batch_and_all_dropped(cuda_lib):
    moe = cuda_lib
    ws = moe.sort_workspace(4, 5, 2)
    x = torch.randn(0, 16, device="cuda")
    xs, offsets, ss, sp = moe.sort_tokens(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 5, ws)
    assert xs.shape == (0, 16) and offsets.tolist() == [0] * 6
    assert moe.return_tokens(xs, sp, torch.zeros(0, 2, device="cuda")).shape == (0, 16)
    ids = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    x = torch.full((4, 16), float("inf"), device="cuda")
    xs, offsets, ss, sp = moe.sort_tokens(x, ids, 5, ws)
    assert bool((xs == 0).all()) and offsets.tolist() == [0] * 6 and ss.tolist() == list(range(8))
    assert sp.flatten().tolist() == [-1 - i for i in range(8)]
    assert bool((moe.return_tokens(torch.full_like(xs, float("nan")), sp, torch.ones(4, 2, device="cuda")) == 0).all())
    assert bool((moe.sort_tokens_backward(torch.full_like(xs, float("nan")), sp) == 0).all())


@pytest.mark.parametrize("T", [5, 900])
def test_out_of_range_ids_are_dropped_and_reported(cuda_lib, T):
    moe = cuda_lib
    E, k = 7, 4
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    ids[T // 2, 1] = E
    ids[T - 1, 3] = 2 ** 31 - 1
    x = torch.randn(T, 32)
    (xs, offsets, ss, sp), ws = run_sort(moe, (T, 32, E, k), ids, x)
    ro, rs, rp = sort_reference(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), ro) and np.array_equal(sp.cpu().numpy(), rp)
    assert moe.device_status(ws) == -1 and moe.device_status(ws) == 0
    # positions out of range (not sort_tokens's) are taken as dropped by the calls that read rows
    bad = sp.clone()
    bad[0, 0] = T * k
    out = moe.return_tokens(torch.ones(T * k, 32, device="cuda"), bad, torch.ones(T, k, device="cuda"))
    n = int((bad[0] >= 0).sum()) - 1
    assert bool((out[0] == n).all())


def test_other_streams_graphs_and_repeats(cuda_lib):
    """The same bits on a side stream, in a captured graph and on repeated calls; a workspace of a larger batch."""
    moe = cuda_lib
    case = (1000, 256, 64, 8, 0.1, BF)
    ids, w, x, ys = make(case)
    T, H, E, k = case[:4]
    x, ids, w, ys = x.cuda(), ids.cuda(), w.cuda(), ys.cuda()
    ws = moe.sort_workspace(4096, 512, 16)

    def step():
        s = moe.sort_tokens(x, ids, E, ws)
        return (*s, moe.return_tokens(ys, s[3], w), *moe.return_tokens_backward(x, ys, s[3], w), moe.sort_tokens_backward(ys, s[3]))

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
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals(cuda_lib):
    moe = cuda_lib
    ws = moe.sort_workspace(16, 8, 2)
    x = torch.randn(16, 64, device="cuda")
    ids = torch.zeros(16, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        moe.sort_tokens(x.half(), ids, 8, ws)
    with pytest.raises(TypeError):
        moe.sort_tokens(x, ids.long(), 8, ws)
    with pytest.raises(ValueError):
        moe.sort_tokens(x, ids[:8], 8, ws)
    with pytest.raises(ValueError):
        moe.sort_tokens(torch.randn(64, 16, device="cuda").t(), ids, 8, ws)
    with pytest.raises(ValueError):
        moe.sort_tokens(x, ids, 8, ws, xs=torch.empty(16, 64, device="cuda"))
    for bad, status in (((x, ids, 0), -2), ((x, ids, 1025), -2), ((x[:, :12].contiguous(), ids, 8), -2),
                        ((x, torch.zeros(16, 17, dtype=torch.int32, device="cuda"), 8), -2)):
        with pytest.raises(moe.MoeError) as e:
            moe.sort_tokens(*bad, ws)
        assert e.value.status == status
    with pytest.raises(moe.MoeError) as e:
        moe.sort_tokens(x, ids, 8, ws[:256])
    assert e.value.status == -3
    odd = torch.randn(16 * 64 + 1, device="cuda")[1:].view(16, 64)       # not on 16 bytes
    with pytest.raises(moe.MoeError) as e:
        moe.sort_tokens(odd, ids, 8, ws)
    assert e.value.status == -1
    with pytest.raises(moe.MoeError):
        moe.sort_workspace(1 << 30, 8, 2)
    with pytest.raises(ValueError):
        moe.return_tokens(x, ids, torch.zeros(16, 2, device="cuda"))
