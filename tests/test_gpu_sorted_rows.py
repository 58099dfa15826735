"""Tokens sorted by expert and back, and the gradients of both, against plain 64-bit sums.

Tolerances, derived from the arithmetic and applied element by element: a result of a sum of n
terms held in fp32 and rounded once to its type differs from the exact sum by at most
(n + 1) 2^-23 times the sum of the terms' magnitudes (any order, one unit in the last place
per operation) plus half a step of the type, eps / 2 relative, plus half the type's smallest
subnormal.  Rows that are only moved are compared bit for bit."""
import numpy as np
import pytest
import torch

import synth
import w4a16_quantized_expert_b200 as moe
from gpu_cases import Case
from w4a16_quantized_expert_b200.device import DeviceLayer

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


def layer(H=256, E=16, k=2, T=64, top_p=0.0):
    z = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    f = torch.float32
    t = {"Wr": z(E, H, t=f), "bias": z(E, t=f), "g": z(E, 64, H // 2), "u": z(E, 64, H // 2), "d": z(E, H, 32),
         "sg": z(E, 64, t=f), "su": z(E, 64, t=f), "sd": z(E, H, t=f)}
    return DeviceLayer({"H": H, "I": 64, "I_sh": 0, "E": E, "k": k, "n_shared": 0, "scaling": 2.5,
                        "fmt": moe.MOE_FMT_INT4_ROWSCALE, "top_p": top_p}, max_tokens=T, tensors=t)


def routing(T, E, k, seed, drop=0.3):
    g = np.random.default_rng(seed)
    idx = np.argsort(g.random((T, E)) + np.linspace(0, 1, E), axis=1)[:, :k].astype(np.int32)
    keep = np.where(g.random(T) < drop, g.integers(0, k + 1, T), k)
    idx[np.arange(k)[None, :] >= keep[:, None]] = -1
    return idx


def sorted_by_hand(idx, E, align):
    """row_of, counts, seg_offsets of a stable sort, entry by entry."""
    counts = np.zeros(E, np.int32)
    for e in idx.reshape(-1):
        if 0 <= e < E:
            counts[e] += 1
    seg = np.zeros(E + 1, np.int32)
    for e in range(E):
        seg[e + 1] = seg[e] + -(-counts[e] // align) * align
    at, row_of = seg.copy(), np.full(idx.size, -1, np.int32)
    for a, e in enumerate(idx.reshape(-1)):
        if 0 <= e < E:
            row_of[a] = at[e]
            at[e] += 1
    return row_of.reshape(idx.shape), counts, seg


def rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def near(got, exact, magnitude, n, what):
    eps = torch.finfo(got.dtype).eps
    tol = eps / 2 * exact.abs() + (n + 1) * 2.0 ** -23 * magnitude + SMALLEST[got.dtype] / 2
    bad = ~((got.double() - exact).abs() <= tol * (1 + 1e-6))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, e.g. {got[bad][0]} for {exact[bad][0]}"


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def status(L):
    torch.cuda.synchronize()
    return moe.moe_get_device_status(L.handle)


SHAPES = [  # T, H, E, k
    (1, 64, 1, 1), (1, 6144, 256, 8), (2, 256, 16, 2), (5, 320, 7, 7), (16, 2048, 256, 8), (37, 256, 1024, 32),
    (63, 192, 40, 3), (257, 128, 16, 8), (300, 576, 256, 7), (1025, 64, 3, 2), (2050, 64, 256, 8), (300, 16384, 5, 1),
]


@pytest.mark.parametrize("T,H,E,k", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_sort_rows(T, H, E, k, dtype):
    L = layer(H, E, k, T)
    align = {"f16": 1, "bf16": 16, "f32": 5}[dtype]
    idx = routing(T, E, k, T + H)
    x = rand((T, H), DT[dtype], 1)
    n = L.sorted_rows(T, align)
    assert n == T * k + min(E, T * k) * (align - 1)
    guard = 3
    buf = torch.full((n + 2 * guard, H), -7.0, dtype=DT[dtype], device="cuda")
    rows = buf[guard:guard + n]
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (rows, torch.empty((T, k), **i32), torch.empty(E, **i32), torch.empty(E + 1, **i32))
    L.sort_tokens(x, torch.from_numpy(idx).cuda(), L.sort_workspace(T), align=align, out=out)
    row_of, counts, seg = sorted_by_hand(idx, E, align)
    assert np.array_equal(out[1].cpu().numpy(), row_of)
    assert np.array_equal(out[2].cpu().numpy(), counts)
    assert np.array_equal(out[3].cpu().numpy(), seg)
    want = torch.full((n, H), -7.0, dtype=DT[dtype], device="cuda")
    want[:seg[E]] = 0
    a = torch.from_numpy(np.flatnonzero(row_of.reshape(-1) >= 0)).cuda()
    want[torch.from_numpy(row_of.reshape(-1)).cuda().long()[a]] = x[a // k]
    assert torch.equal(bits(rows), bits(want)), "rows, padding or what lies behind them"
    assert bool((buf[:guard] == -7).all()) and bool((buf[guard + n:] == -7).all())
    assert status(L) == moe.MOE_OK


def test_sort_equals_group_and_moves_every_bit():
    """row_of is the inverse of moe_group's perm; NaN payloads, infinities and -0 move as they are."""
    T, H, E, k = 200, 128, 32, 4
    L = layer(H, E, k, T)
    idx = torch.from_numpy(routing(T, E, k, 3)).cuda()
    ws = L.workspace(T)
    x = torch.randint(-2 ** 15, 2 ** 15, (T, H), device="cuda", dtype=torch.int32).to(torch.int16).view(torch.float16)
    rows, row_of, counts, seg = L.sort_tokens(x, idx, ws)
    c, o, perm, _, _ = L.group(idx, T, ws)
    n = int(o[-1])
    assert torch.equal(counts, c) and torch.equal(seg, o)
    assert torch.equal(row_of.reshape(-1)[perm[:n].long()], torch.arange(n, device="cuda", dtype=torch.int32))
    assert torch.equal(bits(rows[:n]), bits(x[perm[:n].long() // k]))


def test_sort_shares_the_layers_workspace():
    """The layer's own workspace serves and its counters stay zero: moe_forward is unchanged by a
    sort in between."""
    case = Case(synth.WORKLOADS["tiny"], T=37, max_tokens=64)
    ws = case.dev.workspace(37)
    y0 = case.dev.forward(case.x_dev, ws)
    idx = torch.from_numpy(routing(37, 16, 2, 5)).cuda()
    r0 = case.dev.sort_tokens(case.x_dev.view(torch.float16), idx, ws, align=8)
    y1 = case.dev.forward(case.x_dev, ws)
    r1 = case.dev.sort_tokens(case.x_dev.view(torch.float16), idx, case.dev.sort_workspace(37), align=8)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1)
    live = int(r0[3][-1])
    for a, b in zip(r0[1:], r1[1:]):
        assert torch.equal(a, b)
    assert torch.equal(bits(r0[0][:live]), bits(r1[0][:live]))


def test_sort_bad_indices_are_dropped_and_recorded():
    T, H, E, k = 40, 64, 8, 2
    L = layer(H, E, k, T)
    idx = routing(T, E, k, 9, drop=0)
    bad = idx.copy()
    bad[3, 0], bad[7, 1], bad[11, 0] = E, -2, 2 ** 31 - 1
    _, row_of, counts, seg = L.sort_tokens(rand((T, H), torch.float16, 2), torch.from_numpy(bad).cuda(),
                                           L.sort_workspace(T))
    assert status(L) == moe.MOE_ERR_DEVICE_BOUNDS
    want = sorted_by_hand(bad, E, 1)
    for g, w in zip((row_of, counts, seg), want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert status(L) == moe.MOE_OK


def test_sort_no_token():
    L = layer(64, 8, 2, 4)
    counts = torch.full((8,), 9, dtype=torch.int32, device="cuda")
    seg = torch.full((9,), 9, dtype=torch.int32, device="cuda")
    ws = L.sort_workspace(0)
    moe.moe_sort_tokens(L.handle, None, 0, 0, None, 0, 16, None, 0, None, counts.data_ptr(), seg.data_ptr(),
                        ws.data_ptr(), ws.numel())
    assert not counts.any() and not seg.any()
    # every entry dropped: no rows, all gradients and sums empty
    idx = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    x = rand((4, 64), torch.float16, 1)
    rows, row_of, counts, seg = L.sort_tokens(x, idx, L.sort_workspace(4), align=4)
    assert bool((row_of == -1).all()) and not seg.any()
    w = torch.ones((4, 2), device="cuda")
    assert not L.sort_tokens_backward(rows, row_of).any()
    assert not L.unsort_tokens(rows, row_of, w).any()
    assert not L.unsort_tokens_backward(x, rows, row_of, w)[1].any()


def plan(T, E, k, align, seed, drop=0.3):
    idx = routing(T, E, k, seed, drop)
    row_of, counts, seg = sorted_by_hand(idx, E, align)
    return (torch.from_numpy(row_of).cuda(), torch.from_numpy(counts).cuda(), torch.from_numpy(seg).cuda())


PAIRS = [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "f16"), ("f16", "f32"), ("bf16", "f16"),
         ("f32", "bf16"), ("f16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("T,H,E,k", SHAPES)
@pytest.mark.parametrize("pair", range(3))
def test_back_and_its_adjoint(T, H, E, k, pair):
    """moe_unsort_tokens (with and without a shared row) and moe_sort_tokens_backward."""
    rt, yt = PAIRS[(SHAPES.index((T, H, E, k)) + 3 * pair) % 9]
    align = 4
    L = layer(H, E, k, T)
    row_of, counts, seg = plan(T, E, k, align, T)
    n = L.sorted_rows(T, align)
    rows = rand((n, H), DT[rt], 3)
    live_rows = torch.zeros(n, dtype=torch.bool, device="cuda")
    live_rows[row_of[row_of >= 0].long()] = True
    rows[~live_rows] = float("nan")                          # padding is not read
    w = torch.rand((T, k), device="cuda") + 0.1
    w[0, 0] = 0.0                                            # a weight of zero skips its row
    if row_of[0, 0] >= 0:
        rows[int(row_of[0, 0])] = float("inf")
    shared = rand((T, H), torch.float32, 4) if pair != 1 else None
    y = torch.full((T + 2, H + 8), 5.0, dtype=DT[yt], device="cuda")
    got = L.unsort_tokens(rows, row_of, w, y_shared=shared, y=y[1:T + 1, :H])
    live = (row_of >= 0) & (w != 0)
    wd = torch.where(live, w, torch.zeros_like(w)).double()
    v = torch.where(live[..., None], rows[row_of.clamp(min=0).long()].double(), torch.zeros((), device="cuda").double())
    exact, mag = (wd[..., None] * v).sum(1), (wd[..., None] * v.abs()).sum(1)
    if shared is not None:
        exact, mag = exact + shared.double(), mag + shared.double().abs()
    near(got, exact, mag, 2 * k + 1, "y")
    assert bool((y[0] == 5).all()) and bool((y[T + 1] == 5).all()) and bool((y[:, H:] == 5).all())
    if row_of[0, 0] >= 0:
        rows[int(row_of[0, 0])] = 1.0
    dx = L.sort_tokens_backward(rows, row_of, dx=torch.empty((T, H), dtype=DT[yt], device="cuda"))
    on = row_of >= 0
    v = torch.where(on[..., None], rows[row_of.clamp(min=0).long()].double(), torch.zeros((), device="cuda").double())
    near(dx, v.sum(1), v.abs().sum(1), k, "dx")
    assert status(L) == moe.MOE_OK


@pytest.mark.parametrize("T,H,E,k", SHAPES)
@pytest.mark.parametrize("pair", range(3))
def test_gradients_of_rows_and_weights(T, H, E, k, pair):
    rt, dt = PAIRS[(SHAPES.index((T, H, E, k)) + 3 * pair) % 9]
    align = 3
    L = layer(H, E, k, T)
    row_of, counts, seg = plan(T, E, k, align, T + 1)
    n = L.sorted_rows(T, align)
    rows = rand((n, H), DT[rt], 5)
    wide = rand((T, H + 16), DT[dt], 6)
    dy = wide[:, :H]
    w = torch.rand((T, k), device="cuda") + 0.1
    w[T // 2, 0] = 0.0
    drows = torch.full((n, H), 9.0, dtype=DT[rt], device="cuda")
    dw = torch.full((T, k), 9.0, device="cuda")
    L.unsort_tokens_backward(dy, rows, row_of, w, counts, seg, out=(drows, dw))
    on = row_of >= 0
    at = row_of.clamp(min=0).long()
    g = w.double()[..., None] * dy.double()[:, None, :]
    near(drows[at[on]], g[on], g[on].abs(), 0, "drows")
    prod = dy.double()[:, None, :] * rows[at].double()
    prod[~on] = 0
    near(dw, prod.sum(2), prod.abs().sum(2), H // 32 + 16, "dw")   # (a lane adds at most H / 32 products)
    mask = torch.zeros(n, dtype=torch.bool, device="cuda")
    mask[at[on]] = True
    end = int(seg[-1])
    assert not drows[:end][~mask[:end]].any(), "padding rows are zeroed"
    assert bool((drows[end:] == 9).all()), "rows behind the last segment are left alone"
    again = torch.full_like(drows, 9.0)
    L.unsort_tokens_backward(dy, rows, row_of, w, out=(again, dw))
    assert bool((again[~mask] == 9).all()) and torch.equal(bits(again[mask]), bits(drows[mask]))
    assert status(L) == moe.MOE_OK


def test_gradient_against_differences():
    """y is linear in the rows and in the weights, so differences of any length are exact up to
    rounding: <dy, y(+d) - y(-d)> / 2 against <gradient, d>, all held in fp32."""
    T, H, E, k, align = 33, 256, 16, 4, 2
    L = layer(H, E, k, T)
    row_of, counts, seg = plan(T, E, k, align, 2)
    n = L.sorted_rows(T, align)
    rows, d_rows = rand((n, H), torch.float32, 1), rand((n, H), torch.float32, 2)
    w, d_w = torch.rand((T, k), device="cuda") + 0.5, torch.rand((T, k), device="cuda") * 0.25
    dy = rand((T, H), torch.float32, 3)
    drows, dw = torch.zeros((n, H), device="cuda"), torch.zeros((T, k), device="cuda")
    L.unsort_tokens_backward(dy, rows, row_of, w, counts, seg, out=(drows, dw))
    f = lambda r, v: (L.unsort_tokens(r, row_of, v).double() * dy.double()).sum()  # noqa: E731
    size = float(dy.double().norm() * rows.double().norm())   # every rounding is 2^-24 of such products
    assert abs(float((f(rows + d_rows, w) - f(rows - d_rows, w)) / 2 - (drows.double() * d_rows.double()).sum())) \
        <= 16 * 2.0 ** -24 * size * 4
    assert abs(float((f(rows, w + d_w) - f(rows, w - d_w)) / 2 - (dw.double() * d_w.double()).sum())) \
        <= 16 * 2.0 ** -24 * size * 4
    d_x = rand((T, H), torch.float32, 5)
    idx = torch.from_numpy(routing(T, E, k, 2)).cuda()
    gr = rand((n, H), torch.float32, 6)
    dx = L.sort_tokens_backward(gr, row_of)
    out = L.sort_tokens(d_x, idx, L.sort_workspace(T), align=align,
                        out=(torch.zeros((n, H), device="cuda"), torch.empty_like(row_of), torch.empty_like(counts),
                             torch.empty_like(seg)))
    assert torch.equal(out[1], row_of)
    live = int(seg[-1])
    lhs, rhs = (out[0][:live].double() * gr[:live].double()).sum(), (dx.double() * d_x.double()).sum()
    assert abs(float(lhs - rhs)) <= (k + 2) * 2.0 ** -23 * float(gr.double().norm() * d_x.double().norm()) * k


def test_bad_positions_are_skipped_and_recorded():
    T, H, E, k = 8, 64, 4, 2
    L = layer(H, E, k, T)
    row_of, counts, seg = plan(T, E, k, 1, 1, drop=0)
    rows = rand((T * k, H), torch.float32, 1)
    w = torch.ones((T, k), device="cuda")
    bad = row_of.clone()
    bad[2, 0], bad[5, 1] = T * k, -5
    good = torch.where((bad < 0) | (bad >= T * k), torch.full_like(bad, -1), bad)
    for f in (lambda r: L.unsort_tokens(rows, r, w), lambda r: L.sort_tokens_backward(rows, r),
              lambda r: L.unsort_tokens_backward(rows[:T], rows, r, w,
                                                 out=(torch.zeros_like(rows), torch.zeros_like(w)))[0],
              lambda r: L.unsort_tokens_backward(rows[:T], rows, r, w,
                                                 out=(torch.zeros_like(rows), torch.zeros_like(w)))[1]):
        a = f(bad)
        assert status(L) == moe.MOE_ERR_DEVICE_BOUNDS
        assert torch.equal(a, f(good))
        assert status(L) == moe.MOE_OK
    # segments that do not fit the rows are not zeroed
    far = seg.clone()
    far[-1] = T * k + 1
    L.unsort_tokens_backward(rows[:T], rows, row_of, w, counts, far)
    assert status(L) == moe.MOE_ERR_DEVICE_BOUNDS


def test_refusals():
    T, H, E, k = 8, 64, 4, 2
    L = layer(H, E, k, T)
    x = rand((T, H), torch.float16, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, row_of = torch.zeros((T, k), **i32), torch.full((T, k), -1, **i32)
    counts, seg = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    rows = torch.empty((64, H), dtype=torch.float16, device="cuda")
    ws = L.sort_workspace(T)
    w = torch.ones((T, k), device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731

    def refused(code, fn, *args):
        with pytest.raises(moe.MoeError) as e:
            fn(L.handle, *args)
        assert e.value.code == code

    sort = [p(x), 0, H, p(idx), T, 4, p(rows), 64, p(row_of), p(counts), p(seg), p(ws), ws.numel()]
    for at, v, code in [(0, None, 1), (0, p(x) + 2, 1), (1, 3, 1), (1, -1, 1), (2, H - 8, 1), (2, H + 4, 1), (3, None, 1),
                        (4, T + 1, 1), (4, -1, 1), (5, 0, 1), (5, 1025, 1), (6, None, 1), (6, p(rows) + 8, 1),
                        (7, T * k + 4 * 3 - 1, 3), (8, None, 1), (9, None, 1), (10, None, 1), (11, None, 3),
                        (11, p(ws) + 16, 3), (12, ws.numel() - 1, 3)]:
        a = list(sort)
        a[at] = v
        refused(code, moe.moe_sort_tokens, *a)
    back = [p(rows), 0, 64, p(row_of), T, p(x), 0, H]
    for at, v in [(0, None), (0, p(rows) + 4), (1, 9), (2, 2 ** 31), (3, None), (4, T + 1), (5, None), (6, 5), (7, H - 1)]:
        a = list(back)
        a[at] = v
        refused(1, moe.moe_sort_tokens_backward, *a)
    un = [p(rows), 0, 64, p(row_of), p(w), None, T, p(x), 0, H]
    for at, v in [(0, None), (3, None), (4, None), (5, p(w) + 4), (6, -1), (7, None), (8, -1), (9, 0)]:
        a = list(un)
        a[at] = v
        refused(1, moe.moe_unsort_tokens, *a)
    ub = [p(x), 0, H, p(rows), 0, 64, p(row_of), p(w), None, None, T, p(rows), p(w)]
    for at, v in [(0, None), (2, H + 1), (3, None), (6, None), (7, None), (8, p(counts)), (9, p(seg)), (10, T + 1),
                  (11, None), (12, None)]:
        a = list(ub)
        a[at] = v
        refused(1, moe.moe_unsort_tokens_backward, *a)
    assert L.sorted_rows(T + 1) == 0 and L.sorted_rows(T, 0) == 0 and L.sorted_rows(T, 1025) == 0
    with pytest.raises(ValueError):
        L.sort_tokens(x.t().contiguous().t(), idx, ws)          # columns, not rows
    with pytest.raises(ValueError):
        L.sort_tokens(x.double(), idx, ws)
    with pytest.raises(ValueError):
        L.sort_tokens(x, idx.long(), ws)
    assert status(L) == moe.MOE_OK


def test_captured_and_replayed_on_another_stream():
    T, H, E, k, align = 50, 256, 16, 4, 8
    L = layer(H, E, k, T)
    n = L.sorted_rows(T, align)
    i32 = dict(dtype=torch.int32, device="cuda")
    x, dy = rand((T, H), torch.bfloat16, 1), rand((T, H), torch.bfloat16, 2)
    idx = torch.from_numpy(routing(T, E, k, 1)).cuda()
    w = torch.rand((T, k), device="cuda")
    out = (torch.zeros((n, H), dtype=torch.bfloat16, device="cuda"), torch.empty((T, k), **i32),
           torch.empty(E, **i32), torch.empty(E + 1, **i32))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    grads = (torch.zeros_like(out[0]), torch.empty_like(w))
    ws = L.sort_workspace(T)

    def step():
        L.sort_tokens(x, idx, ws, align=align, out=out)
        L.unsort_tokens(out[0], out[1], w, y=y)
        L.unsort_tokens_backward(dy, out[0], out[1], w, out[2], out[3], out=grads)
        L.sort_tokens_backward(grads[0], out[1], dx=dx)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    for seed in (7, 8):
        x.copy_(rand((T, H), torch.bfloat16, seed))
        idx.copy_(torch.from_numpy(routing(T, E, k, seed)).cuda())
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, grads[1], out[1])]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, dx, grads[1], out[1])):
            assert torch.equal(a, b)
    assert status(L) == moe.MOE_OK


def test_offsets_past_32_bits():
    """Sorted rows of more than 2^31 elements: every token comes back from its eight copies.
    (Eight times an eighth of a value, summed in fp32, is the value itself; of the zeros, -0 comes
    back as +0, as a sum that starts at +0 does: +0 + -0 = +0.)"""
    T, H, E, k = 44000, 6144, 64, 8
    L = layer(H, E, k, T)
    x = rand((T, H), torch.float16, 1)
    idx = torch.randint(0, E - k + 1, (T, 1), device="cuda", dtype=torch.int32) + \
        torch.arange(k, device="cuda", dtype=torch.int32)
    rows, row_of, counts, seg = L.sort_tokens(x, idx, L.sort_workspace(T))
    assert rows.numel() > 2 ** 31 and int(seg[-1]) == T * k
    assert torch.equal(torch.sort(row_of.reshape(-1))[0], torch.arange(T * k, device="cuda", dtype=torch.int32))
    w = torch.full((T, k), 0.125, device="cuda")
    y = L.unsort_tokens(rows, row_of, w)
    assert torch.equal(y, x)
    drows, dw = L.unsort_tokens_backward(x, rows, row_of, w)
    last = row_of[-1].long()
    assert torch.equal(bits(drows[last]), bits((x[-1].float() * 0.125).half().expand(k, H)))
    norm = (x.double() ** 2).sum(1, keepdim=True).expand(T, k)
    near(dw, norm, norm, H // 32 + 16, "dw")
    dx = L.sort_tokens_backward(drows, row_of)
    exact = drows[row_of.long()[-1000:]].double().sum(1)
    near(dx[-1000:], exact, exact.abs(), k, "dx")
    assert status(L) == moe.MOE_OK


@pytest.mark.parametrize("T,E,k", [(64, 256, 8), (128, 1024, 8), (129, 256, 8), (256, 16, 8), (257, 16, 8), (2048, 256, 8),
                                   (2049, 256, 8)])
def test_sort_at_the_borders_of_its_paths(T, E, k):
    """1024 assignments (one launch), 2048 (one chunk) and 16384 (one cluster), and one token more."""
    H, align = 64, 4
    L = layer(H, E, k, T)
    idx = routing(T, E, k, T)
    x = rand((T, H), torch.bfloat16, 1)
    rows, row_of, counts, seg = L.sort_tokens(x, torch.from_numpy(idx).cuda(), L.sort_workspace(T), align=align)
    want = sorted_by_hand(idx, E, align)
    for g, w in zip((row_of, counts, seg), want):
        assert np.array_equal(g.cpu().numpy(), w)
    a = torch.from_numpy(np.flatnonzero(want[0].reshape(-1) >= 0)).cuda()
    assert torch.equal(bits(rows[row_of.reshape(-1)[a].long()]), bits(x[a // k]))


def test_two_streams_at_once():
    """Calls of one handle on two streams, each with a workspace of its own."""
    T, H, E, k = 700, 512, 32, 4
    L = layer(H, E, k, T)
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [rand((T, H), torch.float16, i) for i in range(2)]
    ids = [torch.from_numpy(routing(T, E, k, i)).cuda() for i in range(2)]
    wss = [L.sort_workspace(T) for _ in range(2)]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i] = L.sort_tokens(xs[i], ids[i], wss[i], out=outs[i])
    torch.cuda.synchronize()
    for i in range(2):
        row_of, counts, seg = sorted_by_hand(ids[i].cpu().numpy(), E, 1)
        assert np.array_equal(outs[i][1].cpu().numpy(), row_of)
        a = torch.from_numpy(np.flatnonzero(row_of.reshape(-1) >= 0)).cuda()
        assert torch.equal(bits(outs[i][0][outs[i][1].reshape(-1)[a].long()]), bits(xs[i][a // k]))
    assert status(L) == moe.MOE_OK
