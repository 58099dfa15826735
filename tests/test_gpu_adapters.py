"""Low-rank adapters of many requests and their gradients against plain 64-bit products.

Tolerances, derived from the arithmetic and applied element by element.  A sum of n products
held in fp32 is off by at most n 2^-23 times the sum of their magnitudes (any order, one unit
in the last place per operation).  Where z or dz enters a second product it may be carried as
two 16-bit pieces: off by 2^-16 relative (bf16, half a step of 2^-8 twice) plus 2^-22 of the
largest magnitude of its row or column (fp16, whose pieces end at a fixed exponent).  The
result is rounded once: half a step of its type and half its smallest subnormal."""
import numpy as np
import pytest
import torch

import synth
import w4a16_quantized_expert_b200 as moe
from gpu_cases import Case
from w4a16_quantized_expert_b200.device import DeviceAdapters

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}
ULP = 2.0 ** -23


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


class Pool:
    def __init__(self, K, N, n, R, dtype, T, seed=0, ranks=True):
        g = np.random.default_rng(seed)
        self.K, self.N, self.n, self.R, self.T = K, N, n, R, T
        self.rank = torch.from_numpy(g.integers(0, R + 1, n).astype(np.int32)).cuda() if ranks else None
        if ranks:
            self.rank[0] = R
        self.a = rand((n, R, K), DT[dtype], seed + 1, K ** -0.5)
        self.b = rand((n, N, R), DT[dtype], seed + 2, R ** -0.5)
        self.scaling = rand((n,), torch.float32, seed + 3)
        if ranks:   # what lies past an adapter's rank is never used
            off = torch.arange(R, device="cuda")[None, :] >= self.rank.long()[:, None]
            self.a[off] = float("nan")
            self.b.transpose(1, 2)[off] = float("inf")
        self.h = DeviceAdapters(self.a, self.b, self.scaling, self.rank, max_tokens=T)
        self.ws = self.h.workspace(T)

    def rank_of(self, i):
        return self.R if self.rank is None else int(self.rank[i])

    def tokens(self, adapter_of):
        which = adapter_of.cpu().numpy()
        for i in range(self.n):
            t = np.flatnonzero(which == i)
            if t.size and self.rank_of(i):
                yield i, torch.from_numpy(t).cuda(), self.rank_of(i)


def assign(T, n, seed, kind="runs"):
    g = np.random.default_rng(seed)
    if kind == "runs":     # requests of ragged lengths, some without an adapter
        which = np.repeat(g.integers(-1, n, T), g.integers(1, 40, T))[:T]
    elif kind == "each":   # every token another request
        which = g.integers(-1, n, T)
    else:
        which = np.full(T, n - 1)
    return torch.from_numpy(which.astype(np.int32)).cuda()


def near(got, exact, tol, what):
    eps = torch.finfo(got.dtype).eps
    tol = tol + eps / 2 * (exact.abs() + tol) + SMALLEST[got.dtype] / 2
    bad = ~((got.double() - exact).abs() <= tol * (1 + 1e-6))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, e.g. at {bad.nonzero()[0].tolist()} "
                           f"{got[bad][0]} for {exact[bad][0]}, allowed {tol.expand_as(exact)[bad][0]}")


def pieces(z, ez, dim):
    """Error of z (itself off by ez) once carried as two 16-bit pieces."""
    return ez + 2.0 ** -16 * z.abs() + 2.0 ** -22 * z.abs().amax(dim, keepdim=True)


def check_apply(P, x, adapter_of, y, y_in, z):
    f = torch.float64
    T = x.shape[0]
    exact = torch.zeros((T, P.N), dtype=f, device="cuda") if y_in is None else y_in.to(f)
    tol = ULP * exact.abs()
    zx, zt = torch.zeros((T, P.R), dtype=f, device="cuda"), torch.zeros((T, P.R), dtype=f, device="cuda")
    for i, t, q in P.tokens(adapter_of):
        A, B, s = P.a[i, :q].to(f), P.b[i, :, :q].to(f), float(P.scaling[i])
        zi, ezi = x[t].to(f) @ A.t(), P.K * ULP * (x[t].to(f).abs() @ A.abs().t())
        zx[t, :q], zt[t, :q] = zi, ezi
        exact[t] += s * (zi @ B.t())
        tol[t] += abs(s) * ((pieces(zi, ezi, 1) + (2 * q + 4) * ULP * zi.abs()) @ B.abs().t())
    near(y, exact, tol, "y")
    if z is not None:
        near(z, zx, zt, "z")
        assert not z[zt == 0].any()


def run_apply(P, adapter_of, xt, yt, seed, base=True, in_place=False, want_z=True):
    T = adapter_of.shape[0]
    x = rand((T, P.K + 24), DT[xt], seed)[:, 8:8 + P.K]             # strided rows, 16-byte aligned
    y_in = rand((T, P.N), DT[yt], seed + 1) if base else None
    keep = y_in.clone() if base else None
    buf = torch.full((T + 2, P.N + 3), 3.0, dtype=DT[yt], device="cuda")
    y = y_in if in_place else buf[1:T + 1, :P.N]
    z = torch.full((T, P.R), 9.0, device="cuda") if want_z else None
    P.h.apply(x, adapter_of, P.ws, y_in=y_in, y=y, z=z)
    assert P.h.status() == moe.MOE_OK
    check_apply(P, x, adapter_of, y, keep, z)
    off = adapter_of < 0
    if base:
        assert torch.equal(bits(y[off]), bits(keep[off])), "a token without an adapter keeps its bits"
    assert bool((buf[0] == 3).all()) and bool((buf[T + 1] == 3).all()) and bool((buf[:, P.N:] == 3).all())


SHAPES = [  # T, K, N, n, R, kind
    (1, 8, 1, 1, 8, "one"), (1, 6144, 6144, 64, 16, "one"), (2, 64, 16, 3, 8, "each"), (7, 256, 5, 2, 16, "each"),
    (8, 1000, 264, 64, 24, "each"), (16, 2048, 512, 16, 64, "one"), (17, 72, 129, 4, 40, "each"),
    (31, 520, 256, 1024, 8, "each"), (33, 512, 136, 5, 128, "each"), (64, 6144, 256, 16, 8, "each"),
    (100, 136, 72, 7, 72, "runs"), (129, 264, 1000, 3, 16, "one"), (200, 2048, 512, 2, 8, "runs"),
    (300, 192, 64, 1, 128, "runs"), (515, 320, 328, 9, 56, "runs"), (1000, 64, 64, 1000, 8, "each"),
    (700, 1024, 640, 4, 32, "one"), (2100, 128, 128, 12, 64, "runs"), (70, 96, 37, 3, 16, "each"),
    (400, 64, 257, 2, 120, "runs"),
]


@pytest.mark.parametrize("T,K,N,n,R,kind", SHAPES)
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_apply(T, K, N, n, R, kind, xt):
    i = SHAPES.index((T, K, N, n, R, kind))
    P = Pool(K, N, n, R, xt, T, seed=i, ranks=i % 3 != 0)
    yt = ["f32", xt, "f16", "bf16"][i % 4]
    which = assign(T, n, i, kind)
    run_apply(P, which, xt, yt, 10 * i, base=i % 5 != 1, want_z=i % 2 == 0)
    run_apply(P, which, xt, "f32", 10 * i + 3, in_place=True, want_z=i % 2 == 1)


def check_backward(P, x, z, dy, adapter_of, base, dx, da, db, da0=None, db0=None):
    f = torch.float64
    T = dy.shape[0]
    ex = torch.zeros((T, P.K), dtype=f, device="cuda") if base is None else base.to(f)
    tx = ULP * ex.abs()
    ea = torch.zeros((P.n, P.R, P.K), dtype=f, device="cuda") if da0 is None else da0.to(f)
    eb = torch.zeros((P.n, P.N, P.R), dtype=f, device="cuda") if db0 is None else db0.to(f)
    ta, tb = ULP * ea.abs(), ULP * eb.abs()
    for i, t, q in P.tokens(adapter_of):
        A, B, s = P.a[i, :q].to(f), P.b[i, :, :q].to(f), float(P.scaling[i])
        d, X, Z = dy[t].to(f), x[t].to(f), z[t, :q].to(f)
        dz, edz = s * (d @ B), abs(s) * (P.N + 2) * ULP * (d.abs() @ B.abs())
        ex[t] += dz @ A
        tx[t] += (pieces(dz, edz, 1) + (2 * q + 4) * ULP * dz.abs()) @ A.abs()
        m = (2 * t.numel() + 4) * ULP
        ea[i, :q] += dz.t() @ X
        # (a piece's fixed exponent is set by the largest dz the adapter's tokens have)
        ta[i, :q] += (edz + 2.0 ** -16 * dz.abs() + 2.0 ** -22 * dz.abs().amax() + m * dz.abs()).t() @ X.abs()
        eb[i, :, :q] += s * (d.t() @ Z)
        tb[i, :, :q] += abs(s) * (d.abs().t() @ (2.0 ** -16 * Z.abs() + 2.0 ** -22 * Z.abs().amax() + m * Z.abs()))
    if dx is not None:
        near(dx, ex, tx, "dx")
    if da is not None:
        near(da, ea, ta, "da")
        near(db, eb, tb, "db")


@pytest.mark.parametrize("T,K,N,n,R,kind", [s for s in SHAPES if s[2] % 8 == 0])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_backward(T, K, N, n, R, kind, xt):
    i = SHAPES.index((T, K, N, n, R, kind))
    P = Pool(K, N, n, R, xt, T, seed=i, ranks=i % 3 != 0)
    dt = ["f32", xt, "f16", "bf16"][i % 4]
    which = assign(T, n, i, kind)
    x, dy = rand((T, K + 8), DT[xt], 50 + i)[:, :K], rand((T, N + 16), DT[xt], 60 + i)[:, 16:]
    z = rand((T, R), torch.float32, 70 + i)
    base = rand((T, K + 1), DT[dt], 80 + i)[:, :K] if i % 5 != 1 else None
    # overwritten: every element, zeros where the batch has no token
    da, db = torch.full((n, R, K), 7.0, device="cuda"), torch.full((n, N, R), 7.0, device="cuda")
    dx = torch.empty((T, K), dtype=DT[dt], device="cuda")
    P.h.backward(x, z, dy, which, P.ws, dx_in=base, dx=dx, da=da, db=db)
    assert P.h.status() == moe.MOE_OK
    check_backward(P, x, z, dy, which, base, dx, da, db)
    off = which < 0
    if base is not None:
        assert torch.equal(bits(dx[off]), bits(base[off]))
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    used[which[which >= 0].long()] = True
    assert not da[~used].any() and not db[~used].any()
    if P.rank is not None:
        past = torch.arange(R, device="cuda")[None, :] >= P.rank.long()[:, None]
        assert not da[past].any() and not db.transpose(1, 2)[past].any()
    # the same call again gives the same bits; adding to what is there
    da2, db2 = torch.empty_like(da), torch.empty_like(db)
    P.h.backward(x, z, dy, which, P.ws, da=da2, db=db2, want_dx=False)
    assert torch.equal(da, da2) and torch.equal(db, db2)
    a0, b0 = rand(da.shape, torch.float32, 1), rand(db.shape, torch.float32, 2)
    da3, db3 = a0.clone(), b0.clone()
    P.h.backward(x, z, dy, which, P.ws, da=da3, db=db3, accumulate=True, want_dx=False)
    check_backward(P, x, z, dy, which, base, None, da3, db3, a0, b0)
    assert torch.equal(da3[~used], a0[~used]) and torch.equal(db3[~used], b0[~used])
    # dx alone, in place
    if base is not None:
        d = base.clone()
        P.h.backward(None, None, dy, which, P.ws, dx_in=d, dx=d, want_dw=False)
        assert torch.equal(bits(d), bits(dx))
    assert P.h.status() == moe.MOE_OK


def test_gradients_against_differences():
    """y is linear in x, in A and in B, so central differences of any length are exact up to
    rounding: <dy, y(+d) - y(-d)> / 2 against <gradient, d>."""
    T, K, N, n, R = 48, 256, 128, 3, 16
    P = Pool(K, N, n, R, "f16", T, ranks=False)
    which = assign(T, n, 4, "each")
    x, dy = rand((T, K), torch.float16, 5), rand((T, N), torch.float16, 6)
    z = torch.empty((T, R), device="cuda")
    zero = torch.zeros((T, N), device="cuda")

    def loss(x, z=None):
        y = P.h.apply(x, which, P.ws, y_in=zero, y=torch.empty_like(zero), z=z)
        return (y.double() * dy.double()).sum()

    loss(x, z)
    dx, da, db = P.h.backward(x, z, dy, which, P.ws, dx=torch.empty((T, K), device="cuda"))
    # every value of the two sides is a sum of such products, off by 2^-16 of them at most
    size = float(dy.double().norm() * x.double().norm() * P.a[0].double().norm() * P.b[0].double().norm()
                 * P.scaling.abs().max())
    q = lambda shape, seed: (torch.randint(-4, 5, shape, generator=torch.Generator(device="cuda").manual_seed(seed),  # noqa: E731
                                           device="cuda") / 4).half()
    d = q((T, K), 1)
    x8 = (x * 8).round() / 8                 # so that x + d and x - d are exact in fp16
    lhs = (loss((x8 + d).half()) - loss((x8 - d).half())) / 2
    assert abs(float(lhs - (dx.double() * d.double()).sum())) <= 2.0 ** -16 * size * 4
    for w, g, seed in ((P.a, da, 2), (P.b, db, 3)):
        keep = w.clone()
        d = (q(w.shape, seed) / 16).half()
        w.copy_((keep * 64).round() / 64)
        mid = w.clone()
        z0 = torch.empty((T, R), device="cuda")
        loss(x, z0)
        g = P.h.backward(x, z0, dy, which, P.ws, want_dx=False)[1 if w is P.a else 2]
        w.copy_(mid + d)
        up = loss(x)
        w.copy_(mid - d)
        down = loss(x)
        w.copy_(keep)
        assert abs(float((up - down) / 2 - (g.double() * d.double()).sum())) <= 2.0 ** -16 * size * 4


@pytest.mark.parametrize("T", [8, 200])
def test_bad_adapters_ranks_and_tokens(T):
    P = Pool(64, 40, 4, 16, "f16", T)
    which = assign(T, 4, 1, "each")
    bad = which.clone()
    bad[1], bad[2], bad[T - 1] = 4, -2, 2 ** 31 - 1
    good = torch.where((bad < 0) | (bad >= 4), torch.full_like(bad, -1), bad)
    x, y_in = rand((T, 64), torch.float16, 1), rand((T, 40), torch.float32, 2)
    y0 = P.h.apply(x, good, P.ws, y_in=y_in)
    assert P.h.status() == moe.MOE_OK
    y1 = P.h.apply(x, bad, P.ws, y_in=y_in)
    assert P.h.status() == moe.MOE_ERR_DEVICE_BOUNDS
    assert torch.equal(bits(y0), bits(y1))
    z, dy = rand((T, 16), torch.float32, 3), rand((T, 40), torch.float16, 4)
    g0 = P.h.backward(x, z, dy, good, P.ws)
    assert P.h.status() == moe.MOE_OK
    g1 = P.h.backward(x, z, dy, bad, P.ws)
    assert P.h.status() == moe.MOE_ERR_DEVICE_BOUNDS
    for a, b in zip(g0, g1):
        assert torch.equal(a, b)
    P.rank[0] = 17                                   # counts as rank 0
    which.fill_(0)
    y = P.h.apply(x, which, P.ws, y_in=y_in)
    assert P.h.status() == moe.MOE_ERR_DEVICE_BOUNDS
    assert torch.equal(y, y_in)


@pytest.mark.parametrize("T", [12, 300])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_special_values_stay_in_their_rows(T, xt):
    """Infinities and NaN of one token reach that token alone; -0 and NaN payloads of tokens
    without an adapter keep their bits; fp16 rows whose z leaves the fp16 range are right."""
    P = Pool(512, 72, 3, 16, xt, T, ranks=False)
    which = assign(T, 3, 2, "each")
    which[0], which[1], which[2], which[3], which[4] = 0, 1, -1, 2, 0
    x = rand((T, 512), DT[xt], 1)
    y_in = rand((T, 72), DT[xt], 2)
    y_in[2, 0] = -0.0
    bits_in = torch.tensor([0x7E55 if xt == "f16" else 0x7FD5], dtype=torch.int16, device="cuda")
    y_in[2, 1:2] = bits_in.view(DT[xt])
    clean = P.h.apply(x, which, P.ws, y_in=y_in)
    x[0, 7], x[1, 9] = float("inf"), float("nan")
    y = P.h.apply(x, which, P.ws, y_in=y_in)
    assert torch.equal(bits(y[2:]), bits(clean[2:]))
    assert not torch.isfinite(y[0].float()).any() and torch.isnan(y[1].float()).all()
    assert torch.equal(bits(y[2]), bits(y_in[2]))
    # z of 2^16 and more: 512 products of about 2^8 x 1 each; tiny rows beside them
    P.a.fill_(1.0)
    x = torch.full((T, 512), 255.0, device="cuda").to(DT[xt])
    x[3] = 2.0 ** -20
    out = torch.zeros((T, 72), device="cuda")
    z = torch.empty((T, 16), device="cuda")
    P.h.apply(x, which, P.ws, y_in=out, y=out, z=z)
    check_apply(P, x, which, out, torch.zeros_like(out), z)
    assert float(z[0].max()) > 65504


@pytest.mark.parametrize("T", [20, 260])
def test_gradient_ranges(T):
    """dy and z whose products leave the fp16 range, and an adapter whose gradients are far
    smaller than its neighbour's, keep their precision."""
    P = Pool(128, 64, 2, 8, "f16", T, ranks=False)
    which = assign(T, 2, 3, "each")
    x, dy = rand((T, 128), torch.float16, 1), rand((T, 64), torch.float16, 2, 2000.0)
    z = rand((T, 8), torch.float32, 3, 3.0e5)
    dy[which == 1] = (dy[which == 1].float() * 2.0 ** -20).half()
    z[which == 1] *= 2.0 ** -30
    dx, da, db = P.h.backward(x, z, dy, which, P.ws, dx=torch.empty((T, 128), device="cuda"))
    check_backward(P, x, z, dy, which, None, dx, da, db)


def test_no_token():
    P = Pool(64, 16, 3, 8, "bf16", 4)
    ws = P.h.workspace(0)
    da, db = torch.full((3, 8, 64), 5.0, device="cuda"), torch.full((3, 16, 8), 5.0, device="cuda")
    args = [P.h.handle, None, 0, None, None, 0, None, 0, None, 0, None, 0, 0, da.data_ptr(), db.data_ptr()]
    moe.moe_adapters_backward(*args, 1, ws.data_ptr(), ws.numel())
    assert bool((da == 5).all()) and bool((db == 5).all())
    moe.moe_adapters_backward(*args, 0, ws.data_ptr(), ws.numel())
    assert not da.any() and not db.any()
    moe.moe_adapters_apply(P.h.handle, None, 0, None, 0, None, 0, None, 0, 0, None, None, 0)
    # a batch without any adapter
    x, y_in = rand((4, 64), torch.bfloat16, 1), rand((4, 16), torch.bfloat16, 2)
    none = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    z = torch.full((4, 8), 5.0, device="cuda")
    assert torch.equal(P.h.apply(x, none, P.ws, y_in=y_in, z=z), y_in) and not z.any()
    dx, da, db = P.h.backward(x, z, y_in, none, P.ws)
    assert not dx.any() and not da.any() and not db.any()


def test_guard_bands():
    for T in (9, 140):
        P = Pool(72, 24, 3, 24, "f16", T)
        which = assign(T, 3, 1, "each")
        n = P.ws.numel()
        buf = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        ws = buf[4096:4096 + n]
        g = lambda *s: torch.full((s[0] + 2, *s[1:]), 3.0, device="cuda")  # noqa: E731
        y, z, da, db, dx = g(T, 24), g(T, 24), g(3, 24, 72), g(3, 24, 24), g(T, 72)
        x, dy = rand((T, 72), torch.float16, 1), rand((T, 24), torch.float16, 2)
        P.h.apply(x, which, ws, y=y[1:-1], z=z[1:-1])
        P.h.backward(x, z[1:-1], dy, which, ws, dx=dx[1:-1], da=da[1:-1], db=db[1:-1])
        for t in (y, z, da, db, dx):
            assert bool((t[0] == 3).all()) and bool((t[-1] == 3).all())
        assert bool((buf[:4096] == 0xA5).all()) and bool((buf[4096 + n:] == 0xA5).all())


def test_refusals():
    T = 8
    P = Pool(64, 32, 2, 8, "f16", T)
    x, y, dy = rand((T, 64), torch.float16, 1), rand((T, 32), torch.float16, 2), rand((T, 32), torch.float16, 3)
    z, which = torch.empty((T, 8), device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    da, db = torch.empty((2, 8, 64), device="cuda"), torch.empty((2, 32, 8), device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    ws, nb = p(P.ws), P.ws.numel()

    def refused(code, fn, args, at, v):
        a = list(args)
        a[at] = v
        with pytest.raises(moe.MoeError) as e:
            fn(P.h.handle, *a)
        assert e.value.code == code, (fn, at, v)

    ap = [p(x), 64, p(which), T, p(y), 32, p(y), 0, 32, p(z), ws, nb]
    for at, v, code in [(0, None, 1), (0, p(x) + 2, 1), (1, 60, 1), (1, 68, 1), (2, None, 1), (3, T + 1, 1), (3, -1, 1),
                        (4, p(y) + 1, 1), (5, 31, 1), (5, 40, 1), (6, None, 1), (6, p(y) + 1, 1), (7, 3, 1), (8, 31, 1),
                        (9, p(z) + 4, 1), (10, None, 3), (10, ws + 128, 3), (11, nb - 1, 3)]:
        refused(code, moe.moe_adapters_apply, ap, at, v)
    bw = [p(x), 64, p(z), p(dy), 32, p(which), T, p(x), 64, p(x), 0, 64, p(da), p(db), 0, ws, nb]
    for at, v, code in [(0, None, 1), (1, 63, 1), (2, None, 1), (2, p(z) + 8, 1), (3, None, 1), (3, p(dy) + 2, 1),
                        (4, 33, 1), (5, None, 1), (6, T + 1, 1), (7, p(x) + 1, 1), (8, 72, 1), (10, -1, 1), (11, 8, 1),
                        (12, None, 1), (13, None, 1), (12, p(da) + 4, 1), (9, None, 1), (15, None, 3),
                        (16, nb - 256, 3)]:
        refused(code, moe.moe_adapters_backward, bw, at, v)
    odd = Pool(64, 33, 2, 8, "f16", T)
    with pytest.raises(moe.MoeError):
        odd.h.backward(x, z, rand((T, 33), torch.float16, 1), which, odd.ws)
    for bad in ((x.float(), None), (x[:, :32], None), (x, y.float()), (x.t().contiguous().t(), None)):
        with pytest.raises(ValueError):
            P.h.apply(bad[0], which, P.ws, y_in=bad[1], y=y)
    with pytest.raises(ValueError):
        P.h.apply(x, which.long(), P.ws)
    assert P.h.status() == moe.MOE_OK


def test_captured_and_replayed_on_another_stream():
    for T in (16, 300):
        P = Pool(256, 128, 5, 16, "bf16", T)
        x, dy = rand((T, 256), torch.bfloat16, 1), rand((T, 128), torch.bfloat16, 2)
        which = assign(T, 5, 1, "each")
        y, z = torch.empty((T, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((T, 16), device="cuda")
        dx = torch.empty_like(x)
        da, db = torch.empty((5, 16, 256), device="cuda"), torch.empty((5, 128, 16), device="cuda")

        def step():
            P.h.apply(x, which, P.ws, y=y, z=z)
            P.h.backward(x, z, dy, which, P.ws, dx=dx, da=da, db=db)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step()
        for seed in (5, 6):
            x.copy_(rand((T, 256), torch.bfloat16, seed))
            which.copy_(assign(T, 5, seed, "each"))
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in (y, z, dx, da, db)]
            step()
            torch.cuda.synchronize()
            for a, b in zip(got, (y, z, dx, da, db)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("T", [4, 37])
def test_adapters_and_sorted_rows_in_the_staged_layer(T):
    """The operators as a layer runs them: adapters on the router's logits, routing from those
    logits, experts, adapters on the shared expert's output, and the combine, once by moe_combine
    and once through sorted rows; then the gradient of the way back."""
    case = Case(synth.WORKLOADS["tiny"], T=T, max_tokens=64)
    L, d = case.dev, case.desc
    H, E, k = d["H"], d["E"], d["k"]
    ws = L.workspace(T)
    x = case.x_dev
    xh = x.view(torch.float16)
    _, _, logits = L.route(x, T, ws, want_logits=True)
    which = assign(T, 3, 1, "each")
    which[0] = 1
    on_router, on_shared = Pool(H, E, 3, 8, "f16", T, seed=1), Pool(H, H, 3, 16, "f16", T, seed=2)
    keep = logits.clone()
    on_router.h.apply(xh, which, on_router.ws, y_in=logits, y=logits)
    check_apply(on_router, xh, which, logits, keep, None)
    idx, w, _ = L.route(None, T, ws, logits_in=logits)
    _, offsets, perm, _, _ = L.group(idx, T, ws)
    y_assign, y_shared = L.expert_ffn(x, T, offsets, perm, ws)
    base = y_shared.clone()
    on_shared.h.apply(xh, which, on_shared.ws, y_in=y_shared, y=y_shared)
    check_apply(on_shared, xh, which, y_shared, base, None)
    y = L.combine(y_assign, y_shared, w, T)
    rows, row_of, counts, seg = L.sort_tokens(xh, idx, ws, align=8)
    out = torch.full((rows.shape[0], H), float("nan"), device="cuda")
    out[row_of.reshape(-1).long()] = y_assign                    # the experts' outputs as sorted rows
    y2 = L.unsort_tokens(out, row_of, w, y_shared=y_shared, y=torch.empty((T, H), dtype=torch.float16, device="cuda"))
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16)), "both ways give moe_combine's bits"
    at = row_of.reshape(-1).long()
    assert torch.equal(bits(rows[at]), bits(xh.repeat_interleave(k, 0)))
    dy = rand((T, H), torch.float16, 3)
    drows, dw = L.unsort_tokens_backward(dy, out, row_of, w, counts, seg)
    dx = L.sort_tokens_backward(drows, row_of, dx=torch.empty((T, H), device="cuda"))
    exact = (w.double().sum(1, keepdim=True) * dy.double())     # identity experts: dx = sum_j w_j dy
    near(dx, exact, (k + 2) * ULP * exact.abs(), "dx")
    prod = dy.double()[:, None, :] * y_assign.reshape(T, k, H).double()
    near(dw, prod.sum(2), (H // 32 + 16) * ULP * prod.abs().sum(2), "dw")
    assert moe.moe_get_device_status(L.handle) == moe.MOE_OK
    assert on_router.h.status() == on_shared.h.status() == moe.MOE_OK


def test_no_token_with_an_input_gradient():
    P = Pool(64, 16, 3, 8, "f16", 4)
    ws = P.h.workspace(0)
    dx = torch.empty((1, 64), dtype=torch.float16, device="cuda")
    da, db = torch.full((3, 8, 64), 5.0, device="cuda"), torch.full((3, 16, 8), 5.0, device="cuda")
    moe.moe_adapters_backward(P.h.handle, None, 0, None, None, 0, None, 0, None, 0, dx.data_ptr(), 0, 64,
                              da.data_ptr(), db.data_ptr(), 0, ws.data_ptr(), ws.numel())
    assert not da.any() and not db.any()


@pytest.mark.parametrize("T,K,N,n,R,kind", [
    (20000, 64, 64, 1024, 8, "each"),      # more chunks than a cluster sorts, more adapters than are ranked
    (3000, 4096, 128, 2, 128, "one"),      # one adapter, long chains of both kinds, the widest rank
    (4097, 128, 2048, 130, 24, "runs"),
])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_large_batches(T, K, N, n, R, kind, xt):
    P = Pool(K, N, n, R, xt, T, seed=1)
    which = assign(T, n, 1, kind)
    run_apply(P, which, xt, "f32", 7)
    x, dy = rand((T, K), DT[xt], 1), rand((T, N), DT[xt], 2)
    z = rand((T, R), torch.float32, 3)
    da, db = torch.empty((n, R, K), device="cuda"), torch.empty((n, N, R), device="cuda")
    dx = torch.empty((T, K), device="cuda")
    P.h.backward(x, z, dy, which, P.ws, dx=dx, da=da, db=db)
    check_backward(P, x, z, dy, which, None, dx, da, db)
    assert P.h.status() == moe.MOE_OK


@pytest.mark.parametrize("T", [20, 2100])
def test_offsets_past_32_bits(T):
    """Rows 2^21 elements apart: the last ones lie more than 2^32 elements behind the first
    (for the larger batch)."""
    K, N, n, R = 64, 72, 3, 16
    ld = 2 ** 21 if T > 32 else 2 ** 27
    P = Pool(K, N, n, R, "f16", T)
    which = assign(T, n, 1, "each")
    buf = torch.empty((T, ld), dtype=torch.float16, device="cuda")
    x, y = buf[:, :K], buf[:, K:K + N]
    x.copy_(rand((T, K), torch.float16, 1))
    y_in = rand((T, N), torch.float16, 2)
    y.copy_(y_in)
    z = torch.empty((T, R), device="cuda")
    P.h.apply(x, which, P.ws, y_in=y, y=y, z=z)
    check_apply(P, x, which, y, y_in, z)
    dx = buf[:, 256:256 + K]
    da, db = torch.empty((n, R, K), device="cuda"), torch.empty((n, N, R), device="cuda")
    dy = buf[:, 512:512 + N]
    dy.copy_(rand((T, N), torch.float16, 3))
    P.h.backward(x, z, dy, which, P.ws, dx=dx, da=da, db=db)
    check_backward(P, x, z, dy, which, None, dx, da, db)
    assert P.h.status() == moe.MOE_OK


def test_two_streams_at_once():
    """Calls of one handle on two streams, each with a workspace of its own."""
    T, K, N, n, R = 600, 512, 256, 4, 32
    P = Pool(K, N, n, R, "bf16", T)
    which = assign(T, n, 1, "runs")
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [rand((T, K), torch.bfloat16, i) for i in range(2)]
    dys = [rand((T, N), torch.bfloat16, 5 + i) for i in range(2)]
    wss = [P.h.workspace(T) for _ in range(2)]
    outs = [[torch.empty((T, N), dtype=torch.bfloat16, device="cuda"), torch.empty((T, R), device="cuda"),
             torch.empty((T, K), dtype=torch.bfloat16, device="cuda"), torch.empty((n, R, K), device="cuda"),
             torch.empty((n, N, R), device="cuda")] for _ in range(3)]

    def step(i, o, ws):
        P.h.apply(xs[i], which, ws, y=o[0], z=o[1])
        P.h.backward(xs[i], o[1], dys[i], which, ws, dx=o[2], da=o[3], db=o[4])

    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                step(i, outs[i], wss[i])
    torch.cuda.synchronize()
    for i in range(2):
        step(i, outs[2], P.ws)
        torch.cuda.synchronize()
        for a, b in zip(outs[i], outs[2]):
            assert torch.equal(a, b)
    assert P.h.status() == moe.MOE_OK
