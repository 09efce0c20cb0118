"""Dense layers against 64-bit plain forms: every type, activation and optional argument, over sizes that cross the
kernels' own boundaries (8 rows; 64, 128 and 256 of each direction; sums in parts), and rows off 16 bytes."""
import pytest
import torch

from sparse_embeddings_feature_gb300 import ctr

import _layers_ref as L

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "relu", "silu", "gelu", "sigmoid"]
# rows, n, k, padding of the rows (0: dense)
FEW = [(1, 1, 1, 0), (1, 512, 479, 0), (2, 7, 1030, 1), (3, 100, 64, 8), (5, 33, 2051, 0), (8, 257, 1024, 0)]
SIZES = FEW + [(2, 512, 1024, 0), (3, 512, 1024, 0), (4, 130, 4100, 4), (8, 66, 8200, 0), (9, 24, 40, 0), (16, 1, 3, 0), (64, 128, 64, 0), (65, 130, 72, 8), (127, 479, 129, 0), (128, 128, 128, 0),
               (129, 129, 65, 3), (300, 512, 479, 0), (257, 264, 520, 0), (1000, 96, 1000, 4), (2000, 300, 77, 0),
               (4100, 520, 200, 8), (70, 135, 479, 1), (300, 479, 135, 1)]
LARGE = [(13000, 264, 512, 0), (3000, 2304, 264, 0), (40000, 257, 129, 0), (2500, 1544, 1100, 0)]


def _draw(g, rows, cols, dtype, scale=1.0, pad=0):
    buf = torch.full((max(rows, 1), cols + pad), 7.0, dtype=DT[dtype], device="cuda")
    view = buf[:rows, :cols]
    view.copy_(torch.randn((rows, cols), generator=g, device="cuda") * scale)
    return view


def _blank(rows, cols, dtype, pad):
    buf = torch.full((max(rows, 1), cols + pad), 3.0, dtype=dtype, device="cuda")
    return buf, buf[:rows, :cols]


class Case:
    def __init__(self, rows, n, k, pad, dtype, seed=0, scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed + 31 * rows + n)
        self.rows, self.n, self.k, self.pad, self.dtype = rows, n, k, pad, dtype
        self.x = _draw(g, rows, k, dtype, scale, pad)
        self.w = _draw(g, n, k, dtype, k ** -0.5, 2 * pad)
        self.r = _draw(g, rows, n, dtype, 1.0, pad)
        self.dy = _draw(g, rows, n, dtype, 1.0, pad)
        self.bias = _draw(g, 1, n, dtype)[0].contiguous()
        need = ctr.ctr_dense_workspace_size(rows, n, k, DT[dtype], True, packed=True)
        self.full = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        self.full[:256].zero_()
        self.ws = self.full[:need]

    def finish(self):
        assert ctr.ctr_check_status(self.ws) == 0
        assert bool((self.full[self.ws.numel():] == 0xA5).all()), "a write left the workspace"

    def forward(self, act, bias, residual, pre):
        n, dtype = self.n, self.dtype
        yb, y = _blank(self.rows, n, DT[dtype], self.pad)
        pb, p = _blank(self.rows, n, DT[dtype], self.pad)
        ctr.ctr_dense(self.x, self.w, self.bias if bias else None, ctr.ACTIVATIONS[act], self.r if residual else None, y,
                      p if pre else None, self.ws)
        x, w = self.x.double(), self.w.double()
        z, mag = x @ w.t(), x.abs() @ w.abs().t()
        if bias:
            z, mag = z + self.bias.double(), mag + self.bias.double().abs()
        tol = L.sum_bound(dtype, self.k, mag) + 1e-40
        ref = L.act64(act, z)[0] + (self.r.double() if residual else 0)
        assert L.fits(y, ref, L.act_tol(z, ref, tol) if act != "none" else tol + L.U * ref.abs(), dtype)
        if pre:
            assert L.fits(p, z, tol, dtype)
            if dtype == "f32" and self.rows * n >= 1000:
                assert float((p.double() - z).norm() / z.norm()) <= 16 * L.U
        else:
            assert bool((pb == 3.0).all())
        for b in (yb, pb):
            assert bool((b[:, n:] == 3.0).all()) and bool((b[self.rows:] == 3.0).all()), "a write left its row"
        self.finish()
        return y, p

    def backward(self, act, pre, grad, dx=True, dw=True, db=True):
        rows, n, k, dtype = self.rows, self.n, self.k, self.dtype
        xb, gx = _blank(rows, k, DT[dtype], self.pad)
        wb, gw = _blank(n, k, grad, self.pad)
        gb = torch.full((n,), 3.0, dtype=grad, device="cuda")

        def call():
            ctr.ctr_dense_bwd(self.dy, self.x, self.w, pre if act != "none" else None, ctr.ACTIVATIONS[act],
                              gx if dx else None, gw if dw else None, gb if db else None, self.ws)
        call()
        gtype = "f32" if grad == torch.float32 else "bf16"
        x, w, dy, p = self.x.double(), self.w.double(), self.dy.double(), pre.double()
        dz, off, raw, err = L.dz64(dtype, act, dy, p)
        if dx:
            mag = dz.abs() @ w.abs()
            assert L.fits(gx, dz @ w, L.sum_bound(dtype, n, mag) + off @ w.abs() + 1e-40, dtype)
        if dw:
            mag = dz.abs().t() @ x.abs()
            assert L.fits(gw, dz.t() @ x, L.sum_bound(dtype, max(rows, 1), mag, True) + off.t() @ x.abs() + 1e-40, gtype)
            if dtype == "f32" and act == "none" and rows >= 64 and n * k >= 1000:
                ref = dz.t() @ x
                assert float((gw.double() - ref).norm() / ref.norm()) <= 16 * L.U
        if db:
            # a thread adds a quarter of a strip, four threads, at most 76 + 16 strips
            tol = (max(rows, 32) / 4 + 100) * L.U * raw.abs().sum(0) + err.sum(0) + 1e-40
            assert L.fits(gb, raw.sum(0), tol, gtype)
        assert bool((xb[:, k:] == 3.0).all()) and bool((wb[:, k:] == 3.0).all()), "a write left its row"
        first = [t.clone() for t in (gx, gw, gb)]
        call()
        assert all(torch.equal(a, b) for a, b in zip(first, (gx, gw, gb)))
        self.finish()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k,pad", SIZES)
def test_forward(rows, n, k, pad, dtype):
    c = Case(rows, n, k, pad, dtype)
    for i, act in enumerate(ACTS):
        c.forward(act, bias=i % 2 == 0, residual=i % 3 == 0, pre=i % 4 != 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k,pad", SIZES)
def test_backward(rows, n, k, pad, dtype):
    c = Case(rows, n, k, pad, dtype)
    pre = _draw(torch.Generator(device="cuda").manual_seed(5), rows, n, dtype, 1.5, pad)
    for i, act in enumerate(ACTS):
        c.backward(act, pre, DT[dtype] if i % 2 else torch.float32, dx=i != 3, dw=i != 2, db=i != 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n,k,pad", LARGE)
def test_large(rows, n, k, pad, dtype):
    c = Case(rows, n, k, pad, dtype)
    y, pre = c.forward("silu", True, True, True)
    c.forward("none", False, True, False)
    c.backward("silu", pre, DT[dtype])
    c.backward("none", pre, torch.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_rows(dtype):
    c = Case(0, 40, 24, 0, dtype)
    y = torch.empty((0, 40), dtype=DT[dtype], device="cuda")
    ctr.ctr_dense(c.x, c.w, c.bias, ctr.ACT_RELU, None, y, None, c.ws)
    dw, db = torch.full((40, 24), 5.0, device="cuda"), torch.full((40,), 5.0, device="cuda")
    ctr.ctr_dense_bwd(c.dy, c.x, c.w, y, ctr.ACT_RELU, torch.empty_like(c.x), dw, db, c.ws)
    assert not dw.any() and not db.any()
    dw = torch.full((40, 24), 5.0, device="cuda", dtype=DT[dtype])
    ctr.ctr_dense_bwd(c.dy, c.x, c.w, None, ctr.ACT_NONE, None, dw, None, c.ws)
    assert not dw.any()


def test_gradient_is_the_differences():
    # central differences in 64 bits of L = sum dy y; |L'''| < 1e2: h^2 L''' / 6 < 1e-8, cancellation 1e-16 * 1e3 / 1e-5
    h = 1e-5
    for act in ("silu", "gelu", "sigmoid"):
        c = Case(12, 20, 10, 0, "f32", seed=3)
        y, pre = c.forward(act, True, True, True)
        dx, dw, db = torch.empty_like(c.x), torch.empty_like(c.w), torch.empty_like(c.bias)
        ctr.ctr_dense_bwd(c.dy, c.x, c.w, pre, ctr.ACTIVATIONS[act], dx, dw, db, c.ws)
        x, w, b, dy = c.x.double(), c.w.double(), c.bias.double(), c.dy.double()

        def loss(x, w, b):
            return (dy * L.act64(act, x @ w.t() + b)[0])
        mag = dy.abs().sum() * 4
        for j in range(10):
            e = torch.zeros(10, dtype=torch.float64, device="cuda")
            e[j] = h
            diff = ((loss(x + e, w, b) - loss(x - e, w, b)) / (2 * h)).sum(1)
            assert bool(((dx[:, j].double() - diff).abs() <= 1e-7 + 600 * L.U * mag).all())
        e = h * torch.ones(20, dtype=torch.float64, device="cuda")
        diff = ((loss(x, w, b + e) - loss(x, w, b - e)) / (2 * h)).sum(0)
        assert bool(((db.double() - diff).abs() <= 1e-7 + 600 * L.U * mag).all())
        for i, j in ((0, 0), (7, 3), (19, 9)):
            e = torch.zeros_like(w)
            e[i, j] = h
            diff = ((loss(x, w + e, b) - loss(x, w - e, b)) / (2 * h)).sum()
            assert abs(float(dw[i, j]) - float(diff)) <= 1e-7 + 600 * L.U * float(mag)


@pytest.mark.parametrize("rows", [5, 200])
@pytest.mark.parametrize("act", ACTS)
def test_every_bf16_number_as_bias(rows, act):
    # z = bias: activations and their derivatives over every finite bf16 number
    bits = torch.arange(65536, dtype=torch.int32)
    bits = bits[(bits & 0x7f80) != 0x7f80]
    bias = bits.to(torch.int16).view(torch.bfloat16).cuda()
    n, dt = bias.numel(), torch.bfloat16
    x, w = torch.zeros((rows, 8), dtype=dt, device="cuda"), torch.zeros((n, 8), dtype=dt, device="cuda")
    y, pre = torch.empty((rows, n), dtype=dt, device="cuda"), torch.empty((rows, n), dtype=dt, device="cuda")
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(rows, n, 8, dt, True))
    ctr.ctr_dense(x, w, bias, ctr.ACTIVATIONS[act], None, y, pre, ws)
    z = bias.double()
    assert torch.equal(pre, bias.expand_as(pre))
    ref = L.act64(act, z)[0]
    assert L.fits(y, ref.expand_as(y), L.act_tol(z, ref, 0 * z), "bf16")
    dy = torch.ones_like(y)
    db = torch.empty(n, device="cuda")
    ctr.ctr_dense_bwd(dy, x, w, pre, ctr.ACTIVATIONS[act], None, None, db, ws)
    d = rows * L.act64(act, z)[1]
    d = torch.where(torch.isfinite(d), d, 0.0)   # far out gelu's and silu's second terms are infinity times zero in 64 bits
    assert bool(((db.double() - d).abs() <= rows * 16 * L.U * (1 + z.abs().clamp(max=1e3)) + 40 * L.U * d.abs()).all())


@pytest.mark.parametrize("rows", [3, 40])
def test_fp32_magnitudes_far_apart(rows):
    # numbers over fp32's whole range: planes that round to infinity or vanish; each row has one magnitude
    g = torch.Generator(device="cuda").manual_seed(9)
    k, n = 70, 33
    mags = torch.tensor([3.4e38, 1e30, 1.0, 1e-20, 1e-30, 2.0 ** -100], device="cuda")
    x = (torch.rand((rows, k), generator=g, device="cuda") * 0.5 + 0.5) * mags[torch.arange(rows, device="cuda") % 6][:, None]
    w = torch.zeros((n, k), device="cuda")
    w[torch.arange(n), torch.arange(n)] = 1.0
    w[5, :2] = torch.tensor([0.25, -0.125], device="cuda")
    y = torch.empty((rows, n), device="cuda")
    ws = ctr.workspace(ctr.ctr_dense_workspace_size(rows, n, k, torch.float32))
    ctr.ctr_dense(x, w, None, ctr.ACT_NONE, None, y, None, ws)
    ref, mag = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    # row 12's 2.94e38 + 3.4e38 / 4 - .. is 3.437e38 at column 5, past fp32's largest number, 3.403e38: an infinity
    ref = torch.where(torch.isinf(ref.float()), ref.float().double(), ref)
    assert bool(((y == ref) | ((y.double() - ref).abs() <= 16 * L.U * mag)).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [4, 300])
def test_non_finite_rows_stay_in_their_rows(rows, dtype):
    c = Case(rows, 136, 72, 0, dtype)
    clean, _ = c.forward("silu", True, False, True)
    c.x[1, 5], c.x[3, 71] = float("nan"), float("inf")
    y = torch.empty_like(clean)
    ctr.ctr_dense(c.x, c.w, c.bias, ctr.ACT_NONE, None, y, None, c.ws)
    fine = torch.ones(rows, dtype=torch.bool, device="cuda")
    fine[1] = fine[3] = False
    assert bool(torch.isfinite(y[fine]).all()) and not bool(torch.isfinite(y[~fine]).any())


def test_residual_in_place_two_streams_and_graphs():
    a, b = Case(500, 256, 200, 0, "bf16"), Case(700, 479, 100, 0, "f32")

    def run(c, out):
        ctr.ctr_dense(c.x, c.w, c.bias, ctr.ACT_GELU, out[0], out[0], out[1], c.ws)   # y over the residual
        ctr.ctr_dense_bwd(c.dy, c.x, c.w, out[1], ctr.ACT_GELU, out[2], out[3], out[4], c.ws)
    outs = [[c.r.clone(), torch.empty_like(c.r), torch.empty_like(c.x), torch.empty_like(c.w), torch.empty_like(c.bias)]
            for c in (a, b)]
    sep = torch.empty_like(a.r)
    ctr.ctr_dense(a.x, a.w, a.bias, ctr.ACT_GELU, a.r, sep, None, a.ws)
    for c, o in zip((a, b), outs):
        run(c, o)
    assert torch.equal(sep, outs[0][0])
    again = [[c.r.clone()] + [torch.zeros_like(t) for t in o[1:]] for c, o in zip((a, b), outs)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for c, o, s in zip((a, b), again, side):   # both at once
        with torch.cuda.stream(s):
            run(c, o)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for o, r in zip(outs, again) for p, q in zip(o, r))
    # two graphs that share one workspace, replayed in turn
    shared = ctr.workspace(max(a.ws.numel(), b.ws.numel()))
    a.ws = b.ws = shared
    graphs = []
    for c, o in zip((a, b), again):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(c, o)
        graphs.append(g)
    for _ in range(2):
        for c, o in zip((a, b), again):
            o[0].copy_(c.r)
            for t in o[1:]:
                t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for o, r in zip(outs, again) for p, q in zip(o, r))
    assert ctr.ctr_check_status(shared) == 0


def test_workspace_that_is_too_small_is_refused():
    c = Case(300, 64, 479, 0, "bf16")    # 479: rows off 16 bytes
    small = ctr.workspace(ctr.ctr_dense_workspace_size(300, 64, 479, torch.bfloat16, True, packed=False))
    y = torch.empty_like(c.r)
    with pytest.raises(ctr.CtrError) as e:
        ctr.ctr_dense(c.x, c.w, None, ctr.ACT_NONE, None, y, None, small)
    assert e.value.status == ctr.ERR_WORKSPACE
    with pytest.raises(ctr.CtrError) as e:
        ctr.ctr_dense_bwd(c.dy, c.x, c.w, None, ctr.ACT_NONE, None, torch.empty_like(c.w), None, small)
    assert e.value.status == ctr.ERR_WORKSPACE
