"""GPU results of the linear layers (moe_grouped_linear, moe_linear and their
backward) against float64, element by element within bounds derived from the
arithmetic (linear_util.py), over ragged groups, odd sizes, every activation
and way of saving; the rows of no group, captured graphs, other streams and
bad offsets."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import requires_gpu, say
from linear_util import HALF, TYPES, Layer, make_offsets, rows8_read, within

pytestmark = [pytest.mark.gpu, requires_gpu]


def _mm():
    import mixture_experts_routing_gemm_amd as mm
    return mm


def cu(t):
    return None if t is None else t.cuda()


class Run:
    """One layer's device buffers, filled with a value that no result has."""

    def __init__(self, L, save="none", grad=None, dense=False):
        mm = _mm()
        self.L, self.dense = L, dense
        t, G = TYPES[L.kind], len(L.offsets) - 1
        self.grad = grad or L.kind
        self.s = mm.make_linear_shape(L.rows, L.n_in, L.n_out, groups=G, act=L.kind, fn=L.fn, save=save, grad=self.grad)
        self.save = save
        self.x, self.w, self.bias, self.residual, self.dy = cu(L.x), cu(L.w), cu(L.bias), cu(L.residual), cu(L.dy)
        self.off = torch.from_numpy(L.offsets).cuda()
        f = lambda *s, dtype=t: torch.full(s, 77.0, dtype=dtype, device="cuda")  # noqa: E731
        self.y, self.dx = f(L.rows, L.n_out), f(L.rows, L.n_in)
        self.dw, self.db = f(G, L.n_out, L.n_in, dtype=TYPES[self.grad]), f(G, L.n_out, dtype=TYPES[self.grad])
        self.saved = mm.alloc_linear_saved(self.s)
        if self.saved is not None:
            self.saved.fill_(0x55)
        self.ws = mm.alloc_linear_workspace(self.s, mm.STAGE_LINEAR)
        self.bws = mm.alloc_linear_workspace(self.s, mm.STAGE_LINEAR_BACKWARD)

    def forward(self, stream=None):
        mm = _mm()
        if self.dense:
            mm.moe_linear(self.s, self.x, self.w, self.bias, self.residual, self.y, self.saved, self.ws, stream)
        else:
            mm.moe_grouped_linear(self.s, self.x, self.off, self.w, self.bias, self.residual, self.y, self.saved, self.ws,
                                  stream)

    def backward(self, stream=None):
        mm = _mm()
        if self.dense:
            mm.moe_linear_backward(self.s, self.x, self.w, self.saved, self.dy, self.dx, self.dw, self.db, self.bws, stream)
        else:
            mm.moe_grouped_linear_backward(self.s, self.x, self.off, self.w, self.saved, self.dy, self.dx, self.dw, self.db,
                                           self.bws, stream)

    def saved_z(self):
        L = self.L
        if self.save == "act":
            n = L.rows * L.n_out * (4 if L.kind == "f32" else 2)
            return self.saved[:n].view(TYPES[L.kind]).reshape(L.rows, L.n_out).double().cpu()
        v, codes = rows8_read(self.saved, L.rows, L.n_out)
        return torch.from_numpy(v[:, :L.n_out])

    def check_forward(self):
        y, z, ey, ez = self.L.forward()
        within(self.y, y, ey, "y")
        z, ez = z.cpu(), ez.cpu()
        none = torch.isnan(y[:, 0]).cpu()  # rows of no group keep what they held
        assert bool((self.y.cpu()[none] == 77.0).all())
        if self.save == "act":
            within(self.saved_z(), z, ez + HALF[self.L.kind] * (z.abs() + ez), "z")
        elif self.save == "int8":
            # half a step, at most a 127th of the block's largest magnitude
            top = torch.nn.functional.pad((z.abs() + ez).nan_to_num(), (0, -z.shape[1] % 32))
            top = top.reshape(z.shape[0], -1, 32).amax(2).repeat_interleave(32, 1)[:, :z.shape[1]]
            within(self.saved_z(), z, ez + top / 127.0, "z in 8 bits")

    def check_backward(self):
        zs = self.saved_z() if self.save != "none" else None
        dx, dw, db, ex, ew, eb = self.L.backward(zs, self.grad)
        within(self.dx, dx, ex, "dx")
        none = torch.isnan(dx[:, 0]).cpu()
        assert bool((self.dx.cpu()[none] == 77.0).all())
        within(self.dw, dw, ew, "dw")
        within(self.db, db, eb, "db")
        counts = np.diff(self.L.offsets)
        for g in np.nonzero(counts == 0)[0]:
            assert not self.dw[g].any() and not self.db[g].any()


# (rows, n_in, n_out, groups, offsets): the tile kernels' edges (one row, a
# row more or less than a tile, k shorter than a slice and ending inside one,
# columns ending inside a tile), empty and hot groups
GROUPED = [
    (1, 8, 8, 1, "even"),
    (3, 24, 40, 5, "even"),
    (64, 64, 128, 4, "skewed"),
    (257, 136, 264, 3, "holes"),
    (300, 72, 520, 7, "gap"),
    (512, 264, 136, 2, "last"),
    (1000, 512, 256, 4, "skewed"),
    (1030, 200, 328, 1, "even"),
    (130, 1032, 104, 130, "skewed"),
    (700, 64, 64, 256, "even"),
]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "-".join(map(str, c)))
def test_grouped_forward_and_backward(case, kind):
    rows, n_in, n_out, G, how = case
    if kind == "f32":
        n_in, n_out = n_in + 4, n_out + 4
    L = Layer(rows, n_in, n_out, make_offsets(rows, G, how, 1), kind, "silu", bias=True, seed=rows)
    r = Run(L, save="act")
    say(f"[linear] {kind} rows={rows} {n_in}->{n_out} groups={G} {how}")
    r.forward()
    torch.cuda.synchronize()
    r.check_forward()
    r.backward()
    torch.cuda.synchronize()
    r.check_backward()
    assert _mm().moe_get_device_error(r.ws) == 0 and _mm().moe_get_device_error(r.bws) == 0


# large enough for each tile shape and for k in parts, with edges in every
# direction (float64 on the GPU)
LARGE = [
    ("bf16", 8000, 2056, 4000, 1, "even", "int8"),     # 256 x 256 forward and dW
    ("bf16", 9000, 200, 1544, 6, "skewed", "act"),     # 256 x 128
    ("bf16", 6000, 1032, 2056, 5, "gap", "int8"),
    ("bf16", 33000, 72, 264, 9, "skewed", "int8"),     # 128 x 128, dW in parts
    ("bf16", 100, 4104, 2056, 1, "even", "act"),       # few rows, long k in parts
    ("bf16", 3000, 4104, 104, 40, "holes", "act"),
    ("f32", 3000, 516, 1028, 3, "skewed", "act"),
    ("f32", 20000, 100, 68, 1, "even", "int8"),        # dW in parts
    ("f32", 40, 4100, 2052, 2, "even", "act"),
]


@pytest.mark.parametrize("case", LARGE, ids=lambda c: "-".join(map(str, c)))
def test_large_layers(case):
    kind, rows, n_in, n_out, G, how, save = case
    L = Layer(rows, n_in, n_out, make_offsets(rows, G, how, 5), kind, "silu", residual=True, seed=rows, device="cuda")
    r = Run(L, save=save)
    r.forward()
    r.backward()
    torch.cuda.synchronize()
    r.check_forward()
    r.check_backward()
    first = [t.clone() for t in (r.y, r.dx, r.dw, r.db)]
    r.forward()
    r.backward()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((r.y, r.dx, r.dw, r.db), first))  # the same bits


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("fn", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("save", ["none", "act", "int8"])
def test_every_activation_and_way_of_saving(fn, save, kind):
    off = make_offsets(333, 6, "skewed", 3)
    L = Layer(333, 160, 200, off, kind, fn, bias=fn != "relu", seed=5)
    r = Run(L, save=save, grad="f32")
    r.forward()
    torch.cuda.synchronize()
    r.check_forward()
    if fn == "none" or save != "none":
        r.backward()
        torch.cuda.synchronize()
        r.check_backward()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n_in,n_out", [(1, 512, 1024), (2, 4096, 264), (17, 128, 72), (33, 1000, 1336), (64, 2048, 512),
                                             (129, 96, 640), (600, 320, 776)])
def test_dense_with_residual(rows, n_in, n_out, kind):
    L = Layer(rows, n_in, n_out, np.array([0, rows], dtype=np.int32), kind, "gelu", residual=True, seed=rows)
    r = Run(L, save="int8", dense=True)
    r.forward()
    torch.cuda.synchronize()
    r.check_forward()
    r.backward()
    torch.cuda.synchronize()
    r.check_backward()


def small(kind="bf16", fn="silu", save="act", rows=200, n_in=72, n_out=136, groups=5, how="skewed", seed=9, **kw):
    return Run(Layer(rows, n_in, n_out, make_offsets(rows, groups, how, seed), kind, fn, seed=seed, **kw), save=save)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [40, 700])
def test_offsets_out_of_range_or_decreasing_are_reported_and_touch_nothing_else(kind, rows):
    """Offsets are taken into [0, rows] and to the largest so far: the results
    are those of the offsets so cleaned, and the sticky flag is set."""
    mm = _mm()
    bad = np.array([-5, rows // 3, rows // 5, rows // 2, 1 << 30, rows], dtype=np.int32)
    clean = np.array([0, rows // 3, rows // 3, rows // 2, rows, rows], dtype=np.int32)
    L = Layer(rows, 72, 136, clean, kind, "silu", seed=4)
    r = Run(L, save="act")
    r.off = torch.from_numpy(bad).cuda()
    r.forward()
    r.backward()
    torch.cuda.synchronize()
    r.check_forward()
    r.check_backward()
    assert mm.moe_get_device_error(r.ws) == mm.MOE_ERR_BAD_INDEX
    assert mm.moe_get_device_error(r.bws) == mm.MOE_ERR_BAD_INDEX
    r.off = torch.from_numpy(clean).cuda()
    r.forward()
    r.backward()
    assert mm.moe_get_device_error(r.ws) == 0 and mm.moe_get_device_error(r.bws) == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("fn", ["none", "gelu"])
def test_no_rows_zeroes_the_weight_gradients(kind, fn):
    off = np.zeros(4, dtype=np.int32)
    r = Run(Layer(0, 72, 136, off, kind, fn), save="act" if fn != "none" else "none")
    r.forward()
    r.backward()
    torch.cuda.synchronize()
    assert not r.dw.any() and not r.db.any()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_outputs_that_are_not_asked_for_are_not_needed(kind):
    mm = _mm()
    r = small(kind, save="int8")
    r.forward()
    r.backward()
    torch.cuda.synchronize()
    dx, dw, db = r.dx.clone(), r.dw.clone(), r.db.clone()
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 0, 0)):
        got = [torch.full_like(t, 5.0) for t in (dx, dw, db)]
        o = [g if w else None for g, w in zip(got, want)]
        mm.moe_grouped_linear_backward(r.s, r.x if want[1] else None, r.off, r.w if want[0] else None, r.saved, r.dy, *o, r.bws)
        torch.cuda.synchronize()
        for g, ref, w in zip(got, (dx, dw, db), want):
            assert torch.equal(g, ref) if w else bool((g == 5.0).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n_in,n_out", [(72, 136), (40, 264)])
def test_nan_and_infinite_values_stay_in_their_row_group_or_column(kind, n_in, n_out):
    """n_in and n_out end inside a slice of k and inside a tile: the values past
    a row's end are the next row's, and none of them may count."""
    rows, off = 300, np.array([0, 130, 131, 300], dtype=np.int32)
    L = Layer(rows, n_in, n_out, off, kind, "silu", bias=False, seed=2)
    L.x[7], L.x[130], L.w[2, 5], L.dy[140] = float("nan"), float("inf"), float("nan"), float("nan")
    r = Run(L, save="act")
    r.forward()
    r.saved.zero_()  # finite slopes: dz is dy / 2
    r.backward()
    torch.cuda.synchronize()
    y, dx, dw, db = (t.float().cpu() for t in (r.y, r.dx, r.dw, r.db))
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[130]).any()
    fine = torch.ones(rows, dtype=torch.bool)
    fine[[7, 130]] = False
    fine[131:] = False
    assert torch.isfinite(y[fine]).all()
    assert torch.isnan(y[131:, 5]).all() and torch.isfinite(y[131:, [c for c in range(n_out) if c != 5]]).all()
    assert torch.isfinite(dx[:131]).all()
    assert torch.isnan(dx[131:]).all()  # W_2 has a NaN row, and dx sums over all of them
    assert torch.isnan(dw[0]).all() and not torch.isfinite(dw[1]).any() and torch.isnan(dw[2]).all()
    assert torch.isfinite(db[:2]).all() and torch.isnan(db[2]).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("fn", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("rows", [3, 300])
def test_activations_of_infinities_and_large_values(fn, rows, kind):
    """z is the bias alone (x is zero): fn and its slope at infinities, NaN and
    far out, as torch has them."""
    L = Layer(rows, 64, 128, np.array([0, rows], dtype=np.int32), kind, fn, seed=1)
    L.x.zero_()
    L.bias.zero_()
    vals = [float("inf"), float("-inf"), float("nan"), 1e30, -1e30, 90.0, -90.0, 14.0, -14.0]
    L.bias[0, :len(vals)] = torch.tensor(vals)
    L.dy.fill_(1.0)
    r = Run(L, save="act", grad="f32")
    r.forward()
    r.backward()
    torch.cuda.synchronize()
    z = torch.tensor(vals, dtype=torch.float64)
    ref = {"none": z, "relu": torch.relu(z), "gelu": torch.where(z == float("-inf"), 0 * torch.ones_like(z), torch.nn.functional.gelu(z)),
           "silu": torch.where(z == float("-inf"), 0 * torch.ones_like(z), torch.nn.functional.silu(z))}[fn]
    got = r.y[0, :len(vals)].double().cpu()
    zs = r.saved_z()[0, :len(vals)]
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    ok = torch.isfinite(ref)
    assert torch.equal(got[~ok & ~torch.isnan(ref)], ref[~ok & ~torch.isnan(ref)])
    assert ((got[ok] - ref[ok]).abs() <= (HALF[kind] + 1e-6) * ref[ok].abs() + 1e-30).all()
    slope = {"none": torch.ones_like(z), "relu": (zs > 0).double(), "gelu": (zs > 0).double(), "silu": (zs > 0).double()}[fn]
    db = r.db[0, :len(vals)].double().cpu() / rows
    num = ~torch.isnan(zs)
    assert ((db[num] - slope[num]).abs() <= 2e-5).all()  # silu'(+-14) is 1.1e-5 from 0 and 1
    if fn != "none":
        assert torch.isnan(db[2])


@pytest.mark.parametrize("case", [("bf16", 200, 5, "int8"), ("bf16", 1500, 4, "int8"), ("f32", 200, 5, "act"), ("bf16", 20, 3, "act")],
                         ids=str)
def test_captured_and_replayed_with_other_work_between(case):
    """A forward and a backward in one graph, replayed with other inputs and
    other eager calls between; every replay has the eager result's bits."""
    kind, rows, groups, save = case
    r = small(kind, save=save, rows=rows, n_in=264, n_out=328, groups=groups)
    r.forward()
    r.backward()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.forward()
        r.backward()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            r.forward()
            r.backward()
    torch.cuda.synchronize()
    other = small(kind, save=save, rows=rows + 13, n_in=264, n_out=328, groups=groups, seed=31)
    gen = torch.Generator(device="cuda").manual_seed(0)
    for i in range(4):
        r.x.copy_(torch.randn(r.x.shape, device="cuda", generator=gen))
        r.dy.copy_(torch.randn(r.dy.shape, device="cuda", generator=gen))
        r.forward()
        r.backward()
        torch.cuda.synchronize()
        ref = [t.clone() for t in (r.y, r.dx, r.dw, r.db)]
        for t in (r.y, r.dx, r.dw, r.db):
            t.fill_(3.0)
        other.forward()
        other.backward()
        g.replay()
        torch.cuda.synchronize()
        for t, want in zip((r.y, r.dx, r.dw, r.db), ref):
            assert torch.equal(t, want), f"replay {i}"


def test_two_streams_at_once():
    a, b = small(rows=900, n_in=520, n_out=776, groups=3, seed=1), small(rows=800, n_in=520, n_out=776, groups=3, seed=2)
    for r in (a, b):
        r.forward()
        r.backward()
    torch.cuda.synchronize()
    ref = [[t.clone() for t in (r.y, r.dx, r.dw, r.db)] for r in (a, b)]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for r, s in ((a, sa), (b, sb)):
            r.forward(s)
            r.backward(s)
    torch.cuda.synchronize()
    for r, want in zip((a, b), ref):
        assert all(torch.equal(t, w) for t, w in zip((r.y, r.dx, r.dw, r.db), want))


def test_the_residual_may_be_the_output():
    L = Layer(400, 264, 520, np.array([0, 400], dtype=np.int32), "bf16", "gelu", residual=True, seed=6)
    r = Run(L, dense=True)
    r.forward()
    torch.cuda.synchronize()
    want = r.y.clone()
    r.y.copy_(r.residual)
    r.residual = r.y
    r.forward()
    torch.cuda.synchronize()
    assert torch.equal(r.y, want)


def test_one_workspace_for_layers_of_many_shapes():
    """Calls of different shapes, k in parts or whole, take turns on one
    buffer: the header is as before after every call, and so are the bits."""
    mm = _mm()
    shapes = [("f32", 80, 1336, 40, 1), ("bf16", 48, 4096, 1024, 64), ("bf16", 300, 4096, 520, 1), ("f32", 500, 4096, 260, 1),
              ("bf16", 20000, 72, 136, 1), ("f32", 9000, 68, 132, 2), ("bf16", 600, 2048, 264, 7)]
    layers = [Layer(rows, n_in, n_out, make_offsets(rows, G, "skewed" if G > 1 else "even", 3), kind, "gelu", seed=rows,
                    device="cuda") for kind, rows, n_in, n_out, G in shapes]
    runs = [Run(L, save="act") for L in layers]
    ws = torch.randint(0, 256, (max(max(r.ws.numel(), r.bws.numel()) for r in runs),), dtype=torch.uint8, device="cuda")
    mm.moe_workspace_init(ws)
    want = None
    for _ in range(4):
        for r in runs:
            r.ws = r.bws = ws
            r.forward()
            r.backward()
            torch.cuda.synchronize()
            assert not ws[:256].any()
        got = [t.clone() for r in runs for t in (r.y, r.dx, r.dw, r.db)]
        if want is None:
            want = got
            for r in runs:
                r.check_forward()
                r.check_backward()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_operands_past_4_gib():
    """Row offsets past 32 bits: 2.2 million rows of 1024 values, in two groups
    of very different size; checked on the first and the last rows, and the
    weight gradient of the small last group in full."""
    rows, n_in, n_out, last = 2_200_000, 1024, 64, 300
    mm = _mm()
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(rows, n_in, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 200_000):
        x[i:i + 200_000] = torch.randn(min(200_000, rows - i), n_in, device="cuda", generator=g)
    w = (torch.randn(2, n_out, n_in, device="cuda", generator=g) / 32).bfloat16()
    dy = torch.randn(rows, n_out, device="cuda", generator=g).bfloat16()
    off = torch.tensor([0, rows - last, rows], dtype=torch.int32, device="cuda")
    s = mm.make_linear_shape(rows, n_in, n_out, groups=2, grad="f32")
    y, dx = torch.empty(rows, n_out, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    dw = torch.empty(2, n_out, n_in, device="cuda")
    ws, bws = mm.alloc_linear_workspace(s, mm.STAGE_LINEAR), mm.alloc_linear_workspace(s, mm.STAGE_LINEAR_BACKWARD)
    mm.moe_grouped_linear(s, x, off, w, None, None, y, None, ws)
    mm.moe_grouped_linear_backward(s, x, off, w, None, dy, dx, dw, None, bws)
    torch.cuda.synchronize()
    for lo, hi, k in ((0, 200, 0), (rows - last - 100, rows - last, 0), (rows - last, rows, 1)):
        a, b, d = x[lo:hi].double().cpu(), w[k].double().cpu(), dy[lo:hi].double().cpu()
        e = n_in * 2.0 ** -24 * (a.abs() @ b.abs().T)
        ref = a @ b.T
        within(y[lo:hi], ref, e + HALF["bf16"] * (ref.abs() + e), "y")
        e = n_out * 2.0 ** -24 * (d.abs() @ b.abs())
        ref = d @ b
        within(dx[lo:hi], ref, e + HALF["bf16"] * (ref.abs() + e), "dx")
    a, d = x[rows - last:].double().cpu(), dy[rows - last:].double().cpu()
    ref = d.T @ a
    within(dw[1], ref, (last + 2) * 2.0 ** -24 * (d.abs().T @ a.abs()), "dw")


@pytest.mark.parametrize("wanted", ["dx", "dw", "db"])
@pytest.mark.parametrize("rows,fn", [(40, "none"), (40, "silu"), (2500, "none")])
def test_bad_offsets_are_reported_by_each_gradient_alone(rows, fn, wanted):
    mm = _mm()
    bad = np.array([0, rows // 2, rows // 3, rows], dtype=np.int32)
    L = Layer(rows, 72, 136, np.array([0, rows // 2, rows // 2, rows], dtype=np.int32), "bf16", fn, seed=4)
    r = Run(L, save="none" if fn == "none" else "act")
    r.forward()
    r.off = torch.from_numpy(bad).cuda()
    o = [getattr(r, n) if n == wanted else None for n in ("dx", "dw", "db")]
    mm.moe_grouped_linear_backward(r.s, r.x, r.off, r.w, r.saved, r.dy, *o, r.bws)
    assert mm.moe_get_device_error(r.bws) == mm.MOE_ERR_BAD_INDEX


def test_more_rows_than_one_grid_of_the_bias_gradient():
    """2^29 + 96 rows: more blocks of 32 rows than a launch has work-groups of
    256 threads. dy is 1 in a few rows and 0 elsewhere, so the sums are exact."""
    mm = _mm()
    rows, n = 2 ** 29 + 96, 8
    s = mm.make_linear_shape(rows, n, n, fn="relu", save="act", grad="f32")
    saved = mm.alloc_linear_saved(s)
    z = saved[:rows * n * 2].view(torch.bfloat16).view(rows, n)
    z.fill_(1.0)
    dy = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 31, 32, rows // 2, 2 ** 29 - 33, 2 ** 29 - 32, 2 ** 29, rows - 1], device="cuda")
    for c in range(n):
        dy[at[:c + 1], c] = 1.0
    z[at[-1], 7] = -1.0
    db = torch.full((1, n), 9.0, device="cuda")
    ws = mm.alloc_linear_workspace(s, mm.STAGE_LINEAR_BACKWARD)
    mm.moe_linear_backward(s, None, None, saved, dy, None, None, db, ws)
    torch.cuda.synchronize()
    assert db[0].tolist() == [1.0, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0, 7.0]


def _rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_a_layer_of_two_matrix_experts_with_its_backward():
    """The operators as a layer uses them: gate, dispatch, a GELU expert of two
    grouped linear layers (its input rows and pre-activations kept in 8 bits),
    combine and a dense output projection onto the residual stream; and all of
    it backwards. Against float64 autograd with the same routing. Each of the
    five roundings to bf16 on the longest path is off by 2^-9 on average, and
    the 8-bit values by up to 2^-8 of a block's largest: 2e-2, the bound that
    the other layer tests have, covers them with room."""
    mm = _mm()
    T, d, h, E, k = 600, 256, 384, 8, 2
    g = torch.Generator(device="cuda").manual_seed(11)

    def rnd(*s, sigma=1.0):
        return (torch.randn(*s, device="cuda", generator=g) * sigma).bfloat16()
    x, wg, dout = rnd(T, d), rnd(E, d, sigma=0.1), rnd(T, d)
    w1, w2, wo = rnd(E, h, d, sigma=d ** -0.5), rnd(E, d, h, sigma=h ** -0.5), rnd(1, d, d, sigma=d ** -0.5)
    b1, b2, bo = (torch.randn(E, h, device="cuda", generator=g) * 0.1, torch.randn(E, d, device="cuda", generator=g) * 0.1,
                  torch.randn(1, d, device="cuda", generator=g) * 0.1)
    shape = mm.make_shape(T, d, E, k, 0, h, "bf16")
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    idx, counts, off, dest, src = i32(T, k), i32(E), i32(E + 1), i32(T, k), i32(T * k)
    tw = torch.empty(T, k, device="cuda")
    xp = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")
    mm.moe_gate_topk(shape, x, wg, None, idx, tw)
    mm.moe_dispatch(shape, x, idx, counts, off, dest, src, xp, None, mm.alloc_workspace(shape, mm.STAGE_DISPATCH))
    R = T * k
    up = mm.make_linear_shape(R, d, h, groups=E, fn="gelu", save="int8", grad="f32")
    down = mm.make_linear_shape(R, h, d, groups=E, grad="f32")
    proj = mm.make_linear_shape(T, d, d, grad="f32")
    hid, yp = torch.empty(R, h, dtype=torch.bfloat16, device="cuda"), torch.empty_like(xp)
    z8, hid8 = mm.alloc_linear_saved(up), mm.alloc_rows8(R, h)
    y, out = torch.empty_like(x), torch.empty_like(x)
    f, bk = mm.STAGE_LINEAR, mm.STAGE_LINEAR_BACKWARD
    ws = {n: (mm.alloc_linear_workspace(s, f), mm.alloc_linear_workspace(s, bk)) for n, s in (("up", up), ("down", down), ("proj", proj))}
    mm.moe_grouped_linear(up, xp, off, w1, b1, None, hid, z8, ws["up"][0])
    mm.moe_grouped_linear(down, hid, off, w2, b2, None, yp, None, ws["down"][0])
    mm.moe_pack_rows8(hid, hid8)
    hid.fill_(0)  # only its 8 bits are left for the backward
    mm.moe_combine(shape, yp, None, dest, tw, y)
    mm.moe_linear(proj, y, wo, bo, x, out, None, ws["proj"][0])
    # backward
    dy, dyp, dhid, dxp, dx = torch.empty_like(x), torch.empty_like(yp), torch.empty_like(hid), torch.empty_like(xp), torch.empty_like(x)
    dwo, dbo, dw2, db2, dw1, db1 = (torch.empty(t.shape, device="cuda") for t in (wo, bo, w2, b2, w1, b1))
    dtw = torch.empty_like(tw)
    mm.moe_linear_backward(proj, y, wo, None, dout, dy, dwo, dbo, ws["proj"][1])
    mm.moe_combine_backward(shape, dy, yp, dest, tw, dyp, dtw)
    mm.moe_unpack_rows8(hid8, hid)
    mm.moe_grouped_linear_backward(down, hid, off, w2, None, dyp, dhid, dw2, db2, ws["down"][1])
    mm.moe_grouped_linear_backward(up, xp, off, w1, z8, dhid, dxp, dw1, db1, ws["up"][1])
    mm.moe_dispatch_backward(shape, dxp, dout, dest, dx)  # the residual's gradient rides along
    torch.cuda.synchronize()
    # float64, the routing and its weights held fixed
    p = {n: t.double().cpu().requires_grad_() for n, t in dict(x=x, w1=w1, w2=w2, wo=wo, b1=b1, b2=b2, bo=bo, tw=tw).items()}
    ix = idx.long().cpu()
    acc = 0
    for j in range(k):
        zz = torch.einsum("td,thd->th", p["x"], p["w1"][ix[:, j]]) + p["b1"][ix[:, j]]
        oo = torch.einsum("th,tdh->td", torch.nn.functional.gelu(zz), p["w2"][ix[:, j]]) + p["b2"][ix[:, j]]
        acc = acc + p["tw"][:, j:j + 1] * oo
    ref = acc @ p["wo"][0].T + p["bo"][0] + p["x"]
    ref.backward(dout.double().cpu())
    for name, got, want in (("out", out, ref.detach()), ("dx", dx, p["x"].grad), ("dw1", dw1, p["w1"].grad), ("dw2", dw2, p["w2"].grad),
                            ("dwo", dwo, p["wo"].grad), ("db1", db1, p["b1"].grad), ("db2", db2, p["b2"].grad), ("dbo", dbo, p["bo"].grad),
                            ("dtopk_w", dtw, p["tw"].grad)):
        e = _rel(got.cpu(), want)
        say(f"[two-matrix experts] {name}: rel-L2 {e:.2e}")
        assert e <= 2e-2, name
