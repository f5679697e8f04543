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
        none = torch.isnan(y[:, 0])  # rows of no group keep what they held
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
        none = torch.isnan(dx[:, 0])
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
