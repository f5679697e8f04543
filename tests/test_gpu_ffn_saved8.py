"""The SwiGLU expert stage with its pre-activations kept in 8 bits: the forward's
results are those of moe_grouped_ffn, the kept values are the float64 ones
within half a step, and the backward's gradients are those of the formulas at
the kept values, element by element within bounds derived from the arithmetic."""

from __future__ import annotations

import pytest
import torch

from gpu_util import requires_gpu, say
from linear_util import SLOPE_ERR, U32, fn64, make_offsets, rows8_read, within

pytestmark = [pytest.mark.gpu, requires_gpu]
H16 = 2.0 ** -8


def _mm():
    import mixture_experts_routing_gemm_amd as mm
    return mm


class Case:
    def __init__(self, T, d, E, k, S, h, how, fp8=False, seed=0):
        mm = _mm()
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, sigma=1.0: (torch.randn(*s, generator=g) * sigma).to(torch.bfloat16)  # noqa: E731
        self.T, self.d, self.E, self.k, self.S, self.h = T, d, E, k, S, h
        self.off = make_offsets(T * k, E, how, seed)
        self.x, self.x_perm = rnd(T, d), rnd(T * k, d)
        self.w1, self.w3 = rnd(E + S, h, d, sigma=d ** -0.5), rnd(E + S, h, d, sigma=d ** -0.5)
        self.w2 = rnd(E + S, d, h, sigma=h ** -0.5)
        self.dy, self.dys = rnd(T * k, d, sigma=0.2), rnd(T, d, sigma=0.2)
        self.shape = mm.make_shape(T, d, E, k, S, h, "bf16", dispatch="fp8" if fp8 else None)
        c = lambda t: t.cuda()  # noqa: E731
        self.dev = {n: c(getattr(self, n)) for n in ("x", "x_perm", "w1", "w3", "w2", "dy", "dys")}
        self.qp = None
        if fp8:
            # rows whose codes and (scale, centre) are drawn directly
            codes = torch.randint(0, 127, (T * k, d), generator=g).to(torch.uint8)
            codes[codes == 127] = 0
            self.qp = torch.stack([torch.full((T * k,), 1.0 / 256), torch.randn(T * k, generator=g) * 0.1], 1).float()
            val = codes.view(torch.float8_e4m3fn).float() * self.qp[:, :1] + self.qp[:, 1:]
            self.x_perm = val.to(torch.bfloat16)
            self.dev["x_perm"], self.qp = c(codes), c(self.qp)
        self.offd = torch.from_numpy(self.off).cuda()
        self.saved = mm.alloc_saved8(self.shape)
        self.saved.fill_(0x33)
        f = lambda r, dt=torch.bfloat16: torch.full((r, d), 77.0, dtype=dt, device="cuda")  # noqa: E731
        self.y, self.dx = f(T * k), f(T * k)
        self.ys, self.dxs = (f(T), f(T)) if S else (None, None)
        self.ws, self.bws = mm.alloc_workspace(self.shape, mm.STAGE_FFN), mm.alloc_workspace(self.shape, mm.STAGE_FFN_BACKWARD8)

    def forward(self, which="save8"):
        mm, v = _mm(), self.dev
        args = (self.shape, v["x_perm"], self.qp, self.offd, v["x"] if self.S else None, v["w1"], v["w3"], v["w2"], self.y,
                self.ys)
        if which == "save8":
            mm.moe_grouped_ffn_save8(*args, self.saved, self.ws)
        else:
            mm.moe_grouped_ffn(*args, self.ws)

    def backward(self, grad):
        mm, v = _mm(), self.dev
        t = torch.float32 if grad == "f32" else torch.bfloat16
        G = self.E + self.S
        dw = [torch.full(s, 7.0, dtype=t, device="cuda") for s in ((G, self.h, self.d), (G, self.h, self.d), (G, self.d, self.h))]
        mm.moe_grouped_ffn_backward_saved8(self.shape, v["x_perm"], self.qp, self.offd, v["x"] if self.S else None, v["w1"],
                                           v["w3"], v["w2"], self.saved, v["dy"], v["dys"] if self.S else None, self.dx,
                                           self.dxs, grad, *dw, self.bws)
        return dw

    def kept(self):
        """a and b as the four rows8 buffers say: routed, shared."""
        mm, R, SH = _mm(), self.T * self.k, self.S * self.h
        n = mm.moe_rows8_bytes(R, self.h)
        out = [rows8_read(self.saved[i * n:(i + 1) * n], R, self.h)[0] for i in range(2)]
        if self.S:
            m = mm.moe_rows8_bytes(self.T, SH)
            out += [rows8_read(self.saved[2 * n + i * m:2 * n + (i + 1) * m], self.T, SH)[0] for i in range(2)]
        return [torch.from_numpy(o) for o in out]

    def groups(self):
        """(group, input rows, output gradients, slice of rows, shared index)"""
        for g in range(self.E):
            lo, hi = int(self.off[g]), int(self.off[g + 1])
            if hi > lo:
                yield g, self.x_perm[lo:hi].double(), self.dy[lo:hi].double(), slice(lo, hi), None
        for s in range(self.S):
            yield self.E + s, self.x.double(), self.dys.double(), slice(0, self.T), s


CASES = [
    (1, 256, 2, 1, 0, 128, "first", False),
    (130, 256, 4, 2, 1, 128, "skewed", False),
    (77, 512, 3, 2, 2, 384, "holes", False),
    (300, 256, 8, 4, 0, 640, "last", False),
    (200, 256, 4, 2, 1, 256, "skewed", True),
    (4000, 512, 4, 2, 2, 640, "skewed", False),  # the larger tiles
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_saved8_forward_and_backward(case):
    T, d, E, k, S, h, how, fp8 = case
    say(f"[ffn saved8] {case}")
    c = Case(T, d, E, k, S, h, how, fp8, seed=T)
    c.forward("plain")
    torch.cuda.synchronize()
    y, ys = c.y.clone(), None if c.ys is None else c.ys.clone()
    c.y.fill_(77.0)
    c.forward()
    torch.cuda.synchronize()
    assert torch.equal(y, c.y) and (ys is None or torch.equal(ys, c.ys))
    kept = c.kept()
    for g, v, _, rows, s in c.groups():
        for which, w in ((0, c.w1), (1, c.w3)):
            got = kept[which][rows] if s is None else kept[2 + which][:, s * h:(s + 1) * h]
            ref, size = v @ w[g].double().T, v.abs() @ w[g].double().abs().T
            e = d * U32 * size
            top = (ref.abs() + e).reshape(len(ref), -1, 32).amax(2).repeat_interleave(32, 1)
            within(got, ref, e + top / 127.0, f"kept {'ab'[which]} of group {g}")

    for grad in ("f32", "bf16"):
        half = U32 if grad == "f32" else H16
        dw = c.backward(grad)
        torch.cuda.synchronize()
        dxs = exs = torch.zeros(T, d).double()
        for g, v, dy, rows, s in c.groups():
            w1, w3, w2 = c.w1[g].double(), c.w3[g].double(), c.w2[g].double()
            pick = (lambda i: kept[i][rows]) if s is None else (lambda i: kept[2 + i][:, s * h:(s + 1) * h])
            a, b = pick(0), pick(1)
            u, du = fn64("silu", a)
            dh, edh = dy @ w2, d * U32 * (dy.abs() @ w2.abs())
            eu = 24 * U32 * a.abs()
            rounded = lambda t, e: e + H16 * (t.abs() + e)  # noqa: E731
            hid = u * b
            ehid = rounded(hid, b.abs() * eu + U32 * hid.abs())
            da, db = dh * b * du, dh * u
            eda = rounded(da, (edh * du.abs() + dh.abs() * SLOPE_ERR["silu"]) * b.abs() + 3 * U32 * da.abs())
            edb = rounded(db, edh * u.abs() + (dh.abs() + edh) * eu + 2 * U32 * db.abs())
            dx = da @ w1 + db @ w3
            ex = (eda + h * 2 * U32 * (da.abs() + eda)) @ w1.abs() + (edb + h * 2 * U32 * (db.abs() + edb)) @ w3.abs()
            if s is None:
                within(c.dx[rows], dx, rounded(dx, ex), f"dx of group {g}")
            else:
                dxs, exs = dxs + dx, exs + 2 * ex
            n = len(v)
            for name, got, lhs, elhs, rhs, erhs in (("dw1", dw[0], da, eda, v, 0 * v), ("dw3", dw[1], db, edb, v, 0 * v),
                                                    ("dw2", dw[2], dy, 0 * dy, hid, ehid)):
                ref = lhs.T @ rhs
                e = elhs.T @ (rhs.abs() + erhs) + lhs.abs().T @ erhs + n * U32 * ((lhs.abs() + elhs).T @ (rhs.abs() + erhs))
                within(got[g], ref, e + half * (ref.abs() + e), f"{name} of group {g}")
        if S:
            within(c.dxs, dxs, exs + H16 * (dxs.abs() + exs), "dx_shared")
        for g in range(E):
            if c.off[g] == c.off[g + 1]:
                assert not any(t[g].any() for t in dw)
        again = c.backward(grad)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(dw, again))


def test_no_tokens_zeroes_the_weight_gradients():
    mm = _mm()
    s = mm.make_shape(0, 256, 4, 2, 1, 128, "bf16")
    for grad, t in (("f32", torch.float32), ("bf16", torch.bfloat16)):
        dw = [torch.full((5, 128, 256), 7.0, dtype=t, device="cuda") for _ in range(2)]
        dw.append(torch.full((5, 256, 128), 7.0, dtype=t, device="cuda"))
        w = [torch.ones_like(v, dtype=torch.bfloat16) for v in dw]
        mm.moe_grouped_ffn_save8(s, None, None, None, None, *w, None, None, None, None)
        mm.moe_grouped_ffn_backward_saved8(s, None, None, None, None, *w, None, None, None, None, None, grad, *dw, None)
        torch.cuda.synchronize()
        assert not any(v.any() for v in dw)


def test_saved8_captured_and_replayed():
    """Forward and backward in one graph, replayed on other inputs with eager
    calls between: every replay has the eager result's bits."""
    c, other = Case(260, 512, 4, 2, 1, 256, "skewed", seed=3), Case(130, 512, 4, 2, 1, 256, "even", seed=4)
    mm, v = _mm(), c.dev
    dw = [torch.empty_like(v[n]) for n in ("w1", "w3", "w2")]

    def step():
        c.forward()
        mm.moe_grouped_ffn_backward_saved8(c.shape, v["x_perm"], None, c.offd, v["x"], v["w1"], v["w3"], v["w2"], c.saved, v["dy"],
                                           v["dys"], c.dx, c.dxs, "bf16", *dw, c.bws)
    outs = [c.y, c.ys, c.dx, c.dxs, *dw]
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.synchronize()
    gen = torch.Generator(device="cuda").manual_seed(0)
    for i in range(4):
        for n in ("x", "x_perm", "dy", "dys"):
            v[n].copy_(torch.randn(v[n].shape, device="cuda", generator=gen))
        step()
        torch.cuda.synchronize()
        ref = [t.clone() for t in outs]
        for t in outs:
            t.fill_(3.0)
        other.forward()
        other.backward("f32")
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref)), f"replay {i}"
