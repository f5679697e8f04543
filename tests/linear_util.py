"""A float64 linear layer with its gradients, the rows8 format from its
definition, and the error bounds the GPU results are held to."""

from __future__ import annotations

import math

import numpy as np
import torch

U32 = 2.0 ** -24                                  # half a step of float32
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}     # half a step of an output
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# |fn(z) computed - fn(z)| <= FN_ERR[fn] |z|, and the same for the slope, as an
# absolute value. relu: exact. silu: exp, its argument, the reciprocal, two
# roundings: under 8 float32 half-steps for the |z| <= 16 of the tests, where
# exp's relative error is at most |z| half-steps more: 24. gelu: erf's formula
# is off by 1.5e-7, half of which reaches Phi, and its evaluation adds a few
# half-steps of values below 1 (1e-6 in all covers both); the slope adds z
# times the density's error, under |z| e^(-z^2/2) (z^2 + 8) half-steps < 20.
FN_ERR = {"none": 0.0, "relu": 0.0, "silu": 24 * U32, "gelu": 1e-6}
SLOPE_ERR = {"none": 0.0, "relu": 0.0, "silu": 64 * U32, "gelu": 3e-6}
LIPSCHITZ = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13}
# |fn''| is at most this: how far the slope moves when z does
CURVE = {"none": 0.0, "relu": 0.0, "silu": 0.5, "gelu": 0.8}


def fn64(name, z):
    """(fn(z), fn'(z)) in float64."""
    if name == "relu":
        return torch.clamp(z, min=0.0), (z > 0).double()
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * c, c + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    return z, torch.ones_like(z)


def rows8(v):
    """v (numpy float64 [rows, n], finite) through the 8-bit row format: the values
    read back, and the step of every value."""
    out, steps = np.empty_like(v), np.empty_like(v)
    for c in range(0, v.shape[1], 32):
        b = v[:, c:c + 32]
        top = np.abs(b).max(1)
        e = np.full(top.shape, -126)
        while True:
            low = top > 127.0 * np.ldexp(1.0, e)
            if not low.any():
                break
            e = np.where(low, e + 1, e)
        s = np.ldexp(1.0, e)[:, None]
        out[:, c:c + 32] = np.rint(b / s) * s
        steps[:, c:c + 32] = s
    return out, steps


def rows8_read(packed, rows, n):
    """The values a packed buffer (uint8 tensor) stands for, by the documented layout."""
    n32 = (n + 31) // 32 * 32
    p = packed.cpu().numpy()
    codes = p[:rows * n32].view(np.int8).reshape(rows, n32).astype(np.float64)
    at = (rows * n32 + 255) // 256 * 256
    sc = p[at:at + rows * (n32 // 32)].reshape(rows, n32 // 32).astype(np.int64)
    step = np.where(sc == 255, np.nan, np.ldexp(1.0, np.minimum(sc, 254) - 127))
    return (codes.reshape(rows, -1, 32) * step[:, :, None]).reshape(rows, n32), codes


def make_offsets(rows, groups, kind, seed=0):
    """Ragged group offsets: "even", "skewed", "last" (every row in the last
    group), "first", "holes" (every other group empty), "gap" (rows before the
    first and after the last group belong to none)."""
    r = np.random.default_rng(seed)
    p = np.ones(groups)
    lo, hi = 0, rows
    if kind == "skewed":
        p = 1.0 / np.arange(1, groups + 1) ** 1.5
    elif kind == "last":
        p = (np.arange(groups) == groups - 1).astype(float)
    elif kind == "first":
        p = (np.arange(groups) == 0).astype(float)
    elif kind == "holes":
        p = (np.arange(groups) % 2 == 0).astype(float)
    elif kind == "gap":
        lo, hi = rows // 5, rows - rows // 4
    counts = r.multinomial(hi - lo, p / p.sum())
    return np.concatenate([[lo], lo + np.cumsum(counts)]).astype(np.int32)


class Layer:
    """Inputs of one layer, on the CPU or (large ones) the GPU, and what float64 says of it."""

    def __init__(self, rows, n_in, n_out, offsets, kind="bf16", fn="none", bias=True, residual=False, seed=0,
                 device="cpu"):
        g = torch.Generator(device=device).manual_seed(seed)
        G = len(offsets) - 1
        t = TYPES[kind]

        def rnd(*s, sigma=1.0):
            return (torch.randn(*s, generator=g, device=device) * sigma)
        self.rows, self.n_in, self.n_out, self.offsets, self.kind, self.fn = rows, n_in, n_out, offsets, kind, fn
        self.x = rnd(rows, n_in).to(t)
        self.w = rnd(G, n_out, n_in, sigma=n_in ** -0.5).to(t)
        self.bias = rnd(G, n_out, sigma=0.3) if bias else None
        self.residual = rnd(rows, n_out).to(t) if residual else None
        self.dy = rnd(rows, n_out, sigma=0.3).to(t)

    def groups(self):
        for g in range(len(self.offsets) - 1):
            lo, hi = int(self.offsets[g]), int(self.offsets[g + 1])
            if hi > lo:
                yield g, lo, hi

    def forward(self):
        """y, z and the bounds of their errors; None rows stay NaN."""
        nan = lambda: torch.full((self.rows, self.n_out), float("nan"), dtype=torch.float64, device=self.x.device)  # noqa: E731
        y, z, ey, ez = nan(), nan(), nan(), nan()
        for g, lo, hi in self.groups():
            x, w = self.x[lo:hi].double(), self.w[g].double()
            zz, size = x @ w.T, x.abs() @ w.abs().T
            if self.bias is not None:
                zz = zz + self.bias[g].double()
                size = size + self.bias[g].double().abs()
            # a float32 sum of n_in products and a bias, in any order
            ez[lo:hi] = (self.n_in + 1) * U32 * size
            f, _ = fn64(self.fn, zz)
            e = LIPSCHITZ[self.fn] * ez[lo:hi] + FN_ERR[self.fn] * zz.abs()
            if self.residual is not None:
                f = f + self.residual[lo:hi].double()
                e = e + 2 * U32 * (f.abs() + self.residual[lo:hi].double().abs())
            z[lo:hi], y[lo:hi] = zz, f
            ey[lo:hi] = e + HALF[self.kind] * (f.abs() + e)
        return y, z, ey, ez

    def backward(self, zs, grad):
        """dx, dw, db and their bounds, from the saved pre-activations zs."""
        G = len(self.offsets) - 1
        f64 = dict(dtype=torch.float64, device=self.x.device)
        dx = torch.full((self.rows, self.n_in), float("nan"), **f64)
        ex = dx.clone()
        dw, ew = torch.zeros(G, self.n_out, self.n_in, **f64), torch.zeros(G, self.n_out, self.n_in, **f64)
        db, eb = torch.zeros(G, self.n_out, **f64), torch.zeros(G, self.n_out, **f64)
        zs = None if zs is None else zs.to(self.x.device)
        half_in = HALF[self.kind] if self.fn != "none" else 0.0  # dz is rounded to the act type
        for g, lo, hi in self.groups():
            x, w, dy = self.x[lo:hi].double(), self.w[g].double(), self.dy[lo:hi].double()
            slope = torch.ones_like(dy) if self.fn == "none" else fn64(self.fn, zs[lo:hi])[1]
            dz = dy * slope
            edz = dy.abs() * SLOPE_ERR[self.fn] + (2 * U32) * dz.abs()  # in float32
            if self.fn == "none":
                edz = torch.zeros_like(dz)
            er = edz + half_in * (dz.abs() + edz)  # as rounded
            n = hi - lo
            dx[lo:hi] = dz @ w
            e = er @ w.abs() + self.n_out * U32 * ((dz.abs() + er) @ w.abs())
            ex[lo:hi] = e + HALF[self.kind] * (dx[lo:hi].abs() + e)
            dw[g] = dz.T @ x
            e = er.T @ x.abs() + n * U32 * ((dz.abs() + er).T @ x.abs())
            ew[g] = e + HALF[grad] * (dw[g].abs() + e)
            db[g] = dz.sum(0)
            e = edz.sum(0) + n * U32 * (dz.abs() + edz).sum(0)
            eb[g] = e + HALF[grad] * (db[g].abs() + e)
        return dx, dw, db, ex, ew, eb


def within(got, ref, bound, what):
    """got within the bound of ref, element by element, where ref is a number."""
    got, ref, bound = got.double().cpu(), ref.cpu(), bound.cpu()
    there = ~torch.isnan(ref)
    assert torch.isfinite(got[there]).all(), f"{what}: not finite"
    over = (got[there] - ref[there]).abs() - bound[there]
    if over.numel():
        worst = float(((got[there] - ref[there]).abs() / bound[there].clamp(min=1e-300)).max())
        print(f"{what}: largest error is {worst:.3f} of its bound", flush=True)
        assert float(over.max()) <= 0.0, f"{what}: {worst:.3f} times the bound"
