"""The linear layers', the rows8 format's and the 8-bit FFN checkpoints' entry
points validate on the host (no GPU is touched by anything in this file), and
the CPU reference that the GPU results are held to agrees with differences."""

import ctypes

import numpy as np
import pytest
import torch

from linear_util import Layer, fn64, make_offsets, rows8, rows8_read

FAKE = 0x100000  # an aligned, never-dereferenced address: every call below fails validation
P = ctypes.c_void_p(FAKE)
ODD = ctypes.c_void_p(FAKE + 8)


@pytest.fixture(scope="module")
def mm():
    import mixture_experts_routing_gemm_amd as m
    return m


def forward(mm, s, dense=False, x=P, offsets=P, w=P, bias=None, residual=None, y=P, saved=None, saved_bytes=0, ws=P,
            ws_bytes=1 << 40):
    lib = mm._binding.lib
    sp = ctypes.byref(s) if s is not None else None
    if dense:
        return lib.moe_linear(sp, x, w, bias, residual, y, saved, saved_bytes, ws, ws_bytes, None)
    return lib.moe_grouped_linear(sp, x, offsets, w, bias, residual, y, saved, saved_bytes, ws, ws_bytes, None)


def backward(mm, s, dense=False, x=P, offsets=P, w=P, saved=None, saved_bytes=0, dy=P, dx=P, dw=P, db=P, ws=P,
             ws_bytes=1 << 40):
    lib = mm._binding.lib
    sp = ctypes.byref(s) if s is not None else None
    if dense:
        return lib.moe_linear_backward(sp, x, w, saved, saved_bytes, dy, dx, dw, db, ws, ws_bytes, None)
    return lib.moe_grouped_linear_backward(sp, x, offsets, w, saved, saved_bytes, dy, dx, dw, db, ws, ws_bytes, None)


BAD = [
    (dict(rows=-1), -1), (dict(n_in=0), -1), (dict(n_out=-8), -1), (dict(groups=0), -1), (dict(fn=4), -1),
    (dict(fn=-1), -1), (dict(save=3), -1), (dict(act=2), -2), (dict(act="bf16", grad=2), -2), (dict(act="f32", grad="bf16"), -2),
    (dict(n_in=100), -2), (dict(n_out=12), -2), (dict(act="f32", grad="f32", n_in=66), -2), (dict(groups=257), -2),
    (dict(n_in=(1 << 20) + 8), -2), (dict(rows=(1 << 31) - 4095), -2),
]


@pytest.mark.parametrize("kw,status", BAD, ids=str)
def test_bad_linear_shapes_are_refused(mm, kw, status):
    base = dict(rows=64, n_in=128, n_out=256, groups=4, act="bf16", fn="none", save="none", grad="f32")
    base.update(kw)
    s = mm.make_linear_shape(**base)
    assert forward(mm, s) == status
    assert backward(mm, s) == status
    assert mm.moe_linear_workspace_bytes(s, mm.STAGE_LINEAR) == 0
    assert mm.moe_linear_saved_bytes(s) == 0


def test_linear_pointers_workspaces_and_saved_buffers(mm):
    s = mm.make_linear_shape(64, 128, 256, groups=4, fn="gelu", save="int8")
    n = mm.moe_linear_saved_bytes(s)
    assert n == 64 * 256 + 64 * 8 == mm.moe_rows8_bytes(64, 256)
    ok = dict(saved=P, saved_bytes=n)
    for name in ("x", "w", "y", "offsets"):
        assert forward(mm, s, **ok, **{name: None}) == -1
        assert forward(mm, s, **ok, **{name: ODD}) == -1
    assert forward(mm, s, **ok, bias=ODD) == -1
    assert forward(mm, s, **ok, residual=ODD) == -1
    assert forward(mm, None) == -1 and backward(mm, None) == -1
    # saved: missing, not on 256 bytes, short
    assert forward(mm, s) == -1
    assert forward(mm, s, saved=ctypes.c_void_p(FAKE + 16), saved_bytes=n) == -1
    assert forward(mm, s, saved=P, saved_bytes=n - 1) == -1
    assert backward(mm, s) == -1
    assert backward(mm, s, saved=P, saved_bytes=n - 1) == -1
    # an activation's backward needs what the forward saved
    bare = mm.make_linear_shape(64, 128, 256, groups=4, fn="gelu", save="none")
    assert backward(mm, bare) == -1
    # workspaces: missing, misaligned, short
    for stage, call in ((mm.STAGE_LINEAR, forward), (mm.STAGE_LINEAR_BACKWARD, backward)):
        need = mm.moe_linear_workspace_bytes(s, stage)
        assert need >= 256 and need % 256 == 0
        assert call(mm, s, **ok, ws=None) == -3
        assert call(mm, s, **ok, ws=ctypes.c_void_p(FAKE + 16)) == -3
        assert call(mm, s, **ok, ws_bytes=need - 1) == -3
    assert mm.moe_linear_workspace_bytes(s, mm.STAGE_FORWARD) == 0
    for name in ("dy", "w", "x", "offsets"):
        assert backward(mm, s, **ok, **{name: None}) == -1
    for name in ("dx", "dw", "db"):
        assert backward(mm, s, **ok, **{name: ODD}) == -1
    # one weight matrix
    assert forward(mm, s, dense=True, **ok) == -1
    assert backward(mm, s, dense=True, **ok) == -1


def test_linear_without_rows_is_a_no_op_forward(mm):
    s = mm.make_linear_shape(0, 128, 256, groups=4)
    assert forward(mm, s, x=None, offsets=None, w=None, y=None, ws=None, ws_bytes=0) == 0
    assert mm.moe_linear_saved_bytes(mm.make_linear_shape(0, 128, 256, fn="silu", save="act")) == 0


def test_saved_sizes(mm):
    assert mm.moe_linear_saved_bytes(mm.make_linear_shape(3, 8, 40, save="act")) == 256  # 240, rounded up
    assert mm.moe_linear_saved_bytes(mm.make_linear_shape(3, 8, 40, act="f32", save="act")) == 512
    assert mm.moe_linear_saved_bytes(mm.make_linear_shape(3, 8, 40, save="int8")) == 256 + 256
    assert mm.moe_linear_saved_bytes(mm.make_linear_shape(3, 8, 40)) == 0
    # three times less than a, b and hid in bf16: 2 (1 + 1/32) bytes against 6
    s = mm.make_shape(4096, 2048, 32, 8, 2, 1408, "bf16")
    assert abs(mm.moe_ffn_saved8_bytes(s) / mm.moe_ffn_saved_bytes(s) - 2 * 33 / 32 / 6) < 1e-4


def test_rows8_refusals(mm):
    lib = mm._binding.lib
    assert mm.moe_rows8_bytes(5, 33) == 512 + 256
    for rows, n in ((-1, 4), (4, 0), (4, (1 << 20) + 1), (1 << 40, 4)):
        assert mm.moe_rows8_bytes(rows, n) == 0
    size = mm.moe_rows8_bytes(5, 33)
    for call in (lambda r, n, t, x, p, b: lib.moe_pack_rows8(r, n, t, x, p, b, None),
                 lambda r, n, t, x, p, b: lib.moe_unpack_rows8(r, n, t, p, b, x, None)):
        assert call(5, 33, 1, None, P, size) == -1
        assert call(5, 33, 1, ODD, P, size) == -1
        assert call(5, 33, 1, P, None, size) == -1
        assert call(5, 33, 1, P, ctypes.c_void_p(FAKE + 16), size) == -1
        assert call(5, 33, 1, P, P, size - 1) == -1
        assert call(5, 33, 2, P, P, size) == -2
        assert call(-1, 33, 1, P, P, size) == -1
        assert call(5, 0, 1, P, P, size) == -1
        assert call(5, (1 << 20) + 1, 1, P, P, 1 << 40) == -2
        assert call(0, 33, 1, None, None, 0) == 0


def test_saved8_ffn_refusals(mm):
    lib = mm._binding.lib
    s = mm.make_shape(64, 256, 8, 2, 1, 128, "bf16")
    n = mm.moe_ffn_saved8_bytes(s)
    assert n == 2 * mm.moe_rows8_bytes(128, 128) + 2 * mm.moe_rows8_bytes(64, 128)
    sp, wsn = ctypes.byref(s), mm.moe_workspace_bytes(s, mm.STAGE_FFN)
    save = lambda sv, sn, wn=wsn, shape=sp, ysh=P: lib.moe_grouped_ffn_save8(  # noqa: E731
        shape, P, None, P, P, P, P, P, P, ysh, sv, sn, P, wn, None)
    assert save(None, n) == -1
    assert save(ctypes.c_void_p(FAKE + 16), n) == -1
    assert save(P, n - 256) == -1
    assert save(P, n, wsn - 256) == -3
    assert save(P, n, ysh=None) == -1
    bn = mm.moe_workspace_bytes(s, mm.STAGE_FFN_BACKWARD8)
    assert 0 < bn < mm.moe_workspace_bytes(s, mm.STAGE_FFN_BACKWARD)
    back = lambda sv, sn, wn=bn, shape=sp, grad=0, dw=P, dys=P: lib.moe_grouped_ffn_backward_saved8(  # noqa: E731
        shape, P, None, P, P, P, P, P, sv, sn, P, dys, P, P, grad, dw, P, P, P, wn, None)
    assert back(None, n) == -1
    assert back(P, n - 256) == -1
    assert back(P, n, bn - 256) == -3
    assert back(P, n, grad=2) == -2
    assert back(P, n, dw=None) == -1
    assert back(P, n, dys=None) == -1
    for bad in (mm.make_shape(64, 256, 8, 2, 1, 136, "bf16"), mm.make_shape(64, 128, 8, 2, 1, 128, "bf16"),
                mm.make_shape(64, 256, 8, 2, 1, 128, "f32")):
        assert mm.moe_ffn_saved8_bytes(bad) == 0 and mm.moe_workspace_bytes(bad, mm.STAGE_FFN_BACKWARD8) == 0
        assert save(P, n, shape=ctypes.byref(bad)) == -2
        assert back(P, n, shape=ctypes.byref(bad)) == -2
    # rows of 2h values at 4 GiB and more
    assert mm.moe_ffn_saved8_bytes(mm.make_shape(1 << 18, 256, 8, 4, 0, 1024, "bf16")) == 0


def test_the_binding_checks_tensors_before_the_library(mm):
    s = mm.make_linear_shape(4, 8, 16, act="f32", grad="f32")
    x, w, y = torch.zeros(4, 8), torch.zeros(1, 16, 8), torch.zeros(4, 16)
    with pytest.raises(ValueError):  # not on the GPU
        mm.moe_linear(s, x, w, None, None, y, None, None)
    with pytest.raises(ValueError, match="expected 32 values"):
        mm.moe_linear(s, x[:3], w, None, None, y, None, None)
    with pytest.raises(ValueError, match="x"):
        mm.moe_linear(s, x.bfloat16(), w, None, None, y, None, None)
    with pytest.raises(ValueError, match="offsets"):
        mm.moe_grouped_linear_backward(s, x, None, w, None, y, x, w, None, None)
    with pytest.raises(mm.MoEError):
        mm.alloc_linear_workspace(mm.make_linear_shape(4, 9, 16), mm.STAGE_LINEAR)
    with pytest.raises(mm.MoEError):
        mm.moe_pack_rows8(torch.zeros(2, 4, dtype=torch.float64), torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mm.moe_pack_rows8(torch.zeros(4), torch.zeros(512, dtype=torch.uint8))


# ------------------------------------------------------ the reference itself --
@pytest.mark.parametrize("fn", ["relu", "gelu", "silu", "none"])
def test_the_reference_slopes_are_differences(fn):
    z = torch.linspace(-6, 6, 240, dtype=torch.float64) + 0.0123  # (no point at relu's corner)
    h = 1e-5
    d = (fn64(fn, z + h)[0] - fn64(fn, z - h)[0]) / (2 * h)
    assert float((d - fn64(fn, z)[1]).abs().max()) < 1e-9  # h^2 / 6 of the third derivative, and 1e-16 / h


def test_the_reference_gradients_are_differences():
    L = Layer(7, 8, 16, make_offsets(7, 3, "holes", 1), "f32", "gelu", bias=True, seed=3)
    _, z, _, _ = L.forward()
    dx, dw, db, *_ = L.backward(z, "f32")

    def loss():
        return float((torch.nan_to_num(L.forward()[0]) * L.dy.double()).sum())
    for t, g in ((L.x, dx), (L.w, dw), (L.bias, db)):
        flat, grad = t.view(-1), torch.nan_to_num(g).reshape(-1)
        for i in np.random.default_rng(0).choice(flat.numel(), 12, replace=False):
            keep = float(flat[i])
            step = []
            for s in (1, -1):
                flat[i] = keep + s * 2.0 ** -8
                step.append((float(flat[i]), loss()))
            flat[i] = keep
            (xa, la), (xb, lb) = step
            # a third derivative below 8 times the weights involved
            assert abs((la - lb) / (xa - xb) - float(grad[i])) < 8 * 2.0 ** -16


def test_the_reference_format_by_brute_force():
    r = np.random.default_rng(1)
    v = r.standard_normal((40, 70)) * np.exp(4 * r.standard_normal((40, 1)))
    v[3] = 0.0
    out, step = rows8(v)
    for c in range(0, 70, 32):
        b, s = v[:, c:c + 32], step[:, c:c + 32]
        top = np.abs(b).max(1)
        assert (top <= 127 * s[:, 0]).all()
        assert ((top > 127 * s[:, 0] / 2) | (s[:, 0] == 2.0 ** -126)).all()  # no smaller step would do
    assert (np.abs(out - v) <= step / 2).all() and (np.abs(out / step) <= 127).all()
    assert (out == np.round(out / step) * step).all()


def test_the_layout_reader():
    codes = np.zeros((2, 64), dtype=np.int8)
    codes[0, 0], codes[1, 33] = -127, 5
    buf = np.zeros(512, dtype=np.uint8)
    buf[:128] = codes.view(np.uint8).reshape(-1)
    buf[256:260] = [128, 127, 127, 125]
    v, _ = rows8_read(torch.from_numpy(buf), 2, 40)
    assert v[0, 0] == -254.0 and v[1, 33] == 1.25
