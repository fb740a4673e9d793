"""Plain 64-bit reference of the layer with activation, residual and 8-bit
checkpoints, with elementwise bounds on what a kernel may be off by.

Nothing here calls the library.  All of it is torch in float64 (the quantizers
in float32, whose operations the definition fixes), on the device of its
inputs.

Bounds.  u = 2^-24 is half a step of fp32 relative to a value, h half a step of
the activation dtype (bf16 2^-8, fp32 2^-24).  A sum of n products in fp32 is
off by at most (n + 2) u times the sum of the magnitudes, whatever its order.
"""
import math

import torch

U = 2.0 ** -24
TF32 = 2.0 ** -11      # half a step of tf32 relative to a value
BLOCK = 32


def half_step(dtype):
    return {torch.bfloat16: 2.0 ** -8, torch.float32: U}[dtype]


def row_codes(x):
    """The input quantizer in fp32, one rounding per operation."""
    x = x.float()
    amax = x.abs().amax(dim=1)
    inv = torch.where(amax > 0, torch.full_like(amax, 127.0) / amax, torch.zeros_like(amax))
    return torch.round(x * inv[:, None]).clamp(-127, 127).to(torch.int8), amax / torch.full_like(amax, 127.0)


def block_codes(z):
    """8-bit checkpoint of z in fp32: codes [M, N], scales [ceil(N/32), M]."""
    z = z.float()
    M, N = z.shape
    nb = -(-N // BLOCK)
    zp = torch.zeros((M, nb * BLOCK), dtype=torch.float32, device=z.device)
    zp[:, :N] = z
    zp = zp.view(M, nb, BLOCK)
    amax = zp.abs().amax(dim=2)
    bad = ~torch.isfinite(zp).all(dim=2)
    tiny = amax < 2.0 ** -100
    keep = ~(bad | tiny)
    safe = torch.where(keep, amax, torch.ones_like(amax))
    inv = torch.full_like(safe, 127.0) / safe
    q = torch.round(torch.where(keep[:, :, None], zp, torch.zeros_like(zp)) * inv[:, :, None]).clamp(-127, 127)
    s = torch.where(keep, safe / torch.full_like(safe, 127.0), torch.zeros_like(safe))
    s = torch.where(bad, torch.full_like(s, math.nan), s)
    return q.view(M, nb * BLOCK)[:, :N].to(torch.int8), s.t().contiguous()


def block_values(q, s):
    N = q.shape[1]
    return q.double() * s.double().t().repeat_interleave(BLOCK, dim=1)[:, :N]


def act(name, z):
    if name == "relu":
        return z.clamp_min(0)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        s = torch.sigmoid(2 * k * (z + 0.044715 * z ** 3))
        return s + z * s * (1 - s) * 2 * k * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def forward(X, Wq, sw, bias, A, B, c, name, residual):
    """(Y, Z, bound on Y, bound on Z, xA, bound on xA, codes, scales)."""
    dt = X.dtype
    q, sx = row_codes(X)
    x, a, b = X.double(), A.double(), B.double()
    K, r = A.shape
    xa = x @ a
    xa_err = (K + 2) * U * (x.abs() @ a.abs())
    acc = q.double() @ Wq.double().t()
    main = acc * sx.double()[:, None] * sw.double()
    bs = bias.double() if bias is not None else torch.zeros_like(sw.double())
    z = main + bs + c * (xa @ b)
    # the main term: the accumulator to fp32, two products, one sum; the rank-r
    # sum and the bias: operands in tf32 (bf16 outputs: one half step each of
    # both factors) or in split tf32 (fp32 outputs: the products of the two
    # remainders are dropped and the remainders themselves are tf32, 4 TF32^2),
    # r + 2 fp32 sums of their magnitudes
    lora = abs(c) * (xa.abs() @ b.abs()) + bs.abs()
    part = 2.1 * TF32 if dt == torch.bfloat16 else 4 * TF32 ** 2
    z_err = 6 * U * main.abs() + (part + (r + 6) * U) * lora + abs(c) * (xa_err @ b.abs()) + U * z.abs()
    y = act(name, z)
    # slopes of the activations are below 1.13; their fp32 evaluation: 1.5e-7
    # (the erf approximation) or the two hardware functions (each within 2^-22)
    # times an argument of at most 2 |z| (1 + 0.045 min(z^2, 30)) where the
    # result is not saturated, times |z|
    arg = z.abs() * (1 + 0.045 * (z * z).clamp_max(30.0))
    y_err = 1.13 * z_err + z.abs() * (2.0 ** -22 * (2 + 2 * arg.clamp_max(40.0)) + 1.5e-7) if name != "none" else z_err
    if residual is not None:
        y = y + residual.double()
    y_err = y_err + U * y.abs()
    y_err = y_err + half_step(dt) * (y.abs() + y_err)
    return y, z, y_err, z_err, xa, xa_err, q, sx


def backward(dY, q, sx, Wq, sw, A, B, xA, c, name, z, add):
    """{name: (value, bound)} of dX, dA, dB, dbias; z = (zq, zs) or None."""
    dt = dY.dtype
    dy, a, b = dY.double(), A.double(), B.double()
    M, N = dY.shape
    r = A.shape[1]
    w = Wq.double() * sw.double()[:, None]
    G = dy @ b.t()
    # 24-bit factors: fp32 sums, and the factor's own third term dropped below 2^-24
    # (r > 32 in bf16: 16 bits)
    factor = 2.0 ** -16 if (dt == torch.bfloat16 and r > 32) else 2 * U
    g_mag = dy.abs() @ b.abs().t()
    g_err = ((N + 10) * U + factor) * g_mag
    dx = dy @ w + c * (G @ a.t())
    # the de-quantized kernel in bf16 on the tensor cores, one fp32 rounding else
    dx_err = (half_step(dt) + (N + 4) * U) * (dy.abs() @ w.abs())
    part = 2.1 * TF32 if dt == torch.bfloat16 else 0.0
    dx_err = dx_err + abs(c) * ((g_err + (part + (r + 4) * U) * g_mag) @ a.abs().t()) + 2 * U * dx.abs()
    if name != "none":
        zv = block_values(*z)
        sl = slope(name, zv)
        arg = zv.abs() * (1 + 0.045 * (zv * zv).clamp_max(30.0))
        sl_err = 2.0 ** -21 * (4 + 4 * zv.abs().clamp_max(40.0)) * (1 + arg.clamp_max(40.0)) + 3e-7
        dx_err = dx_err * sl.abs() + (dx.abs() + dx_err) * sl_err
        dx = dx * sl
    if add is not None:
        dx = dx + add.double()
    dx_err = dx_err + 2 * U * dx.abs()
    dx_err = dx_err + half_step(dt) * (dx.abs() + dx_err)
    x = q.double() * sx.double()[:, None]
    da = c * (x.t() @ G)
    V = sx.double()[:, None] * G
    # sx G in fp32 (one rounding) and to 31 bits below its column's maximum, exact sums, one rounding
    v_err = sx.double()[:, None] * g_err + 2 * U * V.abs() + 2.0 ** -29 * V.abs().amax(dim=0, keepdim=True)
    da_err = abs(c) * (q.double().abs().t() @ v_err) + 3 * U * da.abs()
    db = c * (xA.double().t() @ dy)
    db_err = ((M + 10) * U + factor) * abs(c) * (xA.double().abs().t() @ dy.abs()) + 2 * U * db.abs()
    dbias = dy.sum(dim=0)
    dbias_err = (M + 10) * U * dy.abs().sum(dim=0)
    return {"dX": (dx, dx_err), "dA": (da, da_err), "dB": (db, db_err), "dbias": (dbias, dbias_err)}


def check(got, want, err, what, floor=1e-30):
    """got within err of want everywhere (err elementwise, plus underflow)."""
    off = (got.double() - want).abs()
    bad = ~(off <= err + floor)
    if bad.any():
        i = int(torch.argmax((off / (err + floor)).nan_to_num(nan=float("inf")).flatten()))
        raise AssertionError("%s: %d of %d off; worst at %d: got %r, want %r, allowed %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got.flatten()[i]), float(want.flatten()[i]),
            float(err.expand_as(want).flatten()[i])))
