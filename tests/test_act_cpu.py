"""Activation epilogues and 8-bit checkpoints without a GPU: the C ABI's
refusals (made before anything is launched), the binding's, and the 64-bit
reference that the GPU tests compare with, against differences."""
import ctypes
import math

import pytest
import torch

import act_reference as ref

BF16 = torch.bfloat16
P = 1 << 20  # an aligned address that no call reads: every call here is refused


@pytest.fixture(scope="module")
def q():
    from lora_fine_tuning_qlora_b200 import build
    build.build()
    from lora_fine_tuning_qlora_b200 import qlora
    return qlora


def forward_act(q, M=16, act=1, res=None, zq=None, zs=None, X=P, Y=2 * P, Xq=3 * P, d=None, ep=True):
    d = d if d is not None else q.desc(64, 48, 4, 8.0, BF16)
    e = ctypes.byref(q.FwdEpilogue(act, res, zq, zs)) if ep else None
    return q.lib().qlora_forward_act(ctypes.byref(d), M, X, P, P, P, P, P, e, Y, Xq, P, P, None)


def gemm_act(q, name="qlora_gemm_forward_act", M=16, act=1, res=None, zq=None, zs=None, Wq=P, K=64):
    d = q.desc(K, 48, 4, 8.0, BF16)
    e = ctypes.byref(q.FwdEpilogue(act, res, zq, zs))
    return getattr(q.lib(), name)(ctypes.byref(d), M, P, P, Wq, P, P, P, P, e, 2 * P, None)


def backward(q, M=16, act=0, zq=None, zs=None, add=None, Xq=P, ws=P, nbytes=1 << 30, d=None):
    d = d if d is not None else q.desc(64, 48, 4, 8.0, BF16)
    e = ctypes.byref(q.DxEpilogue(act, zq, zs, add))
    return q.lib().qlora_backward_ckpt(ctypes.byref(d), M, Xq, P, P, P, P, P, P, P, e, 2 * P, P, P, P, ws, nbytes, None)


EINVAL, EALIGN, ESHAPE, EUNSUPPORTED = -1, -2, -3, -5


def test_forward_refusals(q):
    assert forward_act(q, act=5) == EINVAL and forward_act(q, act=-1) == EINVAL
    assert forward_act(q, ep=False) == EINVAL
    assert forward_act(q, zq=P) == EINVAL and forward_act(q, zs=P) == EINVAL
    assert forward_act(q, zq=2 * P, zs=P) == EINVAL                     # the codes over Y
    assert forward_act(q, res=P + 8) == EALIGN and forward_act(q, zq=P + 8, zs=P) == EALIGN
    assert forward_act(q, zq=P, zs=P + 2) == EALIGN
    assert forward_act(q, X=None) == EINVAL and forward_act(q, X=P + 4) == EALIGN
    assert forward_act(q, Xq=P + 4) == EALIGN and forward_act(q, Y=P + 2) == EALIGN
    assert forward_act(q, M=-1) == ESHAPE
    assert forward_act(q, d=q.desc(72, 48, 4, 8.0, BF16)) == EUNSUPPORTED
    assert forward_act(q, M=0) == 0


def test_gemm_refusals(q):
    for name in ("qlora_gemm_forward_act", "qlora_gemm_forward_act_int4"):
        assert gemm_act(q, name, act=7) == EINVAL
        assert gemm_act(q, name, res=P + 4) == EALIGN
        assert gemm_act(q, name, Wq=P + 4) == EALIGN
        assert gemm_act(q, name, zq=P) == EINVAL
        assert gemm_act(q, name, M=0) == 0
    assert gemm_act(q, "qlora_gemm_forward_act_int4", K=48) == EUNSUPPORTED
    d = q.desc(64, 48, 4, 8.0, BF16)
    for name in ("qlora_gemm_dx_act", "qlora_gemm_dx_act_int4"):
        f = getattr(q.lib(), name)

        def dx(act=0, zq=None, zs=None, add=None, nbytes=1 << 30, M=16):
            e = ctypes.byref(q.DxEpilogue(act, zq, zs, add))
            return f(ctypes.byref(d), M, P, P, P, P, e, 2 * P, P, nbytes, None)

        assert dx(act=1) == EINVAL and dx(act=1, zq=P) == EINVAL and dx(act=9, zq=P, zs=P) == EINVAL
        assert dx(act=1, zq=P + 8, zs=P) == EALIGN and dx(add=P + 8) == EALIGN
        assert dx(nbytes=16) == EINVAL and dx(M=0) == 0
        assert f(ctypes.byref(d), 16, P, P, P, P, None, 2 * P, P, 1 << 30, None) == EINVAL


def test_backward_refusals(q):
    assert backward(q, act=2) == EINVAL and backward(q, act=2, zq=P) == EINVAL
    assert backward(q, act=2, zq=P + 4, zs=P) == EALIGN and backward(q, add=P + 4) == EALIGN
    assert backward(q, Xq=P + 4) == EALIGN and backward(q, ws=P + 16) == EALIGN
    assert backward(q, Xq=None) == EINVAL
    assert backward(q, nbytes=64) == EINVAL
    assert backward(q, M=1047553) == EUNSUPPORTED
    d = q.desc(64, 48, 4, 8.0, BF16)
    x = q.lib().qlora_lora_grad_x_ckpt
    assert x(ctypes.byref(d), 16, P, P, P, P, 64, None) == EINVAL
    assert x(ctypes.byref(d), 16, P + 1, P, P, P, 1 << 30, None) == EALIGN
    assert x(ctypes.byref(d), 1 << 21, P, P, P, P, 1 << 40, None) == EUNSUPPORTED


def test_checkpoint_refusals(q):
    save, load = q.lib().qlora_ckpt_save, q.lib().qlora_ckpt_load
    assert save(P, 4, 0, 0, P, P, None) == ESHAPE and save(P, -1, 4, 0, P, P, None) == ESHAPE
    assert save(P, 4, 4, 3, P, P, None) == EINVAL and save(None, 4, 4, 0, P, P, None) == EINVAL
    assert save(P + 8, 4, 4, 0, P, P, None) == EALIGN and save(P, 4, 4, 0, P + 8, P, None) == EALIGN
    assert load(P, P, 4, 4, 16, 0, P, None) == EUNSUPPORTED
    assert save(P, 0, 4, 0, P, P, None) == 0 and load(P, P, 0, 4, 32, 0, P, None) == 0


def test_overlap_and_row_limit_refusals(q):
    """Outputs over inputs that are still read, and row counts that would leave
    the kernels' 32-bit block counts or the grid."""
    assert forward_act(q, zq=3 * P, zs=P) == EINVAL and forward_act(q, Xq=2 * P) == EINVAL
    assert forward_act(q, M=(1 << 30) + 1) == ESHAPE and gemm_act(q, M=2147483647) == ESHAPE
    assert backward(q, act=2, zq=2 * P, zs=P) == EINVAL and backward(q, Xq=2 * P) == EINVAL
    d = q.desc(64, 48, 4, 8.0, BF16)
    e = ctypes.byref(q.DxEpilogue(0, None, None, None))
    for M, dX, code in ((16, P, EINVAL), (4194241, 2 * P, ESHAPE)):
        assert q.lib().qlora_gemm_dx_act(ctypes.byref(d), M, P, P, P, P, e, dX, P, 1 << 40, None) == code
    for save in (q.lib().qlora_ckpt_save, lambda *a: q.lib().qlora_ckpt_load(a[0], a[4], a[1], a[2], 32, a[3], *a[5:])):
        for rows, cols in ((2147483647, 1), (1, 2147483647)):
            assert save(P, rows, cols, 0, P, P, None) == ESHAPE


def test_sizes(q):
    lib = q.lib()
    assert lib.qlora_ckpt_scales(5, 32) == 5 and lib.qlora_ckpt_scales(5, 33) == 10
    assert lib.qlora_ckpt_scales(0, 33) == 0 and lib.qlora_ckpt_scales(3, 0) == 0
    assert lib.qlora_ckpt_scales(1 << 20, 1 << 20) == (1 << 20) * (1 << 15)
    d = q.desc(1024, 1024, 8, 8.0, BF16)
    n = q.qlora_ckpt_workspace_bytes(d, 300)
    assert n >= q.qlora_workspace_bytes(d, 300) + 3 * 128 * 32 and n % 256 == 0
    assert q.qlora_ckpt_workspace_bytes(d, 1047552) > 0 and q.qlora_ckpt_workspace_bytes(d, 1047553) == 0
    # the de-quantized kernel's room, for many tokens of a bf16 layer only
    big = q.desc(4096, 4096, 4, 8.0, BF16)
    assert q.qlora_ckpt_workspace_bytes(big, 4096) >= q.qlora_workspace_bytes(big, 4096) + 2 * 4096 * 4096
    f32 = q.desc(4096, 4096, 4, 8.0, torch.float32)
    assert q.qlora_ckpt_workspace_bytes(f32, 4096) < q.qlora_workspace_bytes(f32, 4096) + 4096 * 4096


def test_binding_refusals(q):
    X = torch.zeros(4, 32, dtype=BF16)
    L = q.Layer(torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8), None, torch.zeros(32, 4), torch.zeros(4, 8), 8.0,
                BF16)
    with pytest.raises(ValueError, match="CUDA"):
        q.forward_act(L, X)
    with pytest.raises(ValueError, match="act must be"):
        q.forward_act(L, X, act="tanh")
    with pytest.raises(ValueError, match="CUDA"):
        q.ckpt_save(X)
    k = q.Checkpoint.allocate(5, 32, 3, "cpu")
    assert k.Xq.shape == (5, 32) and k.sx.shape == (5,) and k.xA.shape == (5, 3) and k.z is None
    addr = k._addresses(5, 32, 3, torch.device("cpu"))
    assert addr == (k.Xq.data_ptr(), k.sx.data_ptr(), k.xA.data_ptr()) and addr[0] % 16 == 0
    with pytest.raises(ValueError, match="Xq must be"):
        k._addresses(5, 48, 3, torch.device("cpu"))
    from lora_fine_tuning_qlora_b200.feedforward import FeedForward
    with pytest.raises(ValueError, match="same width"):
        FeedForward(L, L, 4, device="cpu")


@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu", "none"])
def test_reference_slope_is_the_difference_quotient(name):
    z = torch.linspace(-9, 9, 4001, dtype=torch.float64)
    z = z[(z.abs() > 1e-3)] if name == "relu" else z
    h = 1e-4
    num = (ref.act(name, z + h) - ref.act(name, z - h)) / (2 * h)
    # h^2 / 6 times a third derivative below 3, and 64-bit rounding over 2 h
    assert (num - ref.slope(name, z)).abs().max() <= h * h / 2 + 10 * 2.0 ** -53 / h


def test_reference_gradients_are_the_difference_quotients():
    """dX, dA, dB and dbias of the reference against differences of sum(dY * Y0)
    with Y0 = X Wd + bias + c (X A) B at X = Xq sx, which is linear in each."""
    g = torch.Generator().manual_seed(3)
    M, K, N, r, c = 7, 48, 10, 3, 2.0
    X = torch.randn(M, K, generator=g)
    q_, sx = ref.row_codes(X)
    Wq, sw = ref.row_codes(torch.randn(N, K, generator=g) * 0.1)
    A, B, bias = torch.randn(K, r, generator=g), torch.randn(r, N, generator=g), torch.randn(N, generator=g)
    dY = torch.randn(M, N, generator=g)
    x = q_.double() * sx.double()[:, None]
    xA = (x @ A.double()).float()

    def f(X_, A_, B_, b_):
        return ((X_ @ (Wq.double() * sw.double()[:, None]).t() + b_ + c * (X_ @ A_) @ B_) * dY.double()).sum()

    got = ref.backward(dY, q_, sx, Wq, sw, A, B, xA, c, "none", None, None)
    args = [x, A.double(), B.double(), bias.double()]
    for i, key in enumerate(("dX", "dA", "dB", "dbias")):
        for e in range(0, args[i].numel(), max(1, args[i].numel() // 5)):
            up, dn = [a.clone() for a in args], [a.clone() for a in args]
            up[i].view(-1)[e] += 0.5
            dn[i].view(-1)[e] -= 0.5
            # xA in fp32: half a step of each of the M terms of dB
            tol = 1e-9 + (2.0 ** -24 * c * (xA.double().abs().t() @ dY.double().abs()).max() if key == "dB" else 0)
            assert abs(float(f(*up) - f(*dn)) - float(got[key][0].flatten()[e])) <= float(tol)


def test_reference_codes():
    z = torch.tensor([[1.0, -127.0, 0.5, 63.5] + [0.0] * 30])
    codes, s = ref.block_codes(z)
    assert s.shape == (2, 1) and float(s[0, 0]) == 1.0 and float(s[1, 0]) == 0.0
    assert codes[0, :4].tolist() == [1, -127, 0, 64]  # ties to even
    bad = torch.tensor([[math.inf] + [1.0] * 31, [math.nan] + [1.0] * 31, [1e-31] * 32])
    codes, s = ref.block_codes(bad)
    assert codes.abs().sum() == 0 and torch.isnan(s[0, :2]).all() and float(s[0, 2]) == 0.0
