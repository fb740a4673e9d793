"""The layer with activation, residual and 8-bit checkpoints on the GPU,
against the plain 64-bit reference of act_reference.py."""
import math

import pytest
import torch

import act_reference as ref
from lora_fine_tuning_qlora_b200 import qlora

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_layer(K, N, r, act, g, alpha=8.0, bias=True):
    def normal(*s, std=1.0):
        return torch.randn(*s, generator=g, device="cuda") * std

    w, sw = ref.row_codes(normal(N, K, std=0.05))
    return qlora.Layer(Wq=w, sw=sw, bias=normal(N, std=0.1) if bias else None, A=normal(K, r, std=1 / math.sqrt(K)),
                       B=normal(r, N, std=0.1), alpha=alpha, act=act)


def run_forward(M, K, N, r, dt, name, residual, save, seed=0, **kw):
    g = _gen(seed)
    L = make_layer(K, N, r, dt, g, **kw)
    X = torch.randn(M, K, generator=g, device="cuda").to(dt)
    R = torch.randn(M, N, generator=g, device="cuda").to(dt) if residual else None
    Y, keep = qlora.forward_act(L, X, act=name, residual=R, save_z=save)
    y, z, y_err, z_err, xa, xa_err, q, sx = ref.forward(X, L.Wq, L.sw, L.bias, L.A, L.B, L.alpha / r, name, R)
    assert torch.equal(keep.Xq, q) and torch.equal(keep.sx, sx)
    ref.check(keep.xA, xa, xa_err, "xA")
    ref.check(Y, y, y_err, "Y")
    if save:
        # the scale follows the block's maximum; a code is off by half a step,
        # and by what Z itself may be off
        nb = keep.zs.shape[0]
        pad = torch.zeros((M, nb * 32), dtype=torch.float64, device="cuda")
        err = torch.zeros_like(pad)
        pad[:, :N], err[:, :N] = z, z_err
        top = pad.view(M, nb, 32).abs().amax(dim=2).t()
        s_err = err.view(M, nb, 32).amax(dim=2).t() / 127 + 2 * ref.U * top / 127
        ref.check(keep.zs, top / 127, s_err, "zs")
        zv = ref.block_values(keep.zq, keep.zs)
        step = keep.zs.double().t().repeat_interleave(32, dim=1)[:, :N]
        ref.check(zv, z, (0.5 + 128 * ref.U) * step + z_err, "z")
    assert qlora.qlora_device_status() == 0
    return L, X, Y, keep


# tokens on the MMA's N (1 .. 64), split-K, 64- and 128-column tiles, CTA
# pairs; widths that end inside a tile, a checkpoint block and a 16-byte chunk
FORWARD = [
    (1, 2048, 1000, 4), (1, 16, 1, 1), (7, 784, 130, 3), (16, 4096, 512, 4), (17, 96, 33, 8), (64, 528, 257, 16),
    (65, 784, 128, 4), (100, 4096, 128, 8), (130, 2048, 200, 16), (333, 784, 1001, 8), (300, 272, 96, 20),
    (128, 144, 40, 64), (513, 1040, 3000, 4), (2048, 272, 2600, 4), (2050, 512, 2568, 16), (1600, 256, 3333, 8),
]


@pytest.mark.parametrize("M,K,N,r", FORWARD)
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_forward_shapes(M, K, N, r, dt):
    run_forward(M, K, N, r, dt, "gelu_tanh", True, True, seed=M + N)


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("residual,save", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("M,K,N,r,dt", [(5, 272, 160, 4, BF16), (200, 272, 160, 4, BF16), (200, 272, 160, 4, F32),
                                        (2048, 144, 2560, 4, BF16)])
def test_forward_epilogues(M, K, N, r, dt, name, residual, save):
    run_forward(M, K, N, r, dt, name, residual, save, seed=7, bias=residual)


def run_backward(M, K, N, r, dt, name, add, seed=0, z=None, dY=None, want_dx=True):
    g = _gen(seed)
    L = make_layer(K, N, r, dt, g)
    X = torch.randn(M, K, generator=g, device="cuda").to(dt)
    q, sx = ref.row_codes(X)
    xA = X.float() @ L.A
    if dY is None:
        dY = (torch.randn(M, N, generator=g, device="cuda") * 0.3).to(dt)
    if z is None:
        z = ref.block_codes(torch.randn(M, K, generator=g, device="cuda") * 1.5)
    extra = torch.randn(M, K, generator=g, device="cuda").to(dt) if add else None
    ws = qlora.ckpt_workspace(L.desc(), M, "cuda")
    ws.fill_(0xA5)
    keep = qlora.Checkpoint(q, sx, xA)
    dX, dA, dB, dbias = qlora.backward_ckpt(L, keep, dY, ws, act=name, z=z, add=extra, want_dx=want_dx)
    want = ref.backward(dY, q, sx, L.Wq, L.sw, L.A, L.B, xA, L.alpha / r, name, z, extra)
    for key, got in (("dX", dX), ("dA", dA), ("dB", dB), ("dbias", dbias)):
        if got is not None:
            ref.check(got, *want[key], key)
    assert qlora.qlora_device_status() == 0
    return L, keep, dY, z, extra, ws, (dX, dA, dB, dbias)


BACKWARD = [
    (1, 16, 8, 1), (1, 2048, 512, 4), (16, 1024, 2048, 4), (17, 784, 136, 3), (64, 528, 264, 16), (65, 784, 128, 4),
    (127, 48, 64, 8), (129, 272, 200, 16), (333, 784, 1000, 8), (300, 272, 96, 20), (140, 144, 40, 33),
    (256, 144, 72, 64), (77, 160, 10, 4), (1024, 2576, 128, 4), (1030, 2560, 192, 16), (2500, 528, 320, 8),
]


@pytest.mark.parametrize("M,K,N,r", BACKWARD)
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_backward_shapes(M, K, N, r, dt):
    run_backward(M, K, N, r, dt, "gelu", True, seed=M + K)


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("M,K,N,r,dt", [(5, 272, 160, 4, BF16), (200, 272, 160, 4, BF16), (200, 272, 50, 4, F32),
                                        (200, 272, 51, 4, BF16), (1024, 2560, 64, 4, BF16)])
def test_backward_epilogues(M, K, N, r, dt, name, add):
    run_backward(M, K, N, r, dt, name, add, seed=3)


@pytest.mark.parametrize("M,N", [(1, 1), (3, 31), (1, 32), (9, 33), (37, 1030), (128, 4096), (1000, 80), (5, 16384)])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_checkpoint_bits(M, N, dt):
    g = _gen(M * N)
    T = (torch.randn(M, N, generator=g, device="cuda") * torch.logspace(-3, 3, M, device="cuda")[:, None]).to(dt)
    q, s = qlora.ckpt_save(T)
    rq, rs = ref.block_codes(T)
    assert torch.equal(q, rq) and torch.equal(s, rs)
    for out in (BF16, F32):
        back = qlora.ckpt_load(q, s, out)
        assert torch.equal(back, (q.float() * s.t().repeat_interleave(32, dim=1)[:, :N]).to(out))
    rowq, sx = ref.row_codes(T)
    assert torch.equal(qlora.ckpt_load(rowq, sx, dt), (rowq.float() * sx[:, None]).to(dt))
