"""What dX from 8-bit checkpoints multiplies dY with in bf16: the kernel rounded
to bf16, the layer's rule for its input gradient."""
import pytest
import torch

import act_reference as ref
from lora_fine_tuning_qlora_b200 import qlora
from test_gpu_act import BF16, _gen, make_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N,r,add", [(16, 4096, 4096, 4, False), (1001, 784, 1000, 8, True),
                                         (1024, 2560, 512, 4, False), (2048, 2064, 1032, 16, True),
                                         (200, 272, 51, 4, False), (300, 272, 96, 20, True)])
def test_bf16_dx_multiplies_with_the_kernel_rounded_to_bf16(M, K, N, r, add):
    """dX is the formula's with bf16(Wq sw) in the place of Wq sw, to the fp32
    sums and the output's rounding; against Wq sw itself it differs by the
    kernel's rounding and by no more; and a second call on other scratch gives
    the same bits."""
    g = _gen(M)
    L = make_layer(K, N, r, BF16, g)
    X = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    q, sx = ref.row_codes(X)
    dY = (torch.randn(M, N, generator=g, device="cuda") * 0.3).to(BF16)
    z = ref.block_codes(torch.randn(M, K, generator=g, device="cuda") * 1.5)
    extra = torch.randn(M, K, generator=g, device="cuda").to(BF16) if add else None
    keep = qlora.Checkpoint(q, sx, X.float() @ L.A)
    ws = qlora.ckpt_workspace(L.desc(), M)
    ws.fill_(0x5A)
    dX, *_ = qlora.backward_ckpt(L, keep, dY, ws, act="silu", z=z, add=extra)
    ws.fill_(0xA5)
    again, *_ = qlora.backward_ckpt(L, keep, dY, ws, act="silu", z=z, add=extra)
    assert torch.equal(dX, again)
    dy, c = dY.double(), L.alpha / r
    G, g_mag = dy @ L.B.double().t(), dy.abs() @ L.B.double().abs().t()
    zv = ref.block_values(*z)
    sl = ref.slope("silu", zv)
    arg = zv.abs()
    sl_err = 2.0 ** -21 * (4 + 4 * arg) * (1 + arg)
    for W, kernel_err in (((L.Wq.float() * L.sw[:, None]).to(BF16).double(), 0.0),
                          (L.Wq.double() * L.sw.double()[:, None], ref.half_step(BF16))):
        dx = dy @ W + c * (G @ L.A.double().t())
        err = (kernel_err + (N + 4) * ref.U) * (dy.abs() @ W.abs())
        err = err + c * (((N + 12) * ref.U + 2.1 * ref.TF32 + (r + 4) * ref.U) * (g_mag @ L.A.double().abs().t()))
        err = (err + 2 * ref.U * dx.abs()) * sl.abs() + (dx.abs() + err) * sl_err
        want = dx * sl
        if add:
            want = want + extra.double()
        err = err + 2 * ref.U * want.abs()
        ref.check(dX, want, err + ref.half_step(BF16) * (want.abs() + err), "dX")
