"""The activation forms on packed int4 codes against the same codes as int8:
the same bits wherever both take the same kernel form."""
import math

import pytest
import torch

import act_reference as ref
from lora_fine_tuning_qlora_b200 import qlora
from test_gpu_act import BF16, F32, _gen, _pack_int4, make_layer

pytestmark = pytest.mark.gpu

# (the forward's CTA-pair kernels differ between the two where N is a multiple
# of 8; everywhere else, and in dX, both take the same form)
INT4 = [(5, 256, 160, 4, BF16), (200, 288, 161, 8, BF16), (150, 96, 72, 4, F32), (2100, 256, 2565, 16, BF16),
        (2100, 256, 2568, 4, BF16), (1100, 1280, 136, 4, BF16), (64, 2048, 2048, 4, BF16), (16, 4096, 1984, 4, BF16),
        (200, 288, 72, 20, BF16), (130, 96, 51, 4, BF16)]


@pytest.mark.parametrize("M,K,N,r,dt", INT4)
def test_int4_codes_give_the_bits_of_the_same_int8_codes(M, K, N, r, dt):
    g = _gen(11)
    L = make_layer(K, N, r, dt, g)
    L.Wq = torch.randint(-8, 8, (N, K), generator=g, device="cuda", dtype=torch.int8)
    L.sw = L.sw * 16
    Wp = _pack_int4(L.Wq)
    X = torch.randn(M, K, generator=g, device="cuda").to(dt)
    R = torch.randn(M, N, generator=g, device="cuda").to(dt)
    d = L.desc()
    _, keep = qlora.forward_act(L, X)
    out = []
    for W in (L.Wq, Wp):
        Y, z = torch.full((M, N), math.nan, dtype=dt, device="cuda"), qlora.ckpt_buffers(M, N)
        qlora.qlora_gemm_forward_act(d, M, keep.Xq, keep.sx, W, L.sw, L.bias, keep.xA, L.B, Y, "gelu", R, z)
        out.append((Y,) + z)
    if dt is BF16 and r <= 16 and N % 8 == 0 and -(-M // 256) * -(-N // 256) >= 74:
        # fp32 sums of the same terms in another order: (r + 8) U of their
        # magnitudes on either side, a slope of at most 1.13, two roundings
        a, b = keep.xA.double().abs(), L.B.double().abs()
        mag = (keep.Xq.double() @ L.Wq.double().t()).abs() * keep.sx.double()[:, None] * L.sw.double()
        mag = mag + L.bias.double().abs() + L.alpha / r * (a @ b)
        e32 = 2 * (1.13 * (r + 8) * ref.U * mag + 2 * ref.U * (mag + R.double().abs()))
        y8, y4 = out[0][0].double(), out[1][0].double()
        assert bool(((y8 - y4).abs() <= e32 + ref.half_step(dt) * (y8.abs() + y4.abs())).all())
        assert int((out[0][1].int() - out[1][1].int()).abs().max()) <= 1
    else:
        assert all(torch.equal(x, y) for x, y in zip(*out))
    dY = (torch.randn(M, N, generator=g, device="cuda") * 0.3).to(dt)
    zk = ref.block_codes(torch.randn(M, K, generator=g, device="cuda"))
    add = torch.randn(M, K, generator=g, device="cuda").to(dt)
    ws = qlora.ckpt_workspace(d, M)
    small = torch.empty(qlora.qlora_workspace_bytes(d, M), dtype=torch.uint8, device="cuda")
    for w in (ws, small):
        qlora.qlora_lora_grad_dy(d, M, dY, L.B, keep.xA, torch.empty(r, N, device="cuda"),
                                 torch.empty(N, device="cuda"), w)
        dX = [torch.full((M, K), math.nan, dtype=dt, device="cuda") for _ in range(2)]
        for W, o in zip((L.Wq, Wp), dX):
            qlora.qlora_gemm_dx_act(d, M, dY, W, L.sw, L.A, o, w, "gelu", zk, add)
        assert torch.equal(*dX)
    assert qlora.qlora_device_status() == 0
