"""GELU (the normal distribution function) for fp32 activations, to units in the
last place."""
import math

import pytest
import torch

import act_reference as ref
from lora_fine_tuning_qlora_b200 import qlora
from test_gpu_act import F32, _gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(3, 4096), (200, 4096), (2048, 4096), (200, 4001)])
def test_gelu_in_fp32(M, N):
    """z P(z) of z = k / 256, exact biases of a zero kernel on every forward
    form, to a few units in the last place down to P(-8) = 6e-16: P to 10 U,
    the product rounded once, and one more U for P's own value next to it."""
    z = (torch.arange(N, device="cuda") - N // 2) / 256.0
    check_gelu(z, M, 12)


def test_gelu_in_fp32_anywhere():
    """Arguments with 24 bits of their own (few tokens: the bias is added as it
    is): P to the 7 U that its fits and sums leave, one for the product."""
    z = torch.linspace(-12, 12, 16384, device="cuda") + torch.rand(16384, generator=_gen(1), device="cuda") * 1e-3
    check_gelu(z, 1, 8)


def check_gelu(z, M, units):
    N = z.numel()
    L = qlora.Layer(torch.zeros(N, 32, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"), z,
                    torch.zeros(32, 2, device="cuda"), torch.zeros(2, N, device="cuda"), 2.0, F32)
    Y, _ = qlora.forward_act(L, torch.ones(M, 32, device="cuda"), act="gelu")
    want = ref.act("gelu", z.double())
    ref.check(Y, want.expand(M, N), (units * ref.U * want.abs()).expand(M, N), "gelu", floor=2.0 ** -126)


@pytest.mark.parametrize("M,K", [(64, 256), (1600, 784)])
def test_slope_of_gelu_in_fp32(M, K):
    """P(z) + z p(z) of z = q / 16 in dX of a unit kernel: P to 10 U, and of z
    p(z) the exponential (2 units in the last place, 4 U; its argument is
    exact), its constant and two products, 8 U."""
    q = torch.randint(-127, 128, (M, K), generator=_gen(M), device="cuda", dtype=torch.int8)
    zs = torch.full((-(-K // 32), M), 1.0 / 16, device="cuda")
    L = qlora.Layer(torch.eye(K, dtype=torch.int8, device="cuda"), torch.ones(K, device="cuda"), None,
                    torch.zeros(K, 1, device="cuda"), torch.zeros(1, K, device="cuda"), 1.0, F32)
    keep = qlora.Checkpoint(torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda"),
                            torch.zeros(M, 1, device="cuda"))
    dX, *_ = qlora.backward_ckpt(L, keep, torch.ones(M, K, device="cuda"), qlora.ckpt_workspace(L.desc(), M),
                                 act="gelu", z=(q, zs))
    z = q.double() / 16
    P, zp = 0.5 * torch.special.erfc(-z / math.sqrt(2)), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    ref.check(dX, P + zp, 12 * ref.U * P + 10 * ref.U * zp.abs() + 2 * ref.U * (P + zp).abs(), "slope")
