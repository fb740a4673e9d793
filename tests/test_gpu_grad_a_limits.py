"""dA from the kept codes where the int32 sums of its digits come near their
limit, against the exact integers."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from lora_fine_tuning_qlora_b200 import qlora
from test_gpu_act import BF16, _gen, make_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1, -1])
def test_grad_a_with_every_digit_at_its_limit(sign):
    """130944 rows in one CTA with V = +-0x207F7F80 2^-29 throughout: its
    digits are +-(-128, -128, -128, 33), or as near as they come, and with
    codes of +-127 the three low sums reach 127 * 128 * 130944 = 0.991 2^31.
    dA is that integer to its last bit."""
    M, K, r = 1023 * 128 + 5, 16, 4
    V = 0x207F7F80
    L = make_layer(K, 8, r, BF16, _gen(0), alpha=8.0)
    L.B = torch.zeros(r, 8, device="cuda")
    L.B[:, 0] = 1.0
    q = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    q[:, 1::2] = -127
    sx = torch.full((M,), V * 2.0 ** -29, device="cuda")
    assert float(sx[0]) * 2.0 ** 29 == V  # 23 bits: fp32 holds it
    dY = torch.zeros((M, 8), device="cuda", dtype=BF16)
    dY[:, 0] = sign  # G = sign, exactly
    ws = qlora.ckpt_workspace(L.desc(), M)
    prev = qlora.qlora_set_rank_pass_rows(1 << 24)
    try:
        _, dA, _, _ = qlora.backward_ckpt(L, qlora.Checkpoint(q, sx, torch.ones(M, r, device="cuda")), dY, ws,
                                          want_dx=False)
    finally:
        qlora.qlora_set_rank_pass_rows(prev)
    want = float(np.float32(float(Fraction(2 * 127 * V * M, 1 << 29))))  # c = 2
    assert bool((dA[0::2] == sign * want).all()) and bool((dA[1::2] == -sign * want).all())
    assert qlora.qlora_device_status() == 0


def test_grad_a_with_large_sums_of_random_digits():
    """The same rows with scales whose digits differ from row to row: the exact
    integer sum, rounded once."""
    M, K, r = 1023 * 128, 16, 2
    g = _gen(9)
    L = make_layer(K, 8, r, BF16, g)
    L.B = torch.zeros(r, 8, device="cuda")
    L.B[:, 0] = 1.0
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    # V 2^29 = t 2^7 below 2^30: the largest of the column has p = 29
    t = torch.randint(1 << 22, 1 << 23, (M,), generator=g, device="cuda")
    sx = (t.double() * 2.0 ** -22).float()
    dY = torch.zeros((M, 8), device="cuda", dtype=BF16)
    dY[:, 0] = 1
    prev = qlora.qlora_set_rank_pass_rows(1 << 24)
    try:
        _, dA, _, _ = qlora.backward_ckpt(L, qlora.Checkpoint(q, sx, torch.ones(M, r, device="cuda")), dY,
                                          qlora.ckpt_workspace(L.desc(), M), want_dx=False)
    finally:
        qlora.qlora_set_rank_pass_rows(prev)
    sums = (q.long() * t[:, None]).sum(dim=0)  # below 2^23 127 2^17 = 2^47
    want = (sums.double() * (L.alpha / r) * 2.0 ** -22).float()
    assert torch.equal(dA, want[:, None].expand(K, r))
