"""An infinity or a NaN in the layer's input shows in everything that is made
from its row: the row's scale, what the kept codes read back as, the output
and dA; the other rows keep their bits."""
import math

import pytest
import torch

import act_reference as ref
from lora_fine_tuning_qlora_b200 import qlora
from test_gpu_act import BF16, F32, _gen, make_layer

pytestmark = pytest.mark.gpu

# every form of the input quantizer: a row over a cluster (up to one row per
# SM), whole rows per warp (from 2^24 bf16 elements), and the general kernels:
# rows per 32 to 256 threads, A in slices, rows of more than 16384 elements,
# rows staged by bulk copies (from 2^25 elements)
FORMS = [(1, 2048, 4, BF16), (100, 784, 8, F32), (148, 8208, 16, BF16), (12, 96, 3, F32),
         (16400, 1024, 4, BF16), (9000, 1920, 8, BF16), (4100, 4096, 4, BF16), (4100, 4096, 8, BF16),
         (200, 272, 4, BF16), (333, 784, 8, F32), (300, 4112, 16, BF16), (200, 8192, 4, F32), (160, 96, 20, F32),
         (160, 16400, 20, BF16), (150, 17000 // 16 * 16, 33, F32), (200, 16384, 4, BF16)]
# the composite backward has no limit that these meet; the general kernels for
# many rows are reached by the step-level call alone
STAGED = [(33000, 1024, 4), (33000, 1024, 8), (17000, 2048, 4), (8300, 4096, 4), (17000, 2048, 8)]


def poison(X):
    """NaN and infinities in some rows; {row: whether it holds a NaN}."""
    M, K = X.shape
    cases = [((0, math.nan),), ((K - 1, math.nan),), ((K // 2, -math.inf),), ((3, math.inf), (K - 2, math.nan)),
             ((K // 3, -math.nan),), tuple((k, math.nan) for k in range(K))]
    rows = {}
    for i, case in enumerate(cases if M >= 12 else cases[:1]):
        m = i * (M // len(cases)) if M >= 12 else 0
        for k, v in case:
            X[m, k] = v
        rows[m] = any(math.isnan(v) for _, v in case)
    if M >= 12:
        X[M - 1, K - 1], rows[M - 1] = math.nan, True
    return rows


def check_codes(Xq, sx, X, rows):
    nan = torch.zeros(X.shape[0], dtype=torch.bool, device="cuda")
    inf = torch.zeros_like(nan)
    for m, is_nan in rows.items():
        (nan if is_nan else inf)[m] = True
    assert torch.equal(sx.isnan(), nan) and torch.equal(sx.isinf(), inf)
    assert int(Xq[nan | inf].abs().sum()) == 0
    fine = ~(nan | inf)
    q, s = ref.row_codes(torch.where(fine[:, None], X, torch.zeros_like(X)))
    assert torch.equal(Xq[fine], q[fine]) and torch.equal(sx[fine], s[fine])
    return fine


@pytest.mark.parametrize("M,K,r,dt", FORMS)
def test_a_nan_or_an_infinity_in_a_row(M, K, r, dt):
    N = 48
    g = _gen(M + K)
    L = make_layer(K, N, r, dt, g)
    X = torch.randn(M, K, generator=g, device="cuda").to(dt)
    clean, _ = qlora.forward_act(L, X, act="silu")
    rows = poison(X)
    Y, keep = qlora.forward_act(L, X, act="silu", save_z=True)
    fine = check_codes(keep.Xq, keep.sx, X, rows)
    assert torch.equal(Y[fine], clean[fine]) and not bool(Y[~fine].isfinite().any())
    assert bool(keep.zs[:, ~fine].isnan().all()) and not bool(keep.zs[:, fine].isnan().any())
    back = qlora.ckpt_load(keep.Xq, keep.sx, F32)
    assert bool(back[~fine].isnan().all()) and bool(back[fine].isfinite().all())
    dY = torch.randn(M, N, generator=g, device="cuda").to(dt)
    _, dA, _, _ = qlora.backward_ckpt(L, keep, dY, qlora.ckpt_workspace(L.desc(), M))
    assert bool(dA.isnan().all())
    # the step-level quantizer keeps the same codes
    Xq, sx = torch.empty_like(keep.Xq), torch.empty_like(keep.sx)
    qlora.qlora_quantize_input(L.desc(), M, X, L.A, Xq, sx, torch.empty(M, r, device="cuda"))
    assert torch.equal(Xq, keep.Xq) and torch.equal(sx.nan_to_num(nan=-1.0), keep.sx.nan_to_num(nan=-1.0))
    assert qlora.qlora_device_status() == 0


@pytest.mark.parametrize("M,K,r", STAGED)
def test_the_quantizer_for_many_rows(M, K, r):
    L = make_layer(K, 16, r, BF16, _gen(K))
    X = torch.randn(M, K, generator=_gen(M), device="cuda").to(BF16)
    rows = poison(X)
    Xq, sx = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    qlora.qlora_quantize_input(L.desc(), M, X, L.A, Xq, sx, torch.empty(M, r, device="cuda"))
    check_codes(Xq, sx, X, rows)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_the_layer_of_such_rows_is_what_it_was(dt):
    """The plain layer: such rows' outputs are NaN, the others' bits stay."""
    M, K, N = 300, 272, 96
    g = _gen(3)
    L = make_layer(K, N, 4, dt, g)
    X = torch.randn(M, K, generator=g, device="cuda").to(dt)
    ws = qlora.ckpt_workspace(L.desc(), M)
    clean, _ = qlora.forward(L, X, ws)
    rows = poison(X)
    Y, _ = qlora.forward(L, X, ws)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[list(rows)] = True
    assert bool(Y[bad].isnan().all()) and torch.equal(Y[~bad], clean[~bad])
