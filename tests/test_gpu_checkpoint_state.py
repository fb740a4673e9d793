"""A Checkpoint offers only what its last forward wrote."""
import pytest
import torch

from lora_fine_tuning_qlora_b200 import qlora
from test_gpu_act import BF16, _gen, make_layer

pytestmark = pytest.mark.gpu


def test_a_forward_without_z_takes_back_the_z_of_an_earlier_one():
    M, K, N = 40, 64, 96
    g = _gen(1)
    below, above = make_layer(K, N, 4, BF16, g), make_layer(N, K, 4, BF16, g)
    X = torch.randn(2, M, K, generator=g, device="cuda").to(BF16)
    H, keep = qlora.forward_act(below, X[0], act="silu", save_z=True)
    first = keep.z
    assert first[0] is keep.zq and first[1] is keep.zs
    # other tokens through the same checkpoint, their Z not kept
    H, again = qlora.forward_act(below, X[1], act="silu", keep=keep)
    assert again is keep and keep.z is None
    Y, kept = qlora.forward_act(above, H)
    ws = qlora.ckpt_workspace(above.desc(), M)
    with pytest.raises(ValueError, match="needs z"):
        qlora.backward_ckpt(above, kept, Y, ws, act="silu", z=keep.z)
    # kept again, into the same buffers
    qlora.forward_act(below, X[1], act="silu", save_z=True, keep=keep)
    assert keep.z[0] is first[0] and keep.z[1] is first[1]
    qlora.backward_ckpt(above, kept, Y, ws, act="silu", z=keep.z)
    _, fresh = qlora.forward_act(below, X[1], act="silu", save_z=True)
    assert torch.equal(fresh.zq, keep.zq) and torch.equal(fresh.zs, keep.zs)


def test_a_given_z_counts():
    M, K, N = 8, 32, 40
    L = make_layer(K, N, 4, BF16, _gen(2))
    X = torch.randn(M, K, device="cuda").to(BF16)
    keep = qlora.Checkpoint.allocate(M, K, 4)
    assert keep.z is None
    qlora.forward_act(L, X, keep=keep)
    assert keep.z is None
    keep.zq, keep.zs = qlora.ckpt_save(torch.randn(M, N, device="cuda").to(BF16))  # the caller's own
    assert keep.z is not None
    given = qlora.Checkpoint(keep.Xq, keep.sx, keep.xA, keep.zq, keep.zs)
    assert given.z is not None
    with pytest.raises(ValueError, match="save_z needs"):
        qlora.forward_act(L, X, save_z=True, keep=qlora.Checkpoint.allocate(M, K, 4))


def test_a_refused_forward_leaves_no_valid_z():
    """A refused call may have begun to write: its Z does not count."""
    M, K, N = 8, 32, 40
    L = make_layer(K, N, 4, BF16, _gen(2))
    X = torch.randn(M, K, device="cuda").to(BF16)
    _, keep = qlora.forward_act(L, X, act="relu", save_z=True)
    odd = torch.empty(M * K + 4, dtype=BF16, device="cuda")[4:].view(M, K)  # 8-byte aligned
    with pytest.raises(qlora.QLoraError):
        qlora.forward_act(L, odd, act="relu", save_z=True, keep=keep)
    assert keep.z is None
    with pytest.raises(ValueError):  # refused before anything is touched
        qlora.forward_act(L, X.float(), keep=keep)
    qlora.forward_act(L, X, act="relu", save_z=True, keep=keep)
    assert keep.z is not None
    with pytest.raises(ValueError):
        qlora.forward_act(L, X.float(), act="relu", save_z=True, keep=keep)
    assert keep.z is not None
