"""Operators of int8-LoRA training with fused epilogues and 8-bit activation
checkpoints, as one pass each on the GPU: what they are given, their plain
form in elementary torch operations, their definition in 64 bits, and the
bytes and operations that a pass cannot do without.

Three operators:

``forward``   Y = act(Z) + R with Z = (Xq Wq^T) sx sw + bias + c (X A) B, the
              int8 Dense layer with activation and residual; with ``save`` it
              keeps its input as the row codes (Xq, sx) and Z in 8 bits.
``backward``  the layer's gradients from such checkpoints: dX = (dY (Wq sw)^T
              + c G A^T) * act'(z) + add, z the 8-bit pre-activation of the
              layer below; dA = c X^T G with X = Xq sx; dB, dbias; G = dY B^T.
``checkpoint``an activation stored in 8 bits (one scale per 32 columns of a
              row) and read back.
"""
import math

import torch

own = False

BLOCK = 32  # columns of a row that share a scale in an 8-bit checkpoint
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ cases
def _forward(name, M, K, N, r, act, residual, save, dtype="bf16"):
    return {"name": name, "op": "forward", "M": M, "K": K, "N": N, "r": r, "act": act,
            "residual": residual, "save": save, "dtype": dtype}


def _backward(name, M, K, N, r, act, add, dtype="bf16"):
    return {"name": name, "op": "backward", "M": M, "K": K, "N": N, "r": r, "act": act, "add": add,
            "dtype": dtype}


def _checkpoint(name, M, N, dtype="bf16"):
    return {"name": name, "op": "checkpoint", "M": M, "N": N, "dtype": dtype}


def listed():
    return [
        # one token through the up projection of a 2048-wide model's MLP: generation, bound by latency
        _forward("forward_token", 1, 2048, 16384, 4, "gelu_tanh", False, False),
        # sixteen sequences' next tokens through its down projection, added to the residual stream
        _forward("forward_few", 16, 16384, 2048, 4, "none", True, False),
        # an fp32 layer of odd sizes: an MLP on images, a batch that fills no tile
        _forward("forward_odd_fp32", 333, 784, 1001, 8, "gelu", True, False, "f32"),
        # the up projection in training: 4096 tokens, input and pre-activation kept in 8 bits and read back
        _forward("forward_save", 4096, 2048, 16384, 4, "gelu_tanh", False, True),
        # the largest square layer: a long prompt, activation and residual
        _forward("forward_large", 16384, 4096, 4096, 4, "silu", True, False),
        # fine-tuning on very short batches
        _backward("backward_few", 16, 4096, 4096, 4, "silu", False),
        # odd sizes: columns that end inside a tile and inside a block of the checkpoint
        _backward("backward_odd", 1001, 784, 1000, 8, "gelu", True),
        # the small fp32 layer of the MNIST MLP's width
        _backward("backward_fp32", 64, 784, 128, 4, "gelu", True, "f32"),
        # the down projection in training, its gradient taken back through the activation below
        _backward("backward_down", 4096, 16384, 2048, 4, "gelu_tanh", False),
        # the largest square layer with a skip connection around it
        _backward("backward_large", 16384, 4096, 4096, 4, "silu", True),
        # an activation of a long batch kept for the backward pass
        _checkpoint("checkpoint_large", 16384, 4096),
        # a small one whose rows end inside a block, in fp32
        _checkpoint("checkpoint_odd_fp32", 37, 1030, "f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "checkpoint"])
    f32 = rng.random() < 0.2
    dtype = "f32" if f32 else "bf16"
    if op == "checkpoint":
        M, N = _spread(rng, 1, 16384), _spread(rng, 1, 16384)
        while M * N > 1 << 26:
            M, N = max(1, M // 2), N
        return {"op": op, "M": M, "N": N, "dtype": dtype}
    while True:
        M = _spread(rng, 1, 512 if f32 else 16384)
        K = 16 * _spread(rng, 1, 64 if f32 else 1024)
        N = _spread(rng, 8, 1024 if f32 else 16384)
        # odd widths: any for a forward pass; in training those of a classifier's head
        if rng.random() < 0.7 or (op == "backward" and N > 64):
            N = max(8, N // 8 * 8)
        if M * K <= 1 << 26 and M * N <= 1 << 26 and K * N <= 1 << 26 and M * K * N <= 1 << 38:
            break
    r = rng.choice([1, 2, 4, 4, 8, 8, 16])
    act = rng.choice(ACTS)
    if op == "forward":
        return {"op": op, "M": M, "K": K, "N": N, "r": r, "act": act, "residual": rng.random() < 0.5,
                "save": rng.random() < 0.4, "dtype": dtype}
    return {"op": op, "M": M, "K": K, "N": N, "r": r, "act": act, "add": rng.random() < 0.5,
            "dtype": dtype}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _row_codes(x):
    """Row codes of x [rows, cols] fp32: codes and one scale per row."""
    amax = x.abs().amax(dim=1)
    inv = torch.where(amax > 0, torch.div(torch.full_like(amax, 127.0), amax), torch.zeros_like(amax))
    return torch.round(x * inv[:, None]).clamp(-127, 127), torch.div(amax, torch.full_like(amax, 127.0))


def _block_codes(z):
    """8-bit checkpoint of z [M, N] fp32: codes [M, N] and scales [ceil(N/32), M]."""
    M, N = z.shape
    nb = (N + BLOCK - 1) // BLOCK
    zp = torch.nn.functional.pad(z, (0, nb * BLOCK - N)).view(M * nb, BLOCK)
    codes, s = _row_codes(zp)
    return codes.view(M, nb * BLOCK)[:, :N], s.view(M, nb).t().contiguous()


def _block_values(codes, s):
    N = codes.shape[1]
    return codes.float() * s.t().repeat_interleave(BLOCK, dim=1)[:, :N]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    dt = _dtype(case)
    M, N = case["M"], case["N"]
    state = {"case": case}
    if case["op"] == "checkpoint":
        state["T"] = normal(M, N).to(dt)
        return state
    K, r = case["K"], case["r"]
    w, sw = _row_codes(normal(N, K, std=0.02))
    state.update(Wq=w.to(torch.int8).contiguous(), sw=sw, bias=normal(N, std=0.01),
                 A=(torch.rand(K, r, generator=g, device="cuda") * 2 - 1) / math.sqrt(K),
                 B=normal(r, N, std=0.01), alpha=8.0)
    del w
    X = normal(M, K).to(dt)
    if case["op"] == "forward":
        state["X"] = X
        state["R"] = normal(M, N).to(dt) if case["residual"] else None
        return state
    xq, sx = _row_codes(X.float())
    zq, zs = _block_codes(normal(M, K, std=1.5))
    state.update(Xq=xq.to(torch.int8).contiguous(), sx=sx, xA=X.float() @ state["A"],
                 dY=normal(M, N, std=0.1).to(dt), zq=zq.to(torch.int8).contiguous(), zs=zs,
                 add=normal(M, K, std=0.1).to(dt) if case["add"] else None)
    return state


# ------------------------------------------------------------------ the pass
def run(state):
    if own:
        return _run_own(state)
    return {"forward": _plain_forward, "backward": _plain_backward,
            "checkpoint": _plain_checkpoint}[state["case"]["op"]](state)


def _run_own(state):
    from lora_fine_tuning_qlora_b200 import qlora

    case = state["case"]
    if case["op"] == "checkpoint":
        q, s = qlora.ckpt_save(state["T"])
        return {"t": qlora.ckpt_load(q, s, state["T"].dtype)}
    layer = state.get("layer")
    if layer is None:  # what a program keeps: the layer's handle and a workspace
        layer = state["layer"] = qlora.Layer(Wq=state["Wq"], sw=state["sw"], bias=state["bias"], A=state["A"],
                                             B=state["B"], alpha=state["alpha"], act=_dtype(case))
        if case["op"] == "backward":
            state["ws"] = qlora.ckpt_workspace(layer.desc(), case["M"], state["Xq"].device)
    if case["op"] == "forward":
        y, kept = qlora.forward_act(layer, state["X"], act=case["act"], residual=state["R"],
                                    save_z=case["save"])
        out = {"y": y, "xa": kept.xA}
        if case["save"]:
            out["x"] = qlora.ckpt_load(kept.Xq, kept.sx, torch.bfloat16)
            out["z"] = qlora.ckpt_load(kept.zq, kept.zs, torch.bfloat16)
        return out
    kept = qlora.Checkpoint(Xq=state["Xq"], sx=state["sx"], xA=state["xA"])
    dX, dA, dB, dbias = qlora.backward_ckpt(layer, kept, state["dY"], state["ws"], act=case["act"],
                                            z=(state["zq"], state["zs"]), add=state["add"])
    return {"dx": dX, "da": dA, "db": dB, "dbias": dbias}


def _act(act, z):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(act, z):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _plain_forward(state):
    case, dt = state["case"], _dtype(state["case"])
    x = state["X"].float()
    codes, sx = _row_codes(x)
    xa = x @ state["A"]
    z = (codes @ state["Wq"].float().t()) * sx[:, None] * state["sw"] + state["bias"]
    z = z + (state["alpha"] / case["r"]) * (xa @ state["B"])
    y = _act(case["act"], z)
    if state["R"] is not None:
        y = y + state["R"].float()
    out = {"y": y.to(dt), "xa": xa}
    if case["save"]:
        out["x"] = (codes * sx[:, None]).to(torch.bfloat16)
        out["z"] = _block_values(*_block_codes(z)).to(torch.bfloat16)
    return out


def _plain_backward(state):
    case, dt = state["case"], _dtype(state["case"])
    c = state["alpha"] / case["r"]
    dy = state["dY"].float()
    G = dy @ state["B"].t()
    dx = dy @ (state["Wq"].float() * state["sw"][:, None]) + c * (G @ state["A"].t())
    dx = dx * _act_slope(case["act"], _block_values(state["zq"], state["zs"]))
    if state["add"] is not None:
        dx = dx + state["add"].float()
    x = state["Xq"].float() * state["sx"][:, None]
    return {"dx": dx.to(dt), "da": c * (x.t() @ G), "db": c * (state["xA"].t() @ dy), "dbias": dy.sum(dim=0)}


def _plain_checkpoint(state):
    return {"t": _block_values(*_block_codes(state["T"].float())).to(state["T"].dtype)}


# ------------------------------------------------------------------ in 64 bits
def _to32(v):
    """Each value rounded to 32 bits, held in 64."""
    return v.to(torch.float32).to(torch.float64)


def _codes64(v, length):
    """Codes and scales of groups of `length` values along the rows, by the
    quantizer's definition: 32-bit operations, each rounded once, here made
    from 64-bit ones (which hold a product of two 32-bit values exactly and
    round a quotient of them as one rounding would)."""
    rows, cols = v.shape
    groups = -(-cols // length)
    wide = torch.zeros(rows, groups * length, dtype=torch.float64, device=v.device)
    wide[:, :cols] = v
    wide = wide.view(rows, groups, length)
    top = wide.abs().max(dim=2, keepdim=True).values
    inverse = torch.where(top > 0, _to32(127.0 / top), torch.zeros_like(top))
    codes = torch.round(_to32(wide * inverse)).clamp(-127.0, 127.0)
    scale = _to32(top / 127.0)
    return codes.view(rows, -1)[:, :cols], scale.expand(rows, groups, length).reshape(rows, -1)[:, :cols]


def _normal_cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _act64(act, z):
    return {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, torch.zeros_like(z)),
            "gelu": lambda: z * _normal_cdf(z),
            "gelu_tanh": lambda: z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)),
            "silu": lambda: z * torch.sigmoid(z)}[act]()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        q, scale = _codes64(s["T"].double(), BLOCK)
        return {"t": q * scale}
    c = s["alpha"] / case["r"]
    A, B, W = s["A"].double(), s["B"].double(), s["Wq"].double() * s["sw"].double()[:, None]
    if case["op"] == "forward":
        X = s["X"].double()
        q, scale = _codes64(X, case["K"])
        xa = torch.mm(X, A)
        values = q * scale
        z = torch.addmm(s["bias"].double(), values, W.t()) + torch.mm(xa, B) * c
        y = _act64(case["act"], z)
        if s["R"] is not None:
            y = y + s["R"].double()
        out = {"y": y, "xa": xa}
        if case["save"]:
            out["x"] = values
            zq, zscale = _codes64(_to32(z), BLOCK)
            out["z"] = zq * zscale
        return out
    dY = s["dY"].double()
    z = s["zq"].double() * s["zs"].double().t().repeat_interleave(BLOCK, 1)[:, :case["K"]]
    # the slope by the definition of the derivative, from the function itself
    z = z.requires_grad_(True)
    slope, = torch.autograd.grad(_act64(case["act"], z).sum(), z)
    G = torch.mm(dY, B.t())
    dx = (torch.mm(dY, W) + c * torch.mm(G, A.t())) * slope
    if s["add"] is not None:
        dx = dx + s["add"].double()
    X = s["Xq"].double() * s["sx"].double()[:, None]
    return {"dx": dx, "da": c * torch.mm(X.t(), G), "db": c * torch.mm(s["xA"].double().t(), dY),
            "dbias": torch.einsum("mn->n", dY)}


# ------------------------------------------------------------------ the floor
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    M, N = case["M"], case["N"]
    nb = -(-N // BLOCK)
    if case["op"] == "checkpoint":
        return {"bytes": 2.0 * M * N * e + M * N + 4.0 * M * nb, "flops": 5.0 * M * N}
    K, r = case["K"], case["r"]
    small = 4.0 * (2 * N + K * r + r * N)
    if case["op"] == "forward":
        b = M * K * e + K * N + M * N * e * (2 if case["residual"] else 1) + small + 4.0 * M * r
        if case["save"]:
            b += M * K + 4.0 * M + M * N + 4.0 * M * nb + 2.0 * M * (K + N)
        return {"bytes": b, "flops": 2.0 * M * N * K + 2.0 * M * r * (K + N)}
    b = M * N * e + K * N + M * K * e * (2 if case["add"] else 1) + M * K + 4.0 * M * -(-K // BLOCK)
    b += M * K + 4.0 * M + 4.0 * M * r + 2 * small
    return {"bytes": b, "flops": 2.0 * M * N * K + 2.0 * M * r * (2 * K + 2 * N)}
