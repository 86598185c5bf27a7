"""Cases, plain forms and 64-bit references of the gated block in 8-bit integers.

Four operators over the block Y = SiLU(A W1) * (A W2), Out = Y W3 + R:

  int8                 Y from bf16 A, quantised per token, and weights in 8-bit integers with a
                       scale per channel
  down_int8            Out, likewise from bf16 Y and W3
  checkpoint           the training forward: Y, with Gate and Up kept in 8 bits (a scale per token
                       and 128 columns), and Y as the backward pass restores it from them
  backward_checkpoint  dA, dW1, dW2 from the checkpoint and dY, the input too in 8 bits

A group of values x is held as codes and a scale s: with m = max(max |x|, 2^-100), s = m / 127 and
the codes are 127 x / m, rounded to the nearest (halves to even).

``own`` false: elementary torch operations in 32 bits, rounded once at the end.
``own`` true: the library's entry points.
"""
import math

import torch

own = False

_BLOCK = 128      # columns of Gate or Up that share a scale
_LEAST = 2.0 ** -100

# The largest listed case of each kind; a drawn case costs no more.
_MOST = {"int8": 4 * 4096 * 3584 * 18944, "down_int8": 2 * 4096 * 3584 * 18944,
         "checkpoint": 4 * 4096 * 3584 * 18944, "backward_checkpoint": 8 * 4096 * 3584 * 18944}


def listed():
    """Sizes of the 0.5B and 7B gated blocks of this repository's workloads, and ragged ones."""
    return [
        # one user's next token on the smallest block: latency counts
        {"name": "int8 0.5B m1", "op": "int8", "M": 1, "K": 896, "N": 4864},
        # a decode batch: the 8-bit weights are streamed once
        {"name": "int8 7B m16", "op": "int8", "M": 16, "K": 3584, "N": 18944},
        # short prompts of a few requests, sizes that fill no tile
        {"name": "int8 ragged m333", "op": "int8", "M": 333, "K": 1424, "N": 5000},
        # a prefill batch
        {"name": "int8 7B m4096", "op": "int8", "M": 4096, "K": 3584, "N": 18944},
        # the decode batch's second half, with the residual
        {"name": "down_int8 7B m16", "op": "down_int8", "M": 16, "N": 18944, "H": 3584},
        # many small requests on the smallest block
        {"name": "down_int8 0.5B m128", "op": "down_int8", "M": 128, "N": 4864, "H": 896},
        # the prefill batch's second half
        {"name": "down_int8 7B m4096", "op": "down_int8", "M": 4096, "N": 18944, "H": 3584},
        # a short fine-tuning sequence on the smallest block
        {"name": "checkpoint 0.5B m128", "op": "checkpoint", "M": 128, "K": 896, "N": 4864},
        # a training step's micro-batch on the 7B block
        {"name": "checkpoint 7B m4096", "op": "checkpoint", "M": 4096, "K": 3584, "N": 18944},
        # the backward pass of the same two, and of a packed batch that fills no tile
        {"name": "backward_checkpoint 0.5B m128", "op": "backward_checkpoint", "M": 128, "K": 896,
         "N": 4864},
        {"name": "backward_checkpoint ragged m1000", "op": "backward_checkpoint", "M": 1000, "K": 1416,
         "N": 5000},
        {"name": "backward_checkpoint 7B m4096", "op": "backward_checkpoint", "M": 4096, "K": 3584,
         "N": 18944},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, least):
    """A hidden or intermediate size: an odd multiple of 128, or of the least the library takes."""
    step = rng.choice((least, 128))
    return step * (_spread(rng, lo // step, hi // step - 1) | 1)


def draw(rng):
    op = rng.choice(("int8", "down_int8", "checkpoint", "backward_checkpoint"))
    while True:
        m = _spread(rng, 1, 4095)
        m = m if m <= 32 else m | 1
        # rows of 8-bit operands that are summed over are whole 16-byte units
        h = _size(rng, 256, 3584, 16 if op == "int8" else 8)
        n = _size(rng, 768, 18944, 16 if op == "down_int8" else 8)
        c = {"op": op, "M": m, "N": n, ("H" if op == "down_int8" else "K"): h}
        if work(c)["flops"] <= _MOST[op]:
            return c


def work(case):
    m, n = case["M"], case["N"]
    h = case["H"] if "H" in case else case["K"]
    if case["op"] == "int8":  # A and Y in bf16, both weights in 8 bits with a scale a column
        return {"bytes": 2 * m * h + 2 * m * n + 2 * h * n + 8 * n, "flops": 4 * m * h * n}
    if case["op"] == "down_int8":  # Y, R and Out in bf16, the weight in 8 bits
        return {"bytes": 2 * m * n + 4 * m * h + h * n + 4 * h, "flops": 2 * m * h * n}
    kept = 2 * m * n + 8 * m * -(-n // _BLOCK)  # codes and scales of Gate and Up
    if case["op"] == "checkpoint":  # A, both weights; Y, the checkpoint, Y again
        return {"bytes": 2 * m * h + 4 * h * n + 4 * m * n + kept, "flops": 4 * m * h * n}
    # A in 8 bits with a scale a token, dY, the checkpoint, both weights; dA, dW1, dW2
    return {"bytes": m * h + 4 * m + 2 * m * n + kept + 2 * m * h + 8 * h * n, "flops": 8 * m * h * n}


def _quantised(x, dim):
    """Codes (int8) and scales of fp32 x, one scale for each line along `dim`. 64 bits, as whole
    rows of bf16 values lie halfway between two codes where the largest is a multiple of 127."""
    m = x.abs().amax(dim, keepdim=True).clamp(min=_LEAST)
    return torch.round(x.double() * 127 / m.double()).to(torch.int8), (m / 127.0).squeeze(dim)


def _blocks(x):
    """[M, N] as [M, blocks, 128], zeros past the last column."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % _BLOCK)).reshape(x.shape[0], -1, _BLOCK)


def _kept(x):
    """Gate or Up, fp32 [M, N], in 8 bits: codes [M, N], scales [blocks, M]."""
    q, s = _quantised(_blocks(x), 2)
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]].contiguous(), s.t().contiguous()


def _values(q, s):
    """The fp32 values of codes [M, N] and scales [blocks, M]."""
    return (_blocks(q.float()) * s.t()[:, :, None]).reshape(q.shape[0], -1)[:, :q.shape[1]]


def _inputs(case, seed):
    """Activations ~ N(0, 1) times a magnitude of each token's own, weights ~ N(0, 1/fan-in), small
    incoming gradients; 8-bit weights from float ones, the checkpoint from the block's own products."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    def tokens(rows, cols):
        return (normal(rows, cols) * torch.exp(0.5 * normal(rows, 1))).bfloat16()

    m, n = case["M"], case["N"]
    s = {"op": case["op"]}
    if case["op"] == "down_int8":
        h = case["H"]
        s["Y"], s["R"] = tokens(m, n), normal(m, h).bfloat16()
        s["W3"], s["s3"] = _quantised(normal(n, h, std=n ** -0.5), 0)
        return s
    k = case["K"]
    s["A"] = tokens(m, k)
    if case["op"] == "int8":
        s["W1"], s["s1"] = _quantised(normal(k, n, std=k ** -0.5), 0)
        s["W2"], s["s2"] = _quantised(normal(k, n, std=k ** -0.5), 0)
        return s
    s["W1"], s["W2"] = normal(k, n, std=k ** -0.5).bfloat16(), normal(k, n, std=k ** -0.5).bfloat16()
    if case["op"] == "backward_checkpoint":
        s["gate"], gate_scale = _kept((s["A"] @ s["W1"]).float())
        s["up"], up_scale = _kept((s["A"] @ s["W2"]).float())
        s["scale"] = torch.stack((gate_scale, up_scale))
        s["A"], s["sa"] = _quantised(s["A"].float(), 1)
        s["dY"] = normal(m, n, std=0.02).bfloat16()
    return s


def prepare(case, seed):
    """The inputs; with the library, the packed weights and the workspace a program keeps too."""
    s = _inputs(case, seed)
    if not own:
        return s
    import swiglu_gated_mlp_gb300 as sg
    m, n = case["M"], case["N"]
    if case["op"] == "int8":
        s["Wp"] = sg.swiglu_pack_weights_int8(s["W1"], s["W2"])
        s["ws"] = sg.swiglu_int8_workspace(m, case["K"], n)
    elif case["op"] == "down_int8":
        s["W3p"] = sg.swiglu_pack_down_weights_int8(s["W3"])
        s["ws"] = sg.swiglu_down_int8_workspace(m, n, case["H"])
    else:
        s["Wp"] = sg.swiglu_pack_weights(s["W1"], s["W2"])
        if case["op"] == "backward_checkpoint":
            s["ws"] = sg.swiglu_backward_checkpoint_workspace(m, case["K"], n)
    return s


def run(s):
    return _library(s) if own else _plain(s)


def _library(s):
    import swiglu_gated_mlp_gb300 as sg
    if s["op"] == "int8":
        a, sa = sg.swiglu_quantize_int8(s["A"])
        return {"Y": sg.swiglu_forward_int8(a, sa, s["Wp"], s["W1"].shape[1], s["s1"], s["s2"],
                                            workspace=s["ws"])}
    if s["op"] == "down_int8":
        y, sy = sg.swiglu_quantize_int8(s["Y"])
        return {"Out": sg.swiglu_down_forward_int8(y, sy, s["W3p"], s["W3"].shape[1], s["s3"], R=s["R"],
                                                   workspace=s["ws"])}
    if s["op"] == "checkpoint":
        y, gate, up, scale = sg.swiglu_forward_checkpoint(s["A"], s["Wp"], s["W1"].shape[1])
        return {"Y": y, "restored": sg.swiglu_checkpoint_output(gate, up, scale)}
    da, dw1, dw2 = sg.swiglu_backward_checkpoint(s["A"], s["Wp"], s["dY"], s["gate"], s["up"], s["scale"],
                                                 scale_a=s["sa"], workspace=s["ws"])
    return {"dA": da, "dW1": dw1, "dW2": dw2}


def _gated(g, u):
    return g / (1 + torch.exp(-g)) * u


def _plain(s):
    if s["op"] == "int8":
        a, sa = _quantised(s["A"].float(), 1)
        a = a.float()
        g = (a @ s["W1"].float()) * sa[:, None] * s["s1"]
        u = (a @ s["W2"].float()) * sa[:, None] * s["s2"]
        return {"Y": _gated(g, u).bfloat16()}
    if s["op"] == "down_int8":
        y, sy = _quantised(s["Y"].float(), 1)
        out = (y.float() @ s["W3"].float()) * sy[:, None] * s["s3"]
        return {"Out": (out + s["R"].float()).bfloat16()}
    if s["op"] == "checkpoint":
        a = s["A"].float()
        g, u = a @ s["W1"].float(), a @ s["W2"].float()
        return {"Y": _gated(g, u).bfloat16(),
                "restored": _gated(_values(*_kept(g)), _values(*_kept(u))).bfloat16()}
    w1, w2, dy = (s[k].float() for k in ("W1", "W2", "dY"))
    a = s["A"].float() * s["sa"][:, None]
    g, u = _values(s["gate"], s["scale"][0]), _values(s["up"], s["scale"][1])
    sig = 1 / (1 + torch.exp(-g))
    du = dy * g * sig
    dg = dy * u * sig * (1 + g * (1 - sig))
    return {"dA": (dg @ w1.t() + du @ w2.t()).bfloat16(), "dW1": (a.t() @ dg).bfloat16(),
            "dW2": (a.t() @ du).bfloat16()}


def _rounded(x, width):
    """fp64 x [M, N] as groups of `width` columns hold it: whole multiples of the largest / 127."""
    cut = [c.mul(127).div(top).round().mul(top.div(127)) for c in x.split(width, 1)
           for top in [c.abs().max(1, keepdim=True).values.clamp(min=_LEAST)]]
    return torch.cat(cut, 1)


def exact(case, seed):
    """The definition in 64 bits: values on the grid that their group's largest sets, products of those,
    and gradients by differentiating SiLU(gate) * up at the values the checkpoint stands for."""
    s = _inputs(case, seed)
    if case["op"] == "int8":
        a = _rounded(s["A"].double(), case["K"])
        gate, up = (a.mm(s[w].double().mul(s[c].double())) for w, c in (("W1", "s1"), ("W2", "s2")))
        return {"Y": gate.mul(torch.sigmoid(gate)).mul(up)}
    if case["op"] == "down_int8":
        y = _rounded(s["Y"].double(), case["N"])
        return {"Out": torch.addmm(s["R"].double(), y, s["W3"].double().mul(s["s3"].double()))}
    if case["op"] == "checkpoint":
        gate, up = s["A"].double().mm(s["W1"].double()), s["A"].double().mm(s["W2"].double())
        held = [_rounded(x, _BLOCK) for x in (gate, up)]
        return {"Y": gate.mul(torch.sigmoid(gate)).mul(up),
                "restored": held[0].mul(torch.sigmoid(held[0])).mul(held[1])}
    wide = s["scale"].double().repeat_interleave(_BLOCK, 1)[:, :case["N"]].transpose(1, 2)
    gate = s["gate"].double().mul(wide[0]).requires_grad_()
    up = s["up"].double().mul(wide[1]).requires_grad_()
    y = gate.mul(torch.sigmoid(gate)).mul(up)
    dg, du = torch.autograd.grad(y, (gate, up), s["dY"].double())
    at = s["A"].double().mul(s["sa"].double().unsqueeze(1)).t()
    return {"dA": torch.addmm(dg.mm(s["W1"].double().t()), du, s["W2"].double().t()),
            "dW1": at.mm(dg), "dW2": at.mm(du)}
