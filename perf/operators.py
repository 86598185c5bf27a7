"""Cases, plain forms and 64-bit references of the gated block's gradients and adapters.

Four operators over the block Y = SiLU(A W1) * (A W2), Out = Y W3 + R:

  backward       dA, dW1, dW2 from A, W1, W2 and dY
  down_backward  dY, dW3 from dOut, W3 and Y
  lora           Y with one low-rank adapter per token, of a table shared by many requests
  down_lora      Out with one low-rank adapter per token

``own`` false: elementary torch operations in 32 bits, rounded once at the end.
``own`` true: the library's entry points.
"""
import math

import torch

own = False

# The largest listed case of each kind; a drawn case costs no more.
_MOST = {"backward": 12 * 4096 * 3584 * 18944, "down_backward": 4 * 4096 * 3584 * 18944,
         "lora": 4 * 4096 * 3584 * 18944, "down_lora": 2 * 4096 * 3584 * 18944}


def listed():
    """Sizes of the 0.5B and 7B gated blocks of this repository's workloads, and ragged ones."""
    return [
        # a short fine-tuning sequence on the smallest block: latency of a few launches counts
        {"name": "backward 0.5B m128", "op": "backward", "M": 128, "K": 896, "N": 4864},
        # a packed batch whose rows, hidden and intermediate sizes fill no tile
        {"name": "backward ragged m1000", "op": "backward", "M": 1000, "K": 1416, "N": 5000},
        # a training step's micro-batch on the 7B block
        {"name": "backward 7B m4096", "op": "backward", "M": 4096, "K": 3584, "N": 18944},
        # the same two training ends for the second half of the block
        {"name": "down_backward 0.5B m128", "op": "down_backward", "M": 128, "N": 4864, "H": 896},
        {"name": "down_backward 7B m4096", "op": "down_backward", "M": 4096, "N": 18944, "H": 3584},
        # one user's next token through one small adapter
        {"name": "lora 0.5B m1 r8", "op": "lora", "M": 1, "K": 896, "N": 4864, "rank": 8,
         "adapters": 4, "requests": 1},
        # a decode batch, a token a request, several adapters at once
        {"name": "lora 7B m16 r16", "op": "lora", "M": 16, "K": 3584, "N": 18944, "rank": 16,
         "adapters": 8, "requests": 16},
        # short prompts of a few requests, sizes that fill no tile
        {"name": "lora ragged m333 r24", "op": "lora", "M": 333, "K": 1416, "N": 5000, "rank": 24,
         "adapters": 5, "requests": 7},
        # a prefill batch of prompts of several requests
        {"name": "lora 7B m4096 r64", "op": "lora", "M": 4096, "K": 3584, "N": 18944, "rank": 64,
         "adapters": 8, "requests": 12},
        # the decode batch's second half, with the residual
        {"name": "down_lora 7B m16 r16", "op": "down_lora", "M": 16, "N": 18944, "H": 3584,
         "rank": 16, "adapters": 8, "requests": 16},
        # many small requests with an adapter each
        {"name": "down_lora 0.5B m128 r16", "op": "down_lora", "M": 128, "N": 4864, "H": 896,
         "rank": 16, "adapters": 32, "requests": 128},
        {"name": "down_lora 7B m4096 r64", "op": "down_lora", "M": 4096, "N": 18944, "H": 3584,
         "rank": 64, "adapters": 8, "requests": 12},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A hidden or intermediate size: an odd multiple of 128, or of 8 (the least the library takes)."""
    step = rng.choice((8, 128))
    return step * (_spread(rng, lo // step, hi // step - 1) | 1)


def draw(rng):
    op = rng.choice(("backward", "down_backward", "lora", "down_lora"))
    while True:
        m = _spread(rng, 1, 4095)
        m = m if m <= 32 else m | 1
        h, n = _size(rng, 256, 3584), _size(rng, 768, 18944)
        c = {"op": op, "M": m, "N": n, ("H" if op.startswith("down") else "K"): h}
        if op.endswith("lora"):
            c["rank"] = 8 * rng.randint(1, 8)
            c["adapters"] = _spread(rng, 1, 32)
            # a decode batch (a token a request) or prompts
            c["requests"] = m if m <= 128 and rng.random() < 0.5 else min(m, _spread(rng, 1, 16))
        if work(c)["flops"] <= _MOST[op]:
            return c


def _served(case):
    """(requests with an adapter, distinct adapters): every fourth request has none."""
    with_one = case["requests"] - case["requests"] // 4
    return with_one, min(case["adapters"], with_one)


def _tokens_with_adapter(case):
    return case["M"] * _served(case)[0] / case["requests"]


def work(case):
    m, n = case["M"], case["N"]
    h = case["H"] if "H" in case else case["K"]
    if case["op"] == "backward":
        return {"bytes": 2 * (2 * m * h + m * n + 4 * h * n), "flops": 12 * m * h * n}
    if case["op"] == "down_backward":
        return {"bytes": 2 * (m * h + 2 * m * n + 2 * h * n), "flops": 4 * m * h * n}
    r, used, tok = case["rank"], _served(case)[1], _tokens_with_adapter(case)
    if case["op"] == "lora":
        return {"bytes": 2 * (m * h + m * n + 2 * h * n + used * 2 * r * (h + n)) + 4 * m,
                "flops": 4 * m * h * n + 4 * tok * r * (h + n)}
    return {"bytes": 2 * (2 * m * h + m * n + h * n + used * r * (h + n)) + 4 * m,
            "flops": 2 * m * h * n + 2 * tok * r * (h + n)}


def _inputs(case, seed):
    """Activations ~ N(0, 1), weights ~ N(0, 1/fan-in), small incoming gradients; adapters whose
    product is a tenth or so of the projection, as after fine-tuning."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    m, n = case["M"], case["N"]
    s = {"op": case["op"]}
    if case["op"] == "backward":
        k = case["K"]
        s.update(A=normal(m, k), W1=normal(k, n, std=k ** -0.5), W2=normal(k, n, std=k ** -0.5),
                 dY=normal(m, n, std=0.02))
        return s
    if case["op"] == "down_backward":
        h = case["H"]
        s.update(dOut=normal(m, h, std=0.02), W3=normal(n, h, std=n ** -0.5), Y=normal(m, n))
        return s
    r, count, requests = case["rank"], case["adapters"], case["requests"]
    if case["op"] == "lora":
        k = case["K"]
        s.update(A=normal(m, k), W1=normal(k, n, std=k ** -0.5), W2=normal(k, n, std=k ** -0.5),
                 La=normal(count, 2, r, k, std=k ** -0.5), Lb=normal(count, 2, n, r, std=0.1 * r ** -0.5))
    else:
        h = case["H"]
        s.update(Y=normal(m, n), W3=normal(n, h, std=n ** -0.5), R=normal(m, h),
                 La=normal(count, r, n, std=n ** -0.5), Lb=normal(count, h, r, std=0.1 * r ** -0.5))
    s["scale"] = 0.5 + 1.5 * torch.rand(count, generator=g, device=dev)
    # requests are runs of tokens; every fourth has no adapter, the others take the adapters in turn
    order = torch.randperm(count, generator=g, device=dev)
    which = torch.arange(requests, device=dev)
    ranked = which - (which + 1) // 4
    adapter = torch.where(which % 4 == 3, torch.full_like(which, -1), order[ranked % count])
    cuts = torch.randperm(m - 1, generator=g, device=dev)[:requests - 1] + 1
    of_token = torch.zeros(m, dtype=torch.int64, device=dev)
    of_token[cuts] = 1
    s["index"] = adapter[of_token.cumsum(0)].to(torch.int32)
    return s


def prepare(case, seed):
    """The inputs; with the library, the packed weights and the workspace a program keeps too."""
    s = _inputs(case, seed)
    if not own:
        return s
    import swiglu_gated_mlp_gb300 as sg
    m, n = case["M"], case["N"]
    if case["op"] == "backward":
        s["Wp"] = sg.swiglu_pack_weights(s["W1"], s["W2"])
        s["ws"] = sg.swiglu_backward_workspace(m, case["K"], n)
    elif case["op"] == "down_backward":
        s["W3p"] = sg.swiglu_pack_down_weights(s["W3"])
        s["ws"] = sg.swiglu_down_backward_workspace(m, n, case["H"])
    elif case["op"] == "lora":
        s["Wp"] = sg.swiglu_pack_weights(s["W1"], s["W2"])
        s["ws"] = sg.swiglu_lora_workspace(m, case["K"], n, case["rank"])
    else:
        s["W3p"] = sg.swiglu_pack_down_weights(s["W3"])
        s["ws"] = sg.swiglu_down_lora_workspace(m, n, case["H"], case["rank"])
    return s


def run(s):
    return _library(s) if own else _plain(s)


def _library(s):
    import swiglu_gated_mlp_gb300 as sg
    if s["op"] == "backward":
        da, dw1, dw2 = sg.swiglu_backward(s["A"], s["Wp"], s["dY"], workspace=s["ws"])
        return {"dA": da, "dW1": dw1, "dW2": dw2}
    if s["op"] == "down_backward":
        dy, dw3 = sg.swiglu_down_backward(s["dOut"], s["W3p"], s["Y"], workspace=s["ws"])
        return {"dY": dy, "dW3": dw3}
    if s["op"] == "lora":
        return {"Y": sg.swiglu_forward_lora(s["A"], s["Wp"], s["W1"].shape[1], s["La"], s["Lb"],
                                            s["index"], s["scale"], workspace=s["ws"])}
    return {"Out": sg.swiglu_down_forward_lora(s["Y"], s["W3p"], s["W3"].shape[1], s["La"], s["Lb"],
                                               s["index"], s["scale"], R=s["R"], workspace=s["ws"])}


def _adapter_products(x, la, lb, index, scale):
    """scale[a] x[m] la[a]^T lb[a]^T with a = index[m] (none where it is negative); la [L, r, in], lb [L, out, r]."""
    count, r, _ = la.shape
    v = (x @ la.reshape(count * r, -1).t()).reshape(-1, count, r)
    mine = index[:, None] == torch.arange(count, device=x.device, dtype=index.dtype)
    v = v * (mine * scale)[:, :, None]
    return v.reshape(-1, count * r) @ lb.transpose(1, 2).reshape(count * r, -1)


def _plain(s):
    if s["op"] == "backward":
        a, w1, w2, dy = (s[k].float() for k in ("A", "W1", "W2", "dY"))
        g, u = a @ w1, a @ w2
        sig = 1 / (1 + torch.exp(-g))
        du = dy * g * sig
        dg = dy * u * sig * (1 + g * (1 - sig))
        return {"dA": (dg @ w1.t() + du @ w2.t()).bfloat16(), "dW1": (a.t() @ dg).bfloat16(),
                "dW2": (a.t() @ du).bfloat16()}
    if s["op"] == "down_backward":
        do, w3, y = (s[k].float() for k in ("dOut", "W3", "Y"))
        return {"dY": (do @ w3.t()).bfloat16(), "dW3": (y.t() @ do).bfloat16()}
    if s["op"] == "lora":
        a, la, lb = s["A"].float(), s["La"].float(), s["Lb"].float()
        g = a @ s["W1"].float() + _adapter_products(a, la[:, 0], lb[:, 0], s["index"], s["scale"])
        u = a @ s["W2"].float() + _adapter_products(a, la[:, 1], lb[:, 1], s["index"], s["scale"])
        return {"Y": (g / (1 + torch.exp(-g)) * u).bfloat16()}
    y = s["Y"].float()
    out = y @ s["W3"].float() + s["R"].float()
    out = out + _adapter_products(y, s["La"].float(), s["Lb"].float(), s["index"], s["scale"])
    return {"Out": out.bfloat16()}


def exact(case, seed):
    """The definition in 64 bits: gradients by differentiating the forward, adapters one at a time."""
    s = _inputs(case, seed)
    if case["op"] == "backward":
        leaves = [s[k].double().requires_grad_() for k in ("A", "W1", "W2")]
        gate = leaves[0].mm(leaves[1])
        y = gate.mul(torch.sigmoid(gate)).mul(leaves[0].mm(leaves[2]))
        grads = torch.autograd.grad(y, leaves, s["dY"].double())
        return dict(zip(("dA", "dW1", "dW2"), grads))
    if case["op"] == "down_backward":
        y, w3 = s["Y"].double().requires_grad_(), s["W3"].double().requires_grad_()
        return dict(zip(("dY", "dW3"), torch.autograd.grad(y.mm(w3), (y, w3), s["dOut"].double())))
    x = s["A" if case["op"] == "lora" else "Y"].double()
    weights = [s["W1"], s["W2"]] if case["op"] == "lora" else [s["W3"]]
    la, lb = s["La"], s["Lb"]
    if case["op"] != "lora":
        la, lb = la.unsqueeze(1), lb.unsqueeze(1)
    sums = []
    for h, w in enumerate(weights):
        acc = x.mm(w.double())
        for a in range(case["adapters"]):
            rows = (s["index"] == a).nonzero().reshape(-1)
            down = la[a, h].double().mul(s["scale"][a].double())
            acc[rows] += x[rows].mm(down.t()).mm(lb[a, h].double().t())
        sums.append(acc)
    if case["op"] == "lora":
        return {"Y": sums[0].mul(torch.sigmoid(sums[0])).mul(sums[1])}
    return {"Out": sums[0].add(s["R"].double())}
