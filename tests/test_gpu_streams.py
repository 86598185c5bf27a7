"""Calls on another stream than the current one, with work pending on both (needs a GB300)."""
import pytest
import torch

from swiglu_gated_mlp_gb300.workloads import make_inputs, make_inputs_fp8

pytestmark = pytest.mark.gpu

M, K, N, L, R = 200, 512, 1024, 3, 16
CALLS = ["forward", "fp8", "down", "pack", "pack_down", "pack_fp8", "backward", "down_backward", "lora", "down_lora"]


@pytest.fixture(scope="module")
def calls(native_lib):
    """Each call as (function of the stream, bytes of its workspace)."""
    n = native_lib
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 0))
    a8, q1, q2, s = make_inputs_fp8(M, K, N, 0)
    a8, q1, q2 = a8.cuda(), q1.cuda(), q2.cuda()
    wp, wp8, w3p = n.swiglu_pack_weights(w1, w2), n.swiglu_pack_weights_fp8(q1, q2), n.swiglu_pack_down_weights(w1)
    dy = make_inputs(M, N, 8, 1)[0].cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    la, lb = (torch.randn(*x, generator=g, device="cuda").bfloat16() / 8 for x in ((L, 2, R, K), (L, 2, N, R)))
    index = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    scale = torch.ones(L, device="cuda")
    la3, lb3 = la[:, 0].contiguous(), lb[:, 0].contiguous()
    out = {
        "forward": (lambda st: n.swiglu_forward(a, wp, N, stream=st), 0),
        "fp8": (lambda st: n.swiglu_forward_fp8(a8, wp8, N, *s, stream=st), 0),
        "down": (lambda st: n.swiglu_down_forward(a, w3p, N, stream=st), 0),
        "pack": (lambda st: n.swiglu_pack_weights(w1, w2, stream=st), 0),
        "pack_down": (lambda st: n.swiglu_pack_down_weights(w1, stream=st), 0),
        "pack_fp8": (lambda st: n.swiglu_pack_weights_fp8(q1, q2, stream=st), 0),
        "backward": (lambda st: n.swiglu_backward(a, wp, dy, stream=st), n.swiglu_backward_workspace_bytes(M, K, N)),
        "down_backward": (lambda st: n.swiglu_down_backward(dy, w3p, a, stream=st),
                          n.swiglu_down_backward_workspace_bytes(M, K, N)),
        "lora": (lambda st: n.swiglu_forward_lora(a, wp, N, la, lb, index, scale, stream=st),
                 n.swiglu_lora_workspace_bytes(M, K, N, R)),
        "down_lora": (lambda st: n.swiglu_down_forward_lora(a, w3p, N, la3, lb3, index, scale, stream=st),
                      n.swiglu_down_lora_workspace_bytes(M, K, N, R)),
    }
    torch.cuda.synchronize()
    return out


def tensors(x):
    return list(x) if isinstance(x, tuple) else [x]


def same(x, y):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(tensors(x), tensors(y)))


@pytest.mark.parametrize("how", ["stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_freed_blocks_with_pending_work_are_not_handed_out(calls, name, how):
    # tensors of the sizes that the call allocates are freed while the current stream has
    # still to write them; the call on the side stream runs at once and must not get them
    call, ws_bytes = calls[name]
    side = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    sizes = [t.nbytes for t in tensors(want)] + ([ws_bytes] if ws_bytes else [])
    for _ in range(3):
        freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t in freed:
            t.fill_(0xFF)
        del freed, t
        got = call(side if how == "stream" else side.cuda_stream)
        torch.cuda.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_freed_while_the_current_stream_reads_them(calls, name):
    # an output of a call on a side stream, read on the current stream and freed at once:
    # the next call on the side stream must not write its block before that read
    call, _ = calls[name]
    side = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    out = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    read = [t.clone() for t in tensors(out)]
    sizes = [t.nbytes for t in tensors(out)]
    del out
    with torch.cuda.stream(side):
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    assert same(tuple(read), want)
