"""8-bit calls on another stream than the current one, with work pending on both (needs a GB300)."""
import pytest
import torch

from swiglu_gated_mlp_gb300.workloads import make_inputs
from test_gpu_streams import same, tensors

pytestmark = pytest.mark.gpu

CALLS = ["quantize", "pack", "pack_down", "forward", "forward_pairs", "down", "down_pairs", "checkpoint", "output",
         "backward", "backward_codes"]


@pytest.fixture(scope="module")
def calls(native_lib):
    """Each call as (function of the stream, bytes of its workspace)."""
    n = native_lib
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    M, K, N = 200, 512, 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b1, b2 = (t.cuda() for t in make_inputs(M, K, N, 0))
    dy = make_inputs(M, N, 8, 1)[0].cuda()
    out = {"quantize": (lambda st: n.swiglu_quantize_int8(a, stream=st), 0)}
    q, sa = n.swiglu_quantize_int8(a)
    w, w3 = (torch.randint(-128, 128, s, generator=g, dtype=torch.int8, device="cuda") for s in ((K, N), (K, N)))
    s1 = torch.rand(N, generator=g, device="cuda") * 1e-3
    out["pack"] = (lambda st: n.swiglu_pack_weights_int8(w, w3, stream=st), 0)
    out["pack_down"] = (lambda st: n.swiglu_pack_down_weights_int8(w3, stream=st), 0)
    for k, name in ((K, ""), (K - 8, "_pairs")):
        x, v, v3 = (t.contiguous() for t in (q[:, :k], w[:k], w3[:k]))
        wp, w3p = n.swiglu_pack_weights_int8(v, v), n.swiglu_pack_down_weights_int8(v3)
        for plan in (n.swiglu_plan_string_int8(M, k, N), n.swiglu_down_plan_string_int8(M, k, N)):
            assert (" pairs " if name else " ctas ") in plan
        out["forward" + name] = (lambda st, x=x, wp=wp: n.swiglu_forward_int8(x, sa, wp, N, s1, s1, stream=st),
                                 n.swiglu_int8_workspace_bytes(M, k, N))
        out["down" + name] = (lambda st, x=x, w3p=w3p: n.swiglu_down_forward_int8(x, sa, w3p, N, s1, R=dy, stream=st),
                              n.swiglu_down_int8_workspace_bytes(M, k, N))
    bp = n.swiglu_pack_weights(b1, b2)
    kept = n.swiglu_forward_checkpoint(a, bp, N)[1:]
    ws = n.swiglu_backward_checkpoint_workspace_bytes(M, K, N)
    out["checkpoint"] = (lambda st: n.swiglu_forward_checkpoint(a, bp, N, stream=st), 0)
    out["output"] = (lambda st: n.swiglu_checkpoint_output(*kept, stream=st), 0)
    out["backward"] = (lambda st: n.swiglu_backward_checkpoint(a, bp, dy, *kept, stream=st), ws)
    out["backward_codes"] = (lambda st: n.swiglu_backward_checkpoint(q, bp, dy, *kept, scale_a=sa, stream=st), ws)
    torch.cuda.synchronize()
    assert sorted(out) == sorted(CALLS)
    return out


@pytest.mark.parametrize("how", ["stream", "handle", "current"])
@pytest.mark.parametrize("name", CALLS)
def test_freed_blocks_with_pending_work_are_not_handed_out(calls, name, how):
    # tensors of the sizes that the call allocates are freed while the current stream has still to
    # write them; the call on the side stream (given, or made current) runs at once and must not get them
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
        if how == "current":
            with torch.cuda.stream(side):
                got = call(None)
        else:
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
