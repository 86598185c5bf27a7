"""The 8-bit projections on CTA pairs, whose tokens a kernel before widens into the workspace (needs a GB300).

Every test asserts that its shapes take pairs, so that another plan cannot empty it. The bounds are
those of test_gpu_int8.py.
"""
import numpy as np
import pytest
import torch

from oracle import int8_ref as ref
from swiglu_gated_mlp_gb300.workloads import make_inputs
from test_gpu_int8 import assert_within, block, block_weights, codes, f64, native, scales  # noqa: F401

pytestmark = pytest.mark.gpu

# K (N of the down-projection) that is no multiple of 16, where all sizes take pairs, and others
BOTH = [(300, 136, 264), (131, 264, 392), (600, 528, 9000)]


def on_pairs(native, M, K, N, down=None):
    """Asserts that a projection (None: both) takes pairs, and a workspace with them."""
    for d in (False, True) if down is None else (down,):
        assert " pairs " in (native.swiglu_down_plan_string_int8 if d else native.swiglu_plan_string_int8)(M, K, N)
        assert (native.swiglu_down_int8_workspace_bytes if d else native.swiglu_int8_workspace_bytes)(M, K, N) == 2 * M * K


@pytest.mark.parametrize("M,K,N", BOTH)
def test_scales_that_are_not_finite_stay_alone(native, M, K, N):
    on_pairs(native, M, K, N)
    g = torch.Generator().manual_seed(1)
    a, w1, w2 = (t.cuda() for t in (codes(g, M, K), codes(g, K, N), codes(g, K, N)))
    sa, s1, s2 = (t.cuda() for t in (scales(g, M, 0.02), scales(g, N, 0.01), scales(g, N, 0.01)))
    wp, w3p = native.swiglu_pack_weights_int8(w1, w2), native.swiglu_pack_down_weights_int8(w1)
    want = native.swiglu_forward_int8(a, sa, wp, N, s1, s2)
    want3 = native.swiglu_down_forward_int8(a, sa, w3p, N, s1)
    assert torch.isfinite(want).all() and torch.isfinite(want3).all()
    sa[3], sa[M - 1], s1[200] = float("nan"), float("inf"), float("inf")
    got, got3 = native.swiglu_forward_int8(a, sa, wp, N, s1, s2), native.swiglu_down_forward_int8(a, sa, w3p, N, s1)
    rows, cols = (torch.arange(M) != 3) & (torch.arange(M) != M - 1), torch.arange(N) != 200
    for x, y in ((got, want), (got3, want3)):
        assert torch.equal(x[rows][:, cols], y[rows][:, cols])
        assert torch.isnan(x[3]).all()
    assert not torch.isfinite(got3[:, 200]).any() and not torch.isfinite(got3[M - 1]).any()


@pytest.mark.parametrize("M,K,N", BOTH)
def test_outputs_and_workspaces_end_where_they_should(native, M, K, N):
    on_pairs(native, M, K, N)
    g = torch.Generator().manual_seed(2)
    a, w1, w2 = (t.cuda() for t in (codes(g, M, K), codes(g, K, N), codes(g, K, N)))
    sa, s1 = scales(g, M, 0.02).cuda(), scales(g, N, 0.01).cuda()
    wp, w3p = native.swiglu_pack_weights_int8(w1, w2), native.swiglu_pack_down_weights_int8(w1)
    r = make_inputs(M, N, 8, 3)[0].cuda()
    pad, need = 64, 2 * M * K
    forward = lambda **kw: native.swiglu_forward_int8(a, sa, wp, N, s1, s1, **kw)  # noqa: E731
    down = lambda **kw: native.swiglu_down_forward_int8(a, sa, w3p, N, s1, R=r, **kw)  # noqa: E731
    for call, out in ((forward, "Y"), (down, "Out")):
        want = call()
        for value in (0, 0xFF):  # what the workspace holds before means nothing
            buf = torch.full((M * N + 2 * pad,), 3.0, dtype=torch.bfloat16, device="cuda")
            ws = torch.full((need + 2 * pad,), value, dtype=torch.uint8, device="cuda")
            ws[:pad], ws[-pad:] = 55, 55
            call(**{out: buf[pad:-pad].view(M, N), "workspace": ws[pad:-pad]})
            assert torch.equal(buf[pad:-pad].view(M, N), want)
            assert (buf[:pad] == 3).all() and (buf[-pad:] == 3).all() and (ws[:pad] == 55).all() and (ws[-pad:] == 55).all()
            assert (ws[pad:-pad] != value).any()
    x = r.clone()  # in place
    assert torch.equal(native.swiglu_down_forward_int8(a, sa, w3p, N, s1, R=x, Out=x), down())
    for call, name in ((forward, "workspace"), (down, "workspace")):  # one byte short, and none
        for size in (need - 1, 0):
            with pytest.raises(native.SwigluError):
                call(**{name: torch.empty(size, dtype=torch.uint8, device="cuda")})
    native.swiglu_check_device_status()


@pytest.mark.parametrize("M", [1, 5, 200])
def test_streams_and_graphs(native, M):
    K, N = 264, 648
    on_pairs(native, M, K, N, False)
    on_pairs(native, M, N, K, True)
    (w1, s1), (w2, s2), (w3, s3) = block_weights(native, K, N)
    wp, w3p = native.swiglu_pack_weights_int8(w1, w2), native.swiglu_pack_down_weights_int8(w3)
    xs = [make_inputs(M, K, 8, 10 + i)[0].cuda() for i in range(2)]
    alone = [block(native, x, wp, w3p, s1, s2, s3, N, K) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    spaces = [(native.swiglu_int8_workspace(M, K, N), native.swiglu_down_int8_workspace(M, N, K)) for _ in xs]
    torch.cuda.synchronize()
    got = []
    for st, x, ws in zip(streams, xs, spaces):
        with torch.cuda.stream(st):
            for _ in range(10):
                last = block(native, x, wp, w3p, s1, s2, s3, N, K, ws)
            got.append(last)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, got))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(native, x, wp, w3p, s1, s2, s3, N, K)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, alone[i])
    st = streams[0]
    st.wait_stream(torch.cuda.current_stream())
    q, sa = native.swiglu_quantize_int8(xs[1], stream=st)
    y = native.swiglu_forward_int8(q, sa, wp, N, s1, s2, stream=st)
    st.synchronize()
    q2, sa2 = native.swiglu_quantize_int8(xs[1])
    assert torch.equal(q, q2) and torch.equal(y, native.swiglu_forward_int8(q2, sa2, wp, N, s1, s2))


@pytest.mark.parametrize("M", [1, 100, 300])
def test_the_block_as_it_is_served(native, M):
    K, N = 264, 648
    on_pairs(native, M, K, N, False)
    on_pairs(native, M, N, K, True)
    (w1, s1), (w2, s2), (w3, s3) = block_weights(native, K, N)
    x = make_inputs(M, K, 8, 8)[0]
    wp, w3p = native.swiglu_pack_weights_int8(w1, w2), native.swiglu_pack_down_weights_int8(w3)
    out = block(native, x.cuda(), wp, w3p, s1, s2, s3, N, K)
    native.swiglu_check_device_status()
    q, sa = ref.quantise(f64(x))
    y, ey = ref.gated(*ref.product(q, sa, f64(w1), f64(s1)), *ref.product(q, sa, f64(w2), f64(s2)))
    qy, sy = ref.quantise(y)
    # as in test_gpu_int8.py: a value of Y off by ey lands on a code off by at most ey / s + 1
    want, e = ref.product(qy, sy, f64(w3), f64(s3))
    moved = (ey + sy[:, None] * 1.0 + abs(qy) * ey.max(1, keepdims=True) / 127) @ (abs(f64(w3)) * f64(s3))
    assert_within(out, *ref.added(want, e + moved, f64(x)))


@pytest.mark.parametrize("M", [1, 40, 65, 300, 1300])
@pytest.mark.parametrize("N,H", [(8, 8), (1016, 264)])
def test_integer_sums_are_exact(native, M, N, H):
    # |sum| <= 1016 * 2^14 < 2^24: the fp32 sum is the integer, and the output its bf16 rounding
    on_pairs(native, M, N, H, True)
    g = torch.Generator().manual_seed(M + N)
    y, w3 = codes(g, M, N), codes(g, N, H)
    y[0], w3[:, 0] = -128, -128
    one = torch.ones(max(M, H))
    out = native.swiglu_down_forward_int8(y.cuda(), one[:M].cuda(), native.swiglu_pack_down_weights_int8(w3.cuda()),
                                          H, one[:H].cuda())
    assert torch.equal(out.cpu(), (y.to(torch.int64) @ w3.to(torch.int64)).double().bfloat16())


@pytest.mark.parametrize("M", [1, 300])
def test_large_sums(native, M):
    # every product 2^14 and one sign: sums of 18952 * 2^14 = 2^28.2
    N, H = 18952, 136
    on_pairs(native, M, N, H, True)
    y = torch.full((M, N), -128, dtype=torch.int8)
    w3 = torch.full((N, H), -128, dtype=torch.int8)
    w3[:, 1::2] = 127
    sy, s3 = torch.full((M,), 2.0 ** -8), torch.full((H,), 2.0 ** -9)
    out = native.swiglu_down_forward_int8(y.cuda(), sy.cuda(), native.swiglu_pack_down_weights_int8(w3.cuda()), H, s3.cuda())
    assert_within(out, *ref.added(*ref.product(f64(y), f64(sy), f64(w3), f64(s3)), 0.0))


@pytest.mark.parametrize("M,K,N", BOTH)
def test_part_of_a_batch(native, M, K, N):
    # tokens from the third on, as views (rows of codes that start on 16 bytes)
    on_pairs(native, M, K, N)
    on_pairs(native, M - 2, K, N)
    g = torch.Generator().manual_seed(3)
    a, w, r = codes(g, M, K).cuda(), codes(g, K, N).cuda(), make_inputs(M, N, 8, 3)[0].cuda()
    sa, s = scales(g, M, 0.02).cuda(), scales(g, N, 0.01).cuda()
    wp, w3p = native.swiglu_pack_weights_int8(w, w), native.swiglu_pack_down_weights_int8(w)
    assert torch.equal(native.swiglu_forward_int8(a[2:], sa[2:], wp, N, s, s), native.swiglu_forward_int8(a, sa, wp, N, s, s)[2:])
    assert torch.equal(native.swiglu_down_forward_int8(a[2:], sa[2:], w3p, N, s, R=r[2:]),
                       native.swiglu_down_forward_int8(a, sa, w3p, N, s, R=r)[2:])
    if K % 16:  # rows that do not: refused
        with pytest.raises(native.SwigluError):
            native.swiglu_forward_int8(a[1:], sa[1:], wp, N, s, s)


@pytest.mark.parametrize("M,K,N", [(300, 520, 264), (600, 528, 9000)])
def test_a_stalled_pipeline_is_reported(native, M, K, N):
    on_pairs(native, M, K, N)
    g = torch.Generator().manual_seed(1)
    a, w = codes(g, M, K).cuda(), codes(g, K, N).cuda()
    sa, s = scales(g, M, 0.02).cuda(), scales(g, N, 0.01).cuda()
    wp, w3p = native.swiglu_pack_weights_int8(w, w), native.swiglu_pack_down_weights_int8(w)
    want, want3 = native.swiglu_forward_int8(a, sa, wp, N, s, s), native.swiglu_down_forward_int8(a, sa, w3p, N, s)
    native.swiglu_check_device_status()
    for call in (lambda: native.swiglu_forward_int8(a, sa, wp, N, s, s),
                 lambda: native.swiglu_down_forward_int8(a, sa, w3p, N, s)):
        native.swiglu_testing_inject_stall(True, 20)
        try:
            call()
            with pytest.raises(native.SwigluError) as e:
                native.swiglu_check_device_status()
            assert e.value.code == native.SWIGLU_ERR_TIMEOUT
        finally:
            native.swiglu_testing_inject_stall(False, 1000)
        native.swiglu_check_device_status()
    assert torch.equal(native.swiglu_forward_int8(a, sa, wp, N, s, s), want)
    assert torch.equal(native.swiglu_down_forward_int8(a, sa, w3p, N, s), want3)
    native.swiglu_check_device_status()


@pytest.mark.parametrize("M,K,N,op", [(16, 8192, 29568, "int8"), (16, 29568, 8192, "down"), (1000, 8192, 29568, "int8"),
                                      (1000, 29568, 8192, "down"), (1, 5120, 27648, "int8"), (1, 27648, 5120, "down"),
                                      (300, 5120, 27648, "int8"), (300, 27648, 5120, "down")])
def test_the_largest_blocks(native, M, K, N, op):
    # sizes of the 32B and 72B blocks: sampled columns against every token (few tokens on single CTAs)
    if M >= 300:
        on_pairs(native, M, K, N, op == "down")
    g = torch.Generator(device="cuda").manual_seed(5)
    w1, w2 = (torch.randint(-128, 128, (K, N), generator=g, dtype=torch.int8, device="cuda") for _ in range(2))
    h = torch.Generator().manual_seed(6)
    a, sa, s1, s2 = codes(h, M, K), scales(h, M, 0.02), scales(h, N, 2e-3 / K ** 0.5), scales(h, N, 2e-3)
    cols = torch.from_numpy(np.unique(np.concatenate([[0, N - 1, 127, 128], np.random.default_rng(0).integers(0, N, 24)])))
    at = cols.cuda()
    if op == "int8":
        y = native.swiglu_forward_int8(a.cuda(), sa.cuda(), native.swiglu_pack_weights_int8(w1, w2), N, s1.cuda(), s2.cuda())
    else:
        y = native.swiglu_down_forward_int8(a.cuda(), sa.cuda(), native.swiglu_pack_down_weights_int8(w1), N, s1.cuda())
    native.swiglu_check_device_status()
    gate = ref.product(f64(a), f64(sa), f64(w1[:, at]), f64(s1[cols]))
    up = ref.product(f64(a), f64(sa), f64(w2[:, at]), f64(s2[cols]))
    assert_within(y[:, at], *(ref.gated(*gate, *up) if op == "int8" else ref.added(*gate, 0.0)))


def test_two_threads_at_once(native):
    # the calls let go of the interpreter: two threads, each on its own stream, on shared weights
    import threading

    K, N = 264, 648
    (w1, s1), (w2, s2), (w3, s3) = block_weights(native, K, N)
    wp, w3p = native.swiglu_pack_weights_int8(w1, w2), native.swiglu_pack_down_weights_int8(w3)
    xs = [make_inputs(M, K, 8, 20 + M)[0].cuda() for M in (3, 200)]
    alone = [block(native, x, wp, w3p, s1, s2, s3, N, K) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got, ready = [None, None], threading.Barrier(2)

    def work(i):
        with torch.cuda.stream(streams[i]):
            ready.wait(30)
            for _ in range(200):
                out = block(native, xs[i], wp, w3p, s1, s2, s3, N, K)
            streams[i].synchronize()
            got[i] = out

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    native.swiglu_check_device_status()
    assert all(torch.equal(a, b) for a, b in zip(alone, got))
