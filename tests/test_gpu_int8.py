"""Projections in 8-bit integers against exact integer sums and float64 (needs a GB300).

Bounds are worst-case sums of the roundings the kernels make (oracle/int8_ref.py); where every
partial sum stays below 2^24 the fp32 sum has one right value, and so has the output.
"""
import numpy as np
import pytest
import torch

from oracle import int8_ref as ref
from oracle.swiglu_ref import bf16_bits_to_f64
from swiglu_gated_mlp_gb300.workloads import bf16_bits, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def native(native_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return native_lib


def f64(t):
    return bf16_bits_to_f64(bf16_bits(t.cpu())) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


def assert_within(out, want, bound):
    d = np.abs(f64(out) - want)
    worst = np.unravel_index(np.argmax(d / bound), d.shape)
    assert (d <= bound).all(), (worst, d[worst], bound[worst], want[worst])


def codes(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)


def scales(g, n, size):
    return (0.5 + torch.rand(n, generator=g)) * size


# one token, a partial and a full decode tile, the first sizes widened before, one and several token
# groups that fill no tile; K below and past a slice, N below and past a block, K split over clusters
SHAPES = [(1, 16, 8), (1, 896, 4864), (2, 144, 24), (16, 3584, 264), (17, 48, 136), (33, 1424, 1000), (64, 128, 128),
          (65, 128, 264), (100, 272, 520), (128, 896, 1000), (129, 144, 392), (333, 1424, 5000), (513, 2048, 264),
          (1025, 16, 136), (3, 18944, 40), (200, 18944, 136), (1, 8, 8), (5, 72, 136), (33, 520, 264), (301, 1416, 5000)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward(native, M, K, N):
    g = torch.Generator().manual_seed(M + K + N)
    a, w1, w2 = codes(g, M, K), codes(g, K, N), codes(g, K, N)
    sa, s1, s2 = scales(g, M, 0.02), scales(g, N, 0.6 / 5400 / K ** 0.5 * 50), scales(g, N, 0.01)
    wp = native.swiglu_pack_weights_int8(w1.cuda(), w2.cuda())
    y = native.swiglu_forward_int8(a.cuda(), sa.cuda(), wp, N, s1.cuda(), s2.cuda())
    native.swiglu_check_device_status()
    gate = ref.product(f64(a), f64(sa), f64(w1), f64(s1))
    up = ref.product(f64(a), f64(sa), f64(w2), f64(s2))
    assert_within(y, *ref.gated(*gate, *up))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,N,H", SHAPES)
def test_down(native, M, N, H, residual):
    g = torch.Generator().manual_seed(M + N + H)
    y, w3 = codes(g, M, N), codes(g, N, H)
    sy, s3 = scales(g, M, 0.02), scales(g, H, 0.01)
    r = make_inputs(M, H, 8, 3)[0]
    out = native.swiglu_down_forward_int8(y.cuda(), sy.cuda(), native.swiglu_pack_down_weights_int8(w3.cuda()), H,
                                          s3.cuda(), R=r.cuda() if residual else None)
    native.swiglu_check_device_status()
    assert_within(out, *ref.added(*ref.product(f64(y), f64(sy), f64(w3), f64(s3)), f64(r) if residual else 0.0))


@pytest.mark.parametrize("M", [1, 7, 16, 40, 64, 65, 128, 300])
@pytest.mark.parametrize("N,H", [(16, 8), (1008, 264), (1024, 1536)])
def test_integer_sums_are_exact(native, M, N, H):
    # |sum| <= 1024 * 2^14 = 2^24, so the fp32 sum is the integer, and the output its bf16 rounding
    g = torch.Generator().manual_seed(M + N)
    y, w3 = codes(g, M, N), codes(g, N, H)
    y[0], w3[:, 0] = -128, -128
    one = torch.ones(max(M, H))
    out = native.swiglu_down_forward_int8(y.cuda(), one[:M].cuda(), native.swiglu_pack_down_weights_int8(w3.cuda()),
                                          H, one[:H].cuda())
    want = (y.to(torch.int64) @ w3.to(torch.int64)).double().bfloat16()
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("M", [1, 16, 128, 300])
def test_large_sums(native, M):
    # every product 2^14 and one sign: sums of 18944 * 2^14 = 2^28.2
    N, H = 18944, 136
    y = torch.full((M, N), -128, dtype=torch.int8)
    w3 = torch.full((N, H), -128, dtype=torch.int8)
    w3[:, 1::2] = 127
    sy, s3 = torch.full((M,), 2.0 ** -8), torch.full((H,), 2.0 ** -9)
    out = native.swiglu_down_forward_int8(y.cuda(), sy.cuda(), native.swiglu_pack_down_weights_int8(w3.cuda()), H, s3.cuda())
    assert_within(out, *ref.added(*ref.product(f64(y), f64(sy), f64(w3), f64(s3)), 0.0))


@pytest.mark.parametrize("M", [5, 300])
def test_scales_that_are_not_finite_stay_alone(native, M):
    K, N = 144, 264
    g = torch.Generator().manual_seed(1)
    a, w1, w2 = (t.cuda() for t in (codes(g, M, K), codes(g, K, N), codes(g, K, N)))
    sa, s1, s2 = (t.cuda() for t in (scales(g, M, 0.02), scales(g, N, 0.01), scales(g, N, 0.01)))
    wp, w3p = native.swiglu_pack_weights_int8(w1, w2), native.swiglu_pack_down_weights_int8(w1)
    want = native.swiglu_forward_int8(a, sa, wp, N, s1, s2)
    want3 = native.swiglu_down_forward_int8(a, sa, w3p, N, s1)
    sa[3], s1[200] = float("nan"), float("inf")
    got, got3 = native.swiglu_forward_int8(a, sa, wp, N, s1, s2), native.swiglu_down_forward_int8(a, sa, w3p, N, s1)
    rows, cols = torch.arange(M) != 3, torch.arange(N) != 200
    for x, y in ((got, want), (got3, want3)):
        assert torch.equal(x[rows][:, cols], y[rows][:, cols])
        assert torch.isnan(x[3]).all()
    assert not torch.isfinite(got3[:, 200]).any()


@pytest.mark.parametrize("M,K,N", [(3, 144, 136), (70, 144, 136), (131, 272, 392)])
def test_outputs_end_where_they_should(native, M, K, N):
    g = torch.Generator().manual_seed(2)
    a, w1, w2 = (t.cuda() for t in (codes(g, M, K), codes(g, K, N), codes(g, K, N)))
    sa, s1 = scales(g, M, 0.02).cuda(), scales(g, N, 0.01).cuda()
    wp, w3p = native.swiglu_pack_weights_int8(w1, w2), native.swiglu_pack_down_weights_int8(w1)
    r = make_inputs(M, N, 8, 3)[0].cuda()
    pad = 64
    for call, want in ((lambda o: native.swiglu_forward_int8(a, sa, wp, N, s1, s1, Y=o),
                        native.swiglu_forward_int8(a, sa, wp, N, s1, s1)),
                       (lambda o: native.swiglu_down_forward_int8(a, sa, w3p, N, s1, R=r, Out=o),
                        native.swiglu_down_forward_int8(a, sa, w3p, N, s1, R=r))):
        buf = torch.full((M * N + 2 * pad,), 3.0, dtype=torch.bfloat16, device="cuda")
        view = buf[pad:-pad].view(M, N)
        call(view)
        assert torch.equal(view, want) and (buf[:pad] == 3).all() and (buf[-pad:] == 3).all()
    ws = torch.full((native.swiglu_int8_workspace_bytes(M, K, N) + 128,), 55, dtype=torch.uint8, device="cuda")
    inner = ws[64:-64]
    assert torch.equal(native.swiglu_forward_int8(a, sa, wp, N, s1, s1, workspace=inner),
                       native.swiglu_forward_int8(a, sa, wp, N, s1, s1))
    assert (ws[:64] == 55).all() and (ws[-64:] == 55).all()
    x = r.clone()  # in place
    assert torch.equal(native.swiglu_down_forward_int8(a, sa, w3p, N, s1, R=x, Out=x),
                       native.swiglu_down_forward_int8(a, sa, w3p, N, s1, R=r))


def test_no_tokens(native):
    w = torch.ones(64, 136, dtype=torch.int8, device="cuda")
    s, none = torch.ones(136, device="cuda"), torch.empty(0, device="cuda")
    a = torch.empty(0, 64, dtype=torch.int8, device="cuda")
    assert native.swiglu_forward_int8(a, none, native.swiglu_pack_weights_int8(w, w), 136, s, s).shape == (0, 136)
    assert native.swiglu_down_forward_int8(a, none, native.swiglu_pack_down_weights_int8(w), 136, s).shape == (0, 136)


def test_offsets_past_32_bits(native):
    M, K, N = 120001, 18944, 136  # 2.3e9 codes in, then out
    a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda")
    g = torch.Generator().manual_seed(4)
    w, sa, s = codes(g, K, N).cuda(), scales(g, M, 0.02).cuda(), scales(g, N, 1e-4).cuda()
    rows = [0, 1, 60000, 113359, M - 2, M - 1]
    out = native.swiglu_down_forward_int8(a, sa, native.swiglu_pack_down_weights_int8(w), N, s)
    native.swiglu_check_device_status()
    assert_within(out[rows], *ref.added(*ref.product(f64(a[rows]), f64(sa[rows]), f64(w), f64(s)), 0.0))
    del out
    a, w1, w2 = a[:, :16].contiguous(), codes(g, 16, K).cuda(), codes(g, 16, K).cuda()
    s1 = scales(g, K, 1e-2).cuda()
    y = native.swiglu_forward_int8(a, sa, native.swiglu_pack_weights_int8(w1, w2), K, s1, s1)
    native.swiglu_check_device_status()
    products = [ref.product(f64(a[rows]), f64(sa[rows]), f64(x), f64(s1)) for x in (w1, w2)]
    assert_within(y[rows], *ref.gated(*products[0], *products[1]))


@pytest.mark.parametrize("M,K,N,op", [(16, 3584, 18944, "int8"), (4096, 3584, 18944, "int8"),
                                      (16, 18944, 3584, "down"), (128, 4864, 896, "down"), (4096, 18944, 3584, "down")])
def test_workload_shapes(native, M, K, N, op):
    # sampled columns against every token
    g = torch.Generator().manual_seed(5)
    a, w1, w2 = codes(g, M, K), codes(g, K, N), codes(g, K, N)
    sa, s1, s2 = scales(g, M, 0.02), scales(g, N, 2e-3 / K ** 0.5), scales(g, N, 2e-3)
    cols = np.unique(np.concatenate([[0, N - 1, 127, 128], np.random.default_rng(0).integers(0, N, 24)]))
    if op == "int8":
        wp = native.swiglu_pack_weights_int8(w1.cuda(), w2.cuda())
        y = native.swiglu_forward_int8(a.cuda(), sa.cuda(), wp, N, s1.cuda(), s2.cuda())
    else:
        y = native.swiglu_down_forward_int8(a.cuda(), sa.cuda(), native.swiglu_pack_down_weights_int8(w1.cuda()), N, s1.cuda())
    native.swiglu_check_device_status()
    gate = ref.product(f64(a), f64(sa), f64(w1)[:, cols], f64(s1)[cols])
    up = ref.product(f64(a), f64(sa), f64(w2)[:, cols], f64(s2)[cols])
    assert_within(y[:, torch.from_numpy(cols).cuda()], *(ref.gated(*gate, *up) if op == "int8" else ref.added(*gate, 0.0)))


def block(native, x, wp, w3p, s1, s2, s3, N, H, spaces=(None, None)):
    """The gated block on bf16 tokens, quantised before each product."""
    q, sa = native.swiglu_quantize_int8(x)
    y = native.swiglu_forward_int8(q, sa, wp, N, s1, s2, workspace=spaces[0])
    q, sy = native.swiglu_quantize_int8(y)
    return native.swiglu_down_forward_int8(q, sy, w3p, H, s3, R=x, workspace=spaces[1])


def block_weights(native, K, N):
    """8-bit weights, a scale per channel, of float ones; and the float values they stand for."""
    _, w1, w2 = make_inputs(1, K, N, 6)
    w3 = make_inputs(N, K, 8, 7)[0]
    held = []
    for w in (w1, w2, w3):
        q, s = ref.quantise(f64(w).T)
        held.append((torch.from_numpy(q.T.astype(np.int8)).contiguous().cuda(), torch.from_numpy(s.astype(np.float32)).cuda()))
    return held


@pytest.mark.parametrize("M", [1, 16, 100, 300])
def test_the_block_as_it_is_served(native, M):
    K, N = 256, 656
    (w1, s1), (w2, s2), (w3, s3) = block_weights(native, K, N)
    x = make_inputs(M, K, 8, 8)[0]
    wp, w3p = native.swiglu_pack_weights_int8(w1, w2), native.swiglu_pack_down_weights_int8(w3)
    out = block(native, x.cuda(), wp, w3p, s1, s2, s3, N, K)
    native.swiglu_check_device_status()
    q, sa = ref.quantise(f64(x))
    y, ey = ref.gated(*ref.product(q, sa, f64(w1), f64(s1)), *ref.product(q, sa, f64(w2), f64(s2)))
    qy, sy = ref.quantise(y)
    # a value of Y that is off by ey lands on a code off by at most ey / s + 1, its scale by max(ey) / 127
    want, e = ref.product(qy, sy, f64(w3), f64(s3))
    moved = (ey + sy[:, None] * 1.0 + abs(qy) * ey.max(1, keepdims=True) / 127) @ (abs(f64(w3)) * f64(s3))
    assert_within(out, *ref.added(want, e + moved, f64(x)))


def test_streams_and_graphs(native):
    K, N = 272, 656
    (w1, s1), (w2, s2), (w3, s3) = block_weights(native, K, N)
    wp, w3p = native.swiglu_pack_weights_int8(w1, w2), native.swiglu_pack_down_weights_int8(w3)
    for M in (5, 200):
        xs = [make_inputs(M, K, 8, 10 + i)[0].cuda() for i in range(2)]
        alone = [block(native, x, wp, w3p, s1, s2, s3, N, K) for x in xs]
        streams = [torch.cuda.Stream() for _ in xs]
        spaces = [(native.swiglu_int8_workspace(M, K, N), native.swiglu_down_int8_workspace(M, N, K)) for _ in xs]
        torch.cuda.synchronize()
        got = []
        for st, x, ws in zip(streams, xs, spaces):
            with torch.cuda.stream(st):
                for _ in range(5):
                    last = block(native, x, wp, w3p, s1, s2, s3, N, K, ws)
                got.append(last)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, got))
        x = xs[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = block(native, x, wp, w3p, s1, s2, s3, N, K)
        for i in (1, 0):
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


@pytest.mark.parametrize("M", [16, 300])
def test_a_stalled_pipeline_is_reported(native, M):
    K, N = 512, 264
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


def test_refusals(native):
    g = torch.Generator().manual_seed(1)
    a, w, s = codes(g, 4, 64).cuda(), codes(g, 64, 136).cuda(), torch.ones(136, device="cuda")
    sa = s[:4].clone()
    wp, w3p = native.swiglu_pack_weights_int8(w, w), native.swiglu_pack_down_weights_int8(w)
    for bad in (lambda: native.swiglu_pack_weights_int8(w.float(), w),
                lambda: native.swiglu_pack_weights_int8(w, w[:, :128].contiguous()),
                lambda: native.swiglu_pack_weights_int8(w, w, Wpacked=wp[:-1]),
                lambda: native.swiglu_forward_int8(a.view(torch.uint8), sa, wp, 136, s, s),
                lambda: native.swiglu_forward_int8(a, sa[:3], wp, 136, s, s),
                lambda: native.swiglu_forward_int8(a, sa.double(), wp, 136, s, s),
                lambda: native.swiglu_forward_int8(a, sa, wp, 136, s[:128], s),
                lambda: native.swiglu_forward_int8(a, sa, wp[:-32768], 136, s, s),
                lambda: native.swiglu_forward_int8(a, sa, wp, 136, s, s, Y=torch.empty(4, 128, device="cuda").bfloat16()),
                lambda: native.swiglu_forward_int8(a.t(), sa, wp, 136, s, s),
                lambda: native.swiglu_down_forward_int8(a, sa, w3p, 136, s, R=torch.zeros(4, 136, device="cuda")),
                lambda: native.swiglu_down_forward_int8(a, sa, w3p[:100], 136, s),
                lambda: native.swiglu_forward_int8(a, sa.cpu(), wp, 136, s, s)):
        with pytest.raises(ValueError):
            bad()
    # many tokens and columns need a workspace
    big, one, wide = codes(g, 1000, 64).cuda(), torch.ones(1000, device="cuda"), torch.ones(18944, device="cuda")
    assert native.swiglu_int8_workspace_bytes(1000, 64, 18944) == 2 * 1000 * 64
    w = codes(g, 64, 18944).cuda()
    with pytest.raises(native.SwigluError):
        native.swiglu_forward_int8(big, one, native.swiglu_pack_weights_int8(w, w), 18944, wide, wide,
                                   workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("M", [7, 300])
def test_part_of_a_batch(native, M):
    # tokens from the third on, as views: codes start on a row, scales on any float
    K, N = 144, 264
    g = torch.Generator().manual_seed(3)
    a, w, r = codes(g, M, K).cuda(), codes(g, K, N).cuda(), make_inputs(M, N, 8, 3)[0].cuda()
    sa, s = scales(g, M, 0.02).cuda(), scales(g, N, 0.01).cuda()
    wp, w3p = native.swiglu_pack_weights_int8(w, w), native.swiglu_pack_down_weights_int8(w)
    assert torch.equal(native.swiglu_forward_int8(a[3:], sa[3:], wp, N, s, s),
                       native.swiglu_forward_int8(a, sa, wp, N, s, s)[3:])
    assert torch.equal(native.swiglu_down_forward_int8(a[3:], sa[3:], w3p, N, s, R=r[3:].clone()),
                       native.swiglu_down_forward_int8(a, sa, w3p, N, s, R=r)[3:])


def test_the_common_case_and_the_others_agree(native):
    # outputs given, a stream given, a subclass of Tensor: checked and called in Python
    class Mine(torch.Tensor):
        pass

    M, K, N = 40, 272, 264
    g = torch.Generator().manual_seed(4)
    x = make_inputs(M, K, 8, 5)[0].cuda()
    w, s = codes(g, K, N).cuda(), scales(g, N, 0.01).cuda()
    wp = native.swiglu_pack_weights_int8(w, w)
    q, sa = native.swiglu_quantize_int8(x)
    y = native.swiglu_forward_int8(q, sa, wp, N, s, s)
    for q2, sa2 in (native.swiglu_quantize_int8(x, Q=torch.empty_like(q)),
                    native.swiglu_quantize_int8(x, stream=torch.cuda.current_stream()),
                    native.swiglu_quantize_int8(x.as_subclass(Mine))):
        assert torch.equal(q, q2) and torch.equal(sa, sa2)
    for y2 in (native.swiglu_forward_int8(q, sa, wp, N, s, s, Y=torch.empty_like(y)),
               native.swiglu_forward_int8(q, sa, wp, N, s, s, stream=torch.cuda.current_stream()),
               native.swiglu_forward_int8(q, sa, wp, np.int64(N), s, s)):
        assert torch.equal(y, y2)
    with pytest.raises(TypeError):
        native.swiglu_quantize_int8()
    with pytest.raises(ValueError):
        native.swiglu_quantize_int8(3)


def test_one_workspace_in_stream_order(native):
    # calls of several shapes take turns on one workspace
    K, N, H = 272, 4096, 264
    g = torch.Generator().manual_seed(6)
    w, w3 = codes(g, K, N).cuda(), codes(g, N, H).cuda()
    s, s3 = scales(g, N, 0.01).cuda(), scales(g, H, 0.01).cuda()
    wp, w3p = native.swiglu_pack_weights_int8(w, w), native.swiglu_pack_down_weights_int8(w3)
    runs = []
    for M in (2000, 1100, 3):
        a, y, sa = codes(g, M, K).cuda(), codes(g, M, N).cuda(), scales(g, M, 0.02).cuda()
        runs.append((lambda ws, a=a, sa=sa: native.swiglu_forward_int8(a, sa, wp, N, s, s, workspace=ws)))
        runs.append((lambda ws, y=y, sa=sa: native.swiglu_down_forward_int8(y, sa, w3p, H, s3, workspace=ws)))
    need = max(native.swiglu_int8_workspace_bytes(2000, K, N), native.swiglu_down_int8_workspace_bytes(2000, N, H))
    shared = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    want = [f(None) for f in runs]
    got = [f(shared) for _ in range(3) for f in runs]
    assert all(torch.equal(a, b) for a, b in zip(got, want * 3))


@pytest.mark.parametrize("K,N,down,Ms", [(2816, 2640, True, (129, 128)), (2096, 5864, True, (134, 127)),
                                         (464, 9808, True, (200, 150)), (896, 4864, False, (300, 129, 1)),
                                         (520, 264, False, (70, 69, 1))])
def test_a_workspace_for_a_batch_serves_smaller_ones(native, K, N, down, Ms):
    # a larger batch may run on single CTAs, which need none, where a smaller one takes pairs
    need = native.swiglu_down_int8_workspace_bytes if down else native.swiglu_int8_workspace_bytes
    plan = native.swiglu_down_plan_string_int8 if down else native.swiglu_plan_string_int8
    sizes = [need(M, K, N) for M in range(1, 700)]
    assert sizes == sorted(sizes)
    assert all(size == 2 * M * K for M, size in enumerate(sizes, 1) if "pairs" in plan(M, K, N))
    assert need(4097, K, N) >= sizes[-1] and need(1 << 20, K, N) == 2 * K << 20
    g = torch.Generator().manual_seed(K)
    w, s = codes(g, K, N).cuda(), scales(g, N, 0.01).cuda()
    wp = native.swiglu_pack_down_weights_int8(w) if down else native.swiglu_pack_weights_int8(w, w)
    ws = torch.empty(need(Ms[0], K, N), dtype=torch.uint8, device="cuda")
    for M in Ms:
        a, sa = codes(g, M, K).cuda(), scales(g, M, 0.02).cuda()
        call = (lambda ws: native.swiglu_down_forward_int8(a, sa, wp, N, s, workspace=ws)) if down else \
            (lambda ws: native.swiglu_forward_int8(a, sa, wp, N, s, s, workspace=ws))
        assert torch.equal(call(ws), call(None))
    native.swiglu_check_device_status()


def test_calls_made_from_python_agree(native, monkeypatch):
    # every 8-bit call without _torch_calls.so
    M, K, N = 70, 272, 264
    g = torch.Generator().manual_seed(4)
    x, b1, b2 = (t.cuda() for t in make_inputs(M, K, N, 5))
    w, s = codes(g, K, N).cuda(), scales(g, N, 0.01).cuda()
    wp, w3p, bp = native.swiglu_pack_weights_int8(w, w), native.swiglu_pack_down_weights_int8(w), native.swiglu_pack_weights(b1, b2)

    def calls():
        q, sa = native.swiglu_quantize_int8(x)
        y = native.swiglu_forward_int8(q, sa, wp, N, s, s)
        kept = native.swiglu_forward_checkpoint(x, bp, N)
        return (q, sa, y, native.swiglu_down_forward_int8(q, sa, w3p, N, s, R=y), *kept, native.swiglu_checkpoint_output(*kept[1:]),
                *native.swiglu_backward_checkpoint(x, bp, y, *kept[1:]),
                *native.swiglu_backward_checkpoint(q, bp, y, *kept[1:], scale_a=sa))

    want = calls()
    monkeypatch.setattr(native, "_calls", native._NoCalls())
    got = calls()
    native.swiglu_check_device_status()
    assert len(want) == len(got) == 15 and all(torch.equal(a, b) for a, b in zip(want, got))
