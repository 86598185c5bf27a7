"""Tokens in 8 bits, and training with Gate and Up kept in 8 bits, against float64 (needs a GB300).

Codes of bf16 values have one right value; everything else is held to the worst-case
bound of the roundings the kernels make (oracle/int8_ref.py).
"""
import numpy as np
import pytest
import torch

from oracle import int8_ref as ref
from oracle.backward_ref import FP32
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


def tokens(M, K, seed):
    """bf16 rows of magnitudes from 2^-130 to 2^126, with rows that are zero, that hold many exact
    halves (a largest value that is a multiple of 127) and that are all equal."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-20, 20, (M, 1), generator=g).float())
    for i, row in enumerate(x):
        if i % 8 == 1:
            row.zero_()
        elif i % 8 == 2:
            row.copy_(torch.randint(-127, 128, (K,), generator=g) / 2)
            row[0] = 127.0
        elif i % 8 == 3:
            row.fill_(-3.0)
        elif i % 8 == 4:
            row.mul_(2.0 ** (-130 if i % 16 == 4 else 100) / row.abs().max())
        elif i % 8 == 5:
            row.copy_(torch.randint(-254, 255, (K,), generator=g) * 2.0 ** -9)
            row[-1] = -254 * 2.0 ** -9
    return x.bfloat16()


@pytest.mark.parametrize("M,K", [(1, 8), (9, 16), (40, 264), (33, 896), (17, 3584), (1, 18944), (3, 18944),
                                 (2, 40008), (1000, 72)])
def test_quantised_tokens_are_exact(native, M, K):
    x = tokens(M, K, M + K)
    q, s = native.swiglu_quantize_int8(x.cuda())
    codes, scale = ref.quantise(f64(x))
    assert np.array_equal(f64(q), codes)
    assert np.array_equal(s.cpu().numpy(), scale.astype(np.float32))
    assert np.abs(codes).max() <= 127


def test_every_bf16_pair_of_halves(native):
    # each largest value of 8 significant bits with values at and beside the halves of its grid
    tops = torch.arange(128, 256).float()
    rows = [torch.cat([t[None], torch.arange(0, 256).float()[:255] * (t / 254)]) for t in tops]
    x = torch.stack(rows).bfloat16()
    x = torch.cat([x, -x]).repeat(1, 1)
    x[:, 1:] = torch.where(x[:, 1:].abs() > x[:, :1].abs(), x[:, :1].expand(-1, 255), x[:, 1:])
    q, s = native.swiglu_quantize_int8(x.cuda())
    codes, scale = ref.quantise(f64(x))
    assert np.array_equal(f64(q), codes) and np.array_equal(s.cpu().numpy(), scale.astype(np.float32))


def test_rows_with_nan_or_infinity(native):
    x = tokens(24, 136, 5)
    x[6, 3], x[7, 0], x[14, 135] = float("nan"), float("inf"), float("-inf")
    q, s = native.swiglu_quantize_int8(x.cuda())
    bad = [6, 7, 14]
    good = [i for i in range(24) if i not in bad]
    codes, scale = ref.quantise(f64(x)[good])
    assert np.array_equal(f64(q)[good], codes) and np.array_equal(f64(s)[good], scale)
    assert torch.isnan(s[bad]).all()


def test_quantise_writes_nothing_else(native):
    M, K = 5, 72
    x = tokens(M, K, 1).cuda()
    q, s = torch.full((M * K + 64,), 77, dtype=torch.int8, device="cuda"), torch.full((M + 8,), -5.0, device="cuda")
    native.swiglu_quantize_int8(x, Q=q[32:32 + M * K].view(M, K), scale=s[4:4 + M])
    assert (q[:32] == 77).all() and (q[32 + M * K:] == 77).all() and (s[:4] == -5).all() and (s[4 + M:] == -5).all()
    q, s = native.swiglu_quantize_int8(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,)


# one token, a ragged last tile and column block, several tiles, N that is no multiple of 16
SHAPES = [(1, 8, 8), (1, 200, 264), (2, 896, 1000), (33, 72, 136), (128, 896, 1024), (130, 1000, 520),
          (257, 264, 392), (300, 200, 264), (513, 1416, 1000), (2000, 72, 72)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward_keeps_gate_and_up(native, M, K, N):
    a, w1, w2 = make_inputs(M, K, N, M + K + N)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    y, gate, up, scale = native.swiglu_forward_checkpoint(a.cuda(), wp, N)
    native.swiglu_check_device_status()
    # the same accumulators and the same last step as the kernel without the checkpoint
    assert torch.equal(y, native.swiglu_forward_variant(a.cuda(), wp, N, native.SWIGLU_VARIANT_LARGE_M_PAIR))
    for w, codes, s in ((w1, gate, scale[0]), (w2, up, scale[1])):
        x = f64(a) @ f64(w)
        err = K * FP32 * (abs(f64(a)) @ abs(f64(w))) + 1e-30
        s = f64(s)
        # the scale: the largest within the accumulators' error, one division
        top = np.maximum(ref.block_largest(x), ref.LEAST)
        assert (abs(s * 127 - top) <= ref.block_largest(err) + 2 * FP32 * top).all()
        # a value is half a step off, with a step's rounding of the product (127 steps at most)
        step = ref.wide(s, N)
        assert (abs(f64(codes) * step - x) <= (0.5 + 127 * 2 * FP32) * step + err).all()


def kept(M, N, seed):
    """A checkpoint of normal values, with zero and tiny groups."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-127, 128, (2, M, N), generator=g, dtype=torch.int8)
    scale = torch.rand(2, ref.blocks(N), M, generator=g) * 0.03
    scale[:, :, ::5] *= 2.0 ** -60
    codes[:, ::7] = 0
    return codes[0], codes[1], scale


def values(gate, up, scale):
    n = gate.shape[1]
    return f64(gate) * ref.wide(f64(scale[0]), n), f64(up) * ref.wide(f64(scale[1]), n)


@pytest.mark.parametrize("M,N", [(1, 8), (3, 136), (77, 1000), (300, 264), (5, 18944), (2600, 72)])
def test_output_restored(native, M, N):
    ck = kept(M, N, M + N)
    y = native.swiglu_checkpoint_output(*(t.cuda() for t in ck))
    g, u = values(*ck)
    assert_within(y, *ref.gated(g, FP32 * abs(g), u, FP32 * abs(u)))


def gradient_inputs(M, K, N, seed):
    a, w1, w2 = make_inputs(M, K, N, seed)
    return a, w1, w2, make_inputs(M, N, 8, seed + 1)[0], kept(M, N, seed + 2)


def check_gradients(native, M, K, N, seed, eight_bits):
    a, w1, w2, dy, ck = gradient_inputs(M, K, N, seed)
    sa, av, a_err = None, f64(a), 0.0
    if eight_bits:
        a, sa = (t.cpu() for t in native.swiglu_quantize_int8(a.cuda()))
        av = f64(a) * f64(sa)[:, None]
        a_err = 2 * FP32 * abs(av)
        sa = sa.cuda()
    outs = native.swiglu_backward_checkpoint(a.cuda(), native.swiglu_pack_weights(w1.cuda(), w2.cuda()), dy.cuda(),
                                             *(t.cuda() for t in ck), scale_a=sa)
    native.swiglu_check_device_status()
    args = (av, f64(w1), f64(w2), *values(*ck), f64(dy))
    for out, want, bound in zip(outs, ref.backward_values(*args), ref.backward_bounds(*args, a_err)):
        assert_within(out, want, bound)


@pytest.mark.parametrize("eight_bits", [False, True])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_backward_matches_the_formula(native, M, K, N, eight_bits):
    check_gradients(native, M, K, N, M + K + N, eight_bits)


def test_backward_matches_differences(native):
    # central differences of sum(dY * SiLU(g) u) through the checkpoint's values, as dA and dW see
    # them: g and u move with A W1 and A W2
    M, K, N, h = 9, 72, 136, 1e-4
    a, w1, w2, dy, ck = gradient_inputs(M, K, N, 3)
    outs = [f64(t) for t in native.swiglu_backward_checkpoint(
        a.cuda(), native.swiglu_pack_weights(w1.cuda(), w2.cuda()), dy.cuda(), *(t.cuda() for t in ck))]
    base = [f64(t) for t in (a, w1, w2)]
    g, u = values(*ck)
    d = f64(dy)

    def loss(x, p, q):
        return float((ref.silu(g + x @ p - base[0] @ base[1]) * (u + x @ q - base[0] @ base[2]) * d).sum())

    rng = np.random.default_rng(0)
    for which, bound in enumerate(ref.backward_bounds(*base, g, u, d)):
        for _ in range(40):
            at = tuple(rng.integers(0, n) for n in base[which].shape)
            vals = []
            for sign in (1, -1):
                moved = [x.copy() for x in base]
                moved[which][at] += sign * h
                vals.append(loss(*moved))
            assert abs((vals[0] - vals[1]) / (2 * h) - outs[which][at]) <= bound[at] + 1e-6


def test_backward_parts_asked_for(native):
    M, K, N = 130, 256, 392
    a, w1, w2, dy, ck = gradient_inputs(M, K, N, 4)
    wp, dy, ck = native.swiglu_pack_weights(w1.cuda(), w2.cuda()), dy.cuda(), [t.cuda() for t in ck]
    q, sa = native.swiglu_quantize_int8(a.cuda())
    both = native.swiglu_backward_checkpoint(q, wp, dy, *ck, scale_a=sa)
    da, none1, none2 = native.swiglu_backward_checkpoint(q, wp, dy, *ck, scale_a=sa, need_weight=False)
    assert none1 is None and none2 is None and torch.equal(da, both[0])
    none, dw1, dw2 = native.swiglu_backward_checkpoint(q, wp, dy, *ck, scale_a=sa, need_input=False)
    assert none is None and torch.equal(dw1, both[1]) and torch.equal(dw2, both[2])


def test_no_tokens(native):
    w = torch.ones(64, 136, dtype=torch.bfloat16, device="cuda")
    wp = native.swiglu_pack_weights(w, w)
    a = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, gate, up, scale = native.swiglu_forward_checkpoint(a, wp, 136)
    assert y.shape == gate.shape == up.shape == (0, 136) and scale.shape == (2, 2, 0)
    assert native.swiglu_checkpoint_output(gate, up, scale).shape == (0, 136)
    da, dw1, dw2 = native.swiglu_backward_checkpoint(a, wp, y, gate, up, scale)
    assert da.shape == (0, 64) and not dw1.any() and not dw2.any()


def test_a_token_that_is_not_finite_stays_alone(native):
    M, K, N = 300, 136, 264
    a, w1, w2 = make_inputs(M, K, N, 8)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    want = native.swiglu_forward_checkpoint(a.cuda(), wp, N)
    b = a.clone()
    b[7, 3], b[290, 100] = float("nan"), float("inf")
    got = native.swiglu_forward_checkpoint(b.cuda(), wp, N)
    keep = torch.ones(M, dtype=torch.bool)
    keep[[7, 290]] = False
    for x, y in zip(got[:3], want[:3]):
        assert torch.equal(x[keep], y[keep])
    assert torch.equal(got[3][:, :, keep], want[3][:, :, keep])
    assert torch.isnan(got[3][:, :, [7, 290]]).all()
    restored = native.swiglu_checkpoint_output(*got[1:])
    assert torch.isnan(restored[[7, 290]]).all() and torch.isfinite(restored[keep]).all()


def test_outputs_end_where_they_should(native):
    M, K, N, pad = 131, 72, 136, 64
    a, w1, w2 = make_inputs(M, K, N, 9)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    bufs = [torch.full((n + 2 * pad,), v, dtype=t, device="cuda")
            for n, v, t in ((M * N, 3, torch.bfloat16), (M * N, 77, torch.int8), (M * N, 77, torch.int8),
                            (2 * 2 * M, -5, torch.float32))]
    shapes = ((M, N), (M, N), (M, N), (2, 2, M))
    views = [b[pad:-pad].view(s) for b, s in zip(bufs, shapes)]
    native.swiglu_forward_checkpoint(a.cuda(), wp, N, *views)
    assert torch.equal(views[1], native.swiglu_forward_checkpoint(a.cuda(), wp, N)[1])
    for b, v in zip(bufs, (3, 77, 77, -5)):
        assert (b[:pad] == v).all() and (b[-pad:] == v).all()


def test_offsets_past_32_bits(native):
    # codes of 2.3e9 values: rows at both ends against the formula
    M, N, K = 120001, 18944, 16
    gate = torch.randint(-127, 128, (M, N), dtype=torch.int8, device="cuda")
    up = gate.flip(0)
    scale = torch.rand(2, N // 128, M, device="cuda") * 0.03
    rows = [0, 1, 60000, 113999, M - 2, M - 1]
    y = native.swiglu_checkpoint_output(gate, up, scale)
    g, u = values(gate[rows], up[rows], scale[:, :, rows])
    assert_within(y[rows], *ref.gated(g, FP32 * abs(g), u, FP32 * abs(u)))
    a, w1, w2 = make_inputs(M, K, N, 2)
    a, w1, w2 = a.cuda(), w1.cuda(), w2.cuda()
    wp = native.swiglu_pack_weights(w1, w2)
    da, _, _ = native.swiglu_backward_checkpoint(a, wp, y, gate, up, scale, need_weight=False)
    native.swiglu_check_device_status()
    args = (f64(a[rows]), f64(w1), f64(w2), g, u, f64(y[rows]))
    assert_within(da[rows], ref.backward_values(*args)[0], ref.backward_bounds(*args)[0])
    del da, y
    y2, gate2, up2, scale2 = native.swiglu_forward_checkpoint(a, wp, N)
    native.swiglu_check_device_status()
    for w, codes, s in ((w1, gate2, scale2[0]), (w2, up2, scale2[1])):
        x, step = f64(a[rows]) @ f64(w), ref.wide(f64(s[:, rows]), N)
        err = K * FP32 * (abs(f64(a[rows])) @ abs(f64(w)))
        assert (abs(f64(codes[rows]) * step - x) <= (0.5 + 127 * 2 * FP32) * step + err).all()


def step(native, a, wp, w3p, d_out, N, H, workspace=None):
    """A training step of the block with the input, Gate and Up kept in 8 bits."""
    q, sa = native.swiglu_quantize_int8(a)
    y, *ck = native.swiglu_forward_checkpoint(a, wp, N)
    out = native.swiglu_down_forward(y, w3p, H, R=a)
    d_y, d_w3 = native.swiglu_down_backward(d_out, w3p, native.swiglu_checkpoint_output(*ck))
    return (out, d_w3, *native.swiglu_backward_checkpoint(q, wp, d_y, *ck, scale_a=sa, workspace=workspace))


def test_a_training_step(native):
    # against the recomputing backward: they differ by the 8-bit rounding of Gate and Up alone.
    # A code is off by at most half a step, uniform to good measure (step^2 / 12), a step is the
    # block's largest / 127: at most 4 standard deviations / 127 here, 0.009 of one; SiLU' and U
    # each carry such an error into dG, so a gradient is off by some 0.02 of itself; 0.04 bounds it.
    M, K, N = 513, 256, 648
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 12))
    w3, d_out = make_inputs(N, K, 8, 13)[0].cuda() * 0.05, make_inputs(M, K, 8, 14)[0].cuda()
    wp, w3p = native.swiglu_pack_weights(w1, w2), native.swiglu_pack_down_weights(w3)
    out, d_w3, *grads = step(native, a, wp, w3p, d_out, N, K)
    y = native.swiglu_forward(a, wp, N)
    want_dy, want_w3 = native.swiglu_down_backward(d_out, w3p, y)
    want = native.swiglu_backward(a, wp, want_dy)
    assert torch.equal(out, native.swiglu_down_forward(y, w3p, K, R=a)) or \
        (out.float() - native.swiglu_down_forward(y, w3p, K, R=a).float()).norm() < 0.01 * out.float().norm()
    for x, w in zip((d_w3, *grads), (want_w3, *want)):
        assert (x.float() - w.float()).norm() <= 0.04 * w.float().norm()


def test_streams_and_graphs(native):
    # two steps at once on two streams with workspaces of their own, and a captured step replayed
    # on new inputs: bit for bit what each gives alone
    M, K, N = 200, 264, 648
    w = [t.cuda() for t in make_inputs(M, K, N, 20)]
    wp, w3p = native.swiglu_pack_weights(w[1], w[2]), native.swiglu_pack_down_weights(w[1].t().contiguous())
    xs = [make_inputs(M, K, N, 30 + i)[0].cuda() for i in range(2)]
    ds = [make_inputs(M, K, N, 40 + i)[0].cuda() for i in range(2)]
    alone = [step(native, x, wp, w3p, d, N, K) for x, d in zip(xs, ds)]
    streams = [torch.cuda.Stream() for _ in xs]
    spaces = [native.swiglu_backward_checkpoint_workspace(M, K, N) for _ in xs]
    torch.cuda.synchronize()
    got = []
    for s, x, d, ws in zip(streams, xs, ds, spaces):
        with torch.cuda.stream(s):
            for _ in range(3):
                last = step(native, x, wp, w3p, d, N, K, ws)
            got.append(last)
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    x, d = xs[0].clone(), ds[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(native, x, wp, w3p, d, N, K)
    for i in (1, 0):
        x.copy_(xs[i])
        d.copy_(ds[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, alone[i]))
    # and on a stream given to the calls
    s = streams[0]
    s.wait_stream(torch.cuda.current_stream())
    y, *ck = native.swiglu_forward_checkpoint(xs[1], wp, N, stream=s)
    r = native.swiglu_checkpoint_output(*ck, stream=s)
    q, sa = native.swiglu_quantize_int8(xs[1], stream=s)
    g = native.swiglu_backward_checkpoint(q, wp, r, *ck, scale_a=sa, stream=s)
    s.synchronize()
    y1, *ck1 = native.swiglu_forward_checkpoint(xs[1], wp, N)
    r1 = native.swiglu_checkpoint_output(*ck1)
    g1 = native.swiglu_backward_checkpoint(q, wp, r1, *ck1, scale_a=sa)
    assert torch.equal(y, y1) and torch.equal(r, r1) and all(torch.equal(a, b) for a, b in zip(g, g1))


def test_refusals(native):
    a, w1, w2, dy, (gate, up, scale) = gradient_inputs(4, 64, 136, 1)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    a, dy, gate, up, scale = (t.cuda() for t in (a, dy, gate, up, scale))
    for bad in (lambda: native.swiglu_quantize_int8(a.float()),
                lambda: native.swiglu_quantize_int8(a[0]),
                lambda: native.swiglu_quantize_int8(a, Q=gate),
                lambda: native.swiglu_quantize_int8(a, scale=scale[0, 0].double()),
                lambda: native.swiglu_forward_checkpoint(a, wp[:-16384], 136),
                lambda: native.swiglu_forward_checkpoint(a, wp, 136, gate=gate.view(torch.uint8)),
                lambda: native.swiglu_forward_checkpoint(a, wp, 136, scale=scale[:, :1].contiguous()),
                lambda: native.swiglu_checkpoint_output(gate, up[:3], scale),
                lambda: native.swiglu_checkpoint_output(gate.t(), up.t(), scale),
                lambda: native.swiglu_checkpoint_output(gate, up, scale.half()),
                lambda: native.swiglu_backward_checkpoint(a, wp, dy[:3], gate, up, scale),
                lambda: native.swiglu_backward_checkpoint(a.to(torch.int8), wp, dy, gate, up, scale),
                lambda: native.swiglu_backward_checkpoint(a, wp, dy, gate, up, scale, scale_a=scale[0, 0]),
                lambda: native.swiglu_backward_checkpoint(a[:3], wp, dy, gate, up, scale)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(native.SwigluError):  # a workspace too small
        native.swiglu_backward_checkpoint(a, wp, dy, gate, up, scale,
                                          workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(native.SwigluError):  # an output that is an input
        native.swiglu_backward_checkpoint(a, wp, dy, gate, up, scale, dA=a)
    with pytest.raises(native.SwigluError):  # rows that start at 8 bytes
        native.swiglu_checkpoint_output(gate, up, scale, Y=torch.empty(4, 136 + 8, dtype=torch.bfloat16,
                                                                      device="cuda").view(-1)[4:4 + 4 * 136].view(4, 136))


@pytest.mark.parametrize("M", [16, 300])
def test_a_stalled_pipeline_is_reported(native, M):
    K, N = 512, 264
    a, w1, w2, dy, ck = gradient_inputs(M, K, N, 2)
    a, dy, ck = a.cuda(), dy.cuda(), [t.cuda() for t in ck]
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    want = native.swiglu_forward_checkpoint(a, wp, N), native.swiglu_backward_checkpoint(a, wp, dy, *ck)
    native.swiglu_check_device_status()
    for call in (lambda: native.swiglu_forward_checkpoint(a, wp, N),
                 lambda: native.swiglu_backward_checkpoint(a, wp, dy, *ck)):
        native.swiglu_testing_inject_stall(True, 20)
        try:
            call()
            with pytest.raises(native.SwigluError) as e:
                native.swiglu_check_device_status()
            assert e.value.code == native.SWIGLU_ERR_TIMEOUT
        finally:
            native.swiglu_testing_inject_stall(False, 1000)
        native.swiglu_check_device_status()
    got = native.swiglu_forward_checkpoint(a, wp, N), native.swiglu_backward_checkpoint(a, wp, dy, *ck)
    for x, y in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_many_tiles_of_many_slices(native):
    # several rounds of tiles for each pair of CTAs, each a long sum: the checkpoint of a workload's
    # shape on sampled rows and columns, and calls in a row with nothing between them
    M, K, N = 1024, 3584, 18944
    a, w1, w2 = make_inputs(M, K, N, 3)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    first = native.swiglu_forward_checkpoint(a.cuda(), wp, N)
    ad = a.cuda()
    for _ in range(20):
        last = native.swiglu_forward_checkpoint(ad, wp, N)
        restored = native.swiglu_checkpoint_output(*last[1:])
    native.swiglu_check_device_status()
    assert all(torch.equal(x, y) for x, y in zip(first, last))
    rows = np.unique(np.random.default_rng(0).integers(0, M, 12))
    at = torch.from_numpy(rows).cuda()
    for w, codes, s in ((w1, last[1], last[3][0]), (w2, last[2], last[3][1])):
        x, step = f64(a[rows]) @ f64(w), ref.wide(f64(s[:, at]), N)
        err = K * FP32 * (abs(f64(a[rows])) @ abs(f64(w)))
        assert (abs(f64(codes[at]) * step - x) <= (0.5 + 127 * 2 * FP32) * step + err).all()
    g, u = (f64(c[at]) * ref.wide(f64(s[:, at]), N) for c, s in ((last[1], last[3][0]), (last[2], last[3][1])))
    assert_within(restored[at], *ref.gated(g, FP32 * abs(g), u, FP32 * abs(u)))


def test_scales_of_any_size(native):
    # the input's scales from 2^-110 to 2^100, zero, negative and subnormal: dA does not depend on
    # them, and the weight gradients are those of the values (rows of large values would drown the
    # others, so each goes alone)
    M, K, N = 16, 72, 136
    a, w1, w2, dy, ck = gradient_inputs(M, K, N, 6)
    q, _ = (t.cpu() for t in native.swiglu_quantize_int8(a.cuda()))
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    g, u = values(*ck)
    for i, s in enumerate((2.0 ** -110, 3e-20, -0.75, 1.0, 1.9999999, 2.0 ** 100, 0.0, 1e-40)):
        sa = torch.zeros(M)
        sa[i] = s
        outs = native.swiglu_backward_checkpoint(q.cuda(), wp, dy.cuda(), *(t.cuda() for t in ck), scale_a=sa.cuda())
        av = f64(q) * f64(sa)[:, None]
        args = (av, f64(w1), f64(w2), g, u, f64(dy))
        # a subnormal scale keeps its codes times itself in bf16, 2^-133 apart
        bounds = ref.backward_bounds(*args, 2 * FP32 * abs(av) + (2.0 ** -134 if s == 1e-40 else 0.0))
        for out, want, bound in zip(outs, ref.backward_values(*args), bounds):
            assert_within(out, want, bound)
    native.swiglu_check_device_status()


def test_an_input_scale_that_is_not_finite(native):
    # the weight gradients sum over all tokens and are lost; dA of every token is not
    M, K, N = 40, 72, 136
    a, w1, w2, dy, ck = gradient_inputs(M, K, N, 7)
    q, sa = native.swiglu_quantize_int8(a.cuda())
    wp, dy, ck = native.swiglu_pack_weights(w1.cuda(), w2.cuda()), dy.cuda(), [t.cuda() for t in ck]
    want = native.swiglu_backward_checkpoint(q, wp, dy, *ck, scale_a=sa)[0]
    sa[3] = float("nan")
    da, dw1, dw2 = native.swiglu_backward_checkpoint(q, wp, dy, *ck, scale_a=sa)
    keep = torch.arange(M) != 3
    assert torch.equal(da[keep], want[keep]) and torch.isfinite(da).all()
    assert torch.isnan(dw1).any() and torch.isnan(dw2).any()


def test_pair_kernels_behind_a_kernel_of_many_blocks(native):
    # CTAs of a pair kernel that start while another kernel's blocks still fill their SMs, each at its
    # own time: thousands of calls in a row, forward and backward (an allocation of tensor memory that
    # one CTA of a pair came late to once stood still there)
    M, K, N = 4096, 64, 18944
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 5))
    wp = native.swiglu_pack_weights(w1, w2)
    first = native.swiglu_forward_checkpoint(a, wp, N)
    ws = native.swiglu_backward_checkpoint_workspace(M, K, N)
    for _ in range(40):
        for _ in range(100):
            last = native.swiglu_forward_checkpoint(a, wp, N)
            y = native.swiglu_checkpoint_output(*last[1:])
        for _ in range(5):
            grads = native.swiglu_backward_checkpoint(a, wp, y, *last[1:], workspace=ws)
        torch.cuda.synchronize()
    native.swiglu_check_device_status()
    assert all(torch.equal(x, z) for x, z in zip(first, last))
    want = native.swiglu_backward_checkpoint(a, wp, y, *first[1:])
    assert all(torch.equal(x, z) for x, z in zip(grads, want))


@pytest.mark.parametrize("M,K,N", [(868, 8192, 10000), (100, 8264, 20000)])
def test_long_sums_in_several_rounds(native, M, K, N):
    # from 128 slices of K on rounds of tiles are paced and odd ones walk K backwards: with the
    # checkpoint's token boxes too (868 tokens: the last tiles' second CTA has none; 100: no second CTA has)
    assert -(-M // 256) * -(-N // 128) > 2 * 76
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 9))
    wp = native.swiglu_pack_weights(w1, w2)
    y, gate, up, scale = native.swiglu_forward_checkpoint(a, wp, N)
    for _ in range(3):
        again = native.swiglu_forward_checkpoint(a, wp, N)
    native.swiglu_check_device_status()
    assert torch.equal(y, native.swiglu_forward_variant(a, wp, N, native.SWIGLU_VARIANT_LARGE_M_PAIR))
    assert all(torch.equal(p, q) for p, q in zip(again, (y, gate, up, scale)))
    rows = torch.tensor([0, 1, M // 2, M - 1])
    at = rows.cuda()
    for w, c, s in ((w1, gate, scale[0]), (w2, up, scale[1])):
        x, step = f64(a[at]) @ f64(w), ref.wide(f64(s[:, at]), N)
        err = K * FP32 * (abs(f64(a[at])) @ abs(f64(w)))
        assert (abs(f64(c[at]) * step - x) <= (0.5 + 127 * 2 * FP32) * step + err).all()


@pytest.mark.parametrize("N", [0, -8, 1 << 31, 1 << 55, 1 << 62, 1 << 70, True])
def test_sizes_that_no_tensor_has(native, N):
    a, w1, w2 = (t.cuda() for t in make_inputs(4, 64, 136, 1))
    wp = native.swiglu_pack_weights(w1, w2)
    for call in (lambda: native.swiglu_forward_checkpoint(a, wp, N),
                 lambda: native.swiglu_forward_checkpoint(a[:0], wp, N)):
        with pytest.raises((ValueError, native.SwigluError)):
            call()
