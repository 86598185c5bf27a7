"""Gradients of the gated MLP on the GPU against the float64 formulas (needs a GB300).

Every element is held to the worst-case bound of the roundings the kernels make
(oracle/backward_ref.py); no other tolerance is used.
"""
import numpy as np
import pytest
import torch

from oracle.backward_ref import (backward_bounds, backward_values, down_backward_bounds,
                                 down_backward_values)
from oracle.swiglu_ref import bf16_bits_to_f64
from swiglu_gated_mlp_gb300.workloads import bf16_bits, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def native(native_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return native_lib


def f64(t):
    return bf16_bits_to_f64(bf16_bits(t.cpu()))


def inputs(M, K, N, seed):
    a, w1, w2 = make_inputs(M, K, N, seed)
    return a, w1, w2, make_inputs(M, N, 8, seed + 1)[0]


def down_inputs(M, N, H, seed):
    y, w3, _ = make_inputs(M, N, H, seed)
    return make_inputs(M, H, 8, seed + 1)[0], w3, y


def assert_within(outs, refs, bounds):
    for i, (o, ref, bound) in enumerate(zip(outs, refs, bounds)):
        d = np.abs(f64(o) - ref)
        worst = np.unravel_index(np.argmax(d / bound), d.shape)
        assert (d <= bound).all(), (i, worst, d[worst], bound[worst], ref[worst])


# one token, fewer than a row group, a ragged last tile, one and several output
# tiles, sums in one part and in many, K and N from 8 up
SHAPES = [
    (1, 8, 8), (1, 200, 264), (2, 896, 1000), (31, 64, 128), (33, 72, 136), (128, 896, 1024),
    (127, 256, 512), (130, 1000, 520), (256, 512, 256), (257, 264, 392), (300, 200, 264),
    (513, 1416, 1000), (1025, 128, 256), (64, 2048, 4864), (2000, 72, 72),
]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_backward_matches_the_formula(native, M, K, N):
    a, w1, w2, dy = inputs(M, K, N, seed=M + K + N)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    outs = native.swiglu_backward(a.cuda(), wp, dy.cuda())
    native.swiglu_check_device_status()
    args = [f64(t) for t in (a, w1, w2, dy)]
    assert_within(outs, backward_values(*args), backward_bounds(*args))


@pytest.mark.parametrize("M,N,H", SHAPES)
def test_down_backward_matches_the_formula(native, M, N, H):
    dout, w3, y = down_inputs(M, N, H, seed=M + N + H)
    w3p = native.swiglu_pack_down_weights(w3.cuda())
    outs = native.swiglu_down_backward(dout.cuda(), w3p, y.cuda())
    native.swiglu_check_device_status()
    args = [f64(t) for t in (dout, w3, y)]
    assert_within(outs, down_backward_values(*args), down_backward_bounds(*args))


def sampled(n, count, seed):
    rng = np.random.default_rng(seed)
    return np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, count)]))


@pytest.mark.parametrize("M,K,N", [(128, 896, 4864), (4096, 3584, 18944)])
def test_backward_at_the_workload_shapes(native, M, K, N):
    # dA on sampled rows (all of N), dW on sampled columns (all tokens)
    a, w1, w2, dy = inputs(M, K, N, seed=5)
    dev = [t.cuda() for t in (a, w1, w2, dy)]
    da, dw1, dw2 = native.swiglu_backward(dev[0], native.swiglu_pack_weights(dev[1], dev[2]), dev[3])
    native.swiglu_check_device_status()
    rows, cols = sampled(M, 20, 1), sampled(N, 20, 2)
    ar, dyr = f64(a)[rows], f64(dy)[rows]
    args = (ar, f64(w1), f64(w2), dyr)
    assert_within([da[torch.from_numpy(rows).cuda()]], [backward_values(*args)[0]],
                  [backward_bounds(*args)[0]])
    at = torch.from_numpy(cols).cuda()
    args = (f64(a), f64(w1)[:, cols], f64(w2)[:, cols], f64(dy)[:, cols])
    assert_within([dw1[:, at], dw2[:, at]], backward_values(*args)[1:], backward_bounds(*args)[1:])


def test_down_backward_at_the_workload_shape(native):
    M, N, H = 4096, 18944, 3584
    dout, w3, y = down_inputs(M, N, H, seed=6)
    dy, dw3 = native.swiglu_down_backward(dout.cuda(), native.swiglu_pack_down_weights(w3.cuda()),
                                          y.cuda())
    native.swiglu_check_device_status()
    rows, cols = sampled(M, 20, 1), sampled(H, 20, 2)
    args = (f64(dout)[rows], f64(w3), f64(y)[rows])
    assert_within([dy[torch.from_numpy(rows).cuda()]], [down_backward_values(*args)[0]],
                  [down_backward_bounds(*args)[0]])
    args = (f64(dout)[:, cols], f64(w3)[:, cols], f64(y))
    assert_within([dw3[:, torch.from_numpy(cols).cuda()]], [down_backward_values(*args)[1]],
                  [down_backward_bounds(*args)[1]])


def test_backward_matches_differences_of_the_forward(native):
    # central differences of sum(dY * Y) in float64, at sampled entries. Their own error is
    # about h^2 |Y'''| = 1e-8; the kernel's is its bound.
    M, K, N, h = 9, 72, 136, 1e-4
    a, w1, w2, dy = inputs(M, K, N, seed=3)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    outs = [f64(t) for t in native.swiglu_backward(a.cuda(), wp, dy.cuda())]
    args = [f64(t) for t in (a, w1, w2)]
    d = f64(dy)

    def loss(x, p, q):
        g = x @ p
        return float((g / (1 + np.exp(-g)) * (x @ q) * d).sum())

    rng = np.random.default_rng(0)
    for which, bound in enumerate(backward_bounds(*args, d)):
        for _ in range(40):
            at = tuple(rng.integers(0, n) for n in args[which].shape)
            vals = []
            for sign in (1, -1):
                moved = [x.copy() for x in args]
                moved[which][at] += sign * h
                vals.append(loss(*moved))
            assert abs((vals[0] - vals[1]) / (2 * h) - outs[which][at]) <= bound[at] + 1e-6


def test_backward_parts_asked_for(native):
    M, K, N = 130, 256, 392
    a, w1, w2, dy = (t.cuda() for t in inputs(M, K, N, seed=4))
    wp = native.swiglu_pack_weights(w1, w2)
    full = native.swiglu_backward(a, wp, dy)
    only_a = native.swiglu_backward(a, wp, dy, need_weight=False)
    only_w = native.swiglu_backward(a, wp, dy, need_input=False)
    assert only_a[1] is None and only_a[2] is None and only_w[0] is None
    assert torch.equal(only_a[0], full[0])
    assert torch.equal(only_w[1], full[1]) and torch.equal(only_w[2], full[2])
    assert native.swiglu_backward(a, wp, dy, need_input=False, need_weight=False) == (None,) * 3
    y = make_inputs(M, N, 8, 1)[0].cuda()
    w3p = native.swiglu_pack_down_weights(make_inputs(1, N, K, 2)[1].cuda())
    dout = a
    dy_full, dw_full = native.swiglu_down_backward(dout, w3p, y)
    assert torch.equal(native.swiglu_down_backward(dout, w3p, None, N=N, need_weight=False)[0], dy_full)
    assert torch.equal(native.swiglu_down_backward(dout, None, y, need_input=False)[1], dw_full)
    native.swiglu_check_device_status()


def test_backward_of_no_tokens_is_zero(native):
    K, N = 64, 128
    _, w1, w2 = make_inputs(1, K, N, 0)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    none_a = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    none_y = torch.empty(0, N, dtype=torch.bfloat16, device="cuda")
    dw = [torch.full((K, N), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    da, dw1, dw2 = native.swiglu_backward(none_a, wp, none_y, dW1=dw[0], dW2=dw[1])
    assert da.shape == (0, K) and not dw1.any() and not dw2.any()
    w3p = native.swiglu_pack_down_weights(make_inputs(1, N, K, 2)[1].cuda())
    dw3 = torch.full((N, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    dy, dw3 = native.swiglu_down_backward(none_a, w3p, none_y, dW3=dw3)
    assert dy.shape == (0, N) and not dw3.any()


@pytest.mark.parametrize("M,K,N", [(37, 136, 200), (300, 264, 392), (128, 896, 4864)])
def test_backward_writes_its_outputs_and_nothing_else(native, M, K, N):
    # outputs in the middle of larger buffers of a sentinel, every element written
    a, w1, w2, dy = (t.cuda() for t in inputs(M, K, N, seed=8))
    wp = native.swiglu_pack_weights(w1, w2)
    pad, bufs, views = 4096, [], []
    for shape in ((M, K), (K, N), (K, N)):
        b = torch.empty(shape[0] * shape[1] + 2 * pad, dtype=torch.bfloat16, device="cuda")
        b.view(torch.int16).fill_(0x7FBF)
        bufs.append(b)
        views.append(b[pad:-pad].view(shape))
    n = native.swiglu_backward_workspace_bytes(M, K, N)
    ws = torch.full((n + 2048,), 0xA5, dtype=torch.uint8, device="cuda")
    want = native.swiglu_backward(a, wp, dy)
    native.swiglu_backward(a, wp, dy, *views, workspace=ws[1024:1024 + n])
    native.swiglu_check_device_status()
    for b, v, w in zip(bufs, views, want):
        assert torch.equal(v, w)
        assert (b[:pad].view(torch.int16) == 0x7FBF).all() and (b[-pad:].view(torch.int16) == 0x7FBF).all()
    assert (ws[:1024] == 0xA5).all() and (ws[-1024:] == 0xA5).all()


def test_backward_repeats_bit_for_bit_on_other_streams(native):
    M, K, N = 200, 512, 1000
    a, w1, w2, dy = (t.cuda() for t in inputs(M, K, N, seed=9))
    wp = native.swiglu_pack_weights(w1, w2)
    want = native.swiglu_backward(a, wp, dy)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):  # interleaved calls, workspaces of their own
        got.append(native.swiglu_backward(a, wp, dy, stream=streams[i % 2]))
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_backward_extreme_gates(native):
    # gates up to +-240: SiLU' saturates, nothing overflows or turns to NaN
    M, K, N = 64, 64, 128
    a = torch.eye(64).repeat(1, 1).to(torch.bfloat16) * 16
    g = torch.linspace(-15, 15, K * N).reshape(K, N)
    w1, w2 = g.to(torch.bfloat16), make_inputs(1, K, N, 0)[2]
    dy = make_inputs(M, N, 8, 1)[0]
    outs = native.swiglu_backward(a.cuda(), native.swiglu_pack_weights(w1.cuda(), w2.cuda()), dy.cuda())
    args = [f64(t) for t in (a, w1, w2, dy)]
    # the fast exponential's relative error grows with |G|: |G| 2^-21 <= 2^-13, the same in dG and dU
    bounds = [b + 2.0 ** -13 * s for b, s in zip(backward_bounds(*args), _term_sums(*args))]
    assert_within(outs, backward_values(*args), bounds)


def _term_sums(a, w1, w2, dy):
    g = a @ w1
    x = np.abs(dy) * (1 + np.abs(g) + np.abs(a @ w2))
    return x @ np.abs(w1).T + x @ np.abs(w2).T, np.abs(a).T @ x, np.abs(a).T @ x


def test_backward_keeps_a_bad_token_to_itself(native):
    # a NaN in one token's dY reaches that row of dA (and the weight sums), no other row
    M, K, N = 300, 128, 256
    a, w1, w2, dy = inputs(M, K, N, seed=11)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    want = native.swiglu_backward(a.cuda(), wp, dy.cuda(), need_weight=False)[0]
    dy[17, 3] = float("nan")
    da, dw1, _ = native.swiglu_backward(a.cuda(), wp, dy.cuda())
    keep = torch.ones(M, dtype=torch.bool)
    keep[17] = False
    assert torch.equal(da.cpu()[keep], want.cpu()[keep]) and da[17].isnan().all()
    assert dw1[:, 3].isnan().all() and not dw1[:, 4:].isnan().any()


def test_backward_stalled_wait_is_reported(native):
    M, K, N = 128, 256, 256
    a, w1, w2, dy = (t.cuda() for t in inputs(M, K, N, seed=12))
    wp = native.swiglu_pack_weights(w1, w2)
    want = native.swiglu_backward(a, wp, dy)
    native.swiglu_check_device_status()
    native.swiglu_testing_inject_stall(True, timeout_ms=200)
    try:
        native.swiglu_backward(a, wp, dy)
        with pytest.raises(native.SwigluError) as err:
            native.swiglu_check_device_status()
        assert err.value.code == native.SWIGLU_ERR_TIMEOUT
    finally:
        native.swiglu_testing_inject_stall(False, timeout_ms=1000)
    assert all(torch.equal(x, y) for x, y in zip(native.swiglu_backward(a, wp, dy), want))


def test_backward_workspace_too_small_is_rejected(native):
    M, K, N = 128, 256, 256
    a, w1, w2, dy = (t.cuda() for t in inputs(M, K, N, seed=13))
    wp = native.swiglu_pack_weights(w1, w2)
    n = native.swiglu_backward_workspace_bytes(M, K, N)
    with pytest.raises(native.SwigluError) as err:
        native.swiglu_backward(a, wp, dy, workspace=torch.empty(n - 16, dtype=torch.uint8, device="cuda"))
    assert err.value.code == native.SWIGLU_ERR_INVALID_ARG


def test_binding_refuses_what_does_not_fit(native):
    a, w1, w2, dy = (t.cuda() for t in inputs(20, 64, 128, seed=14))
    wp = native.swiglu_pack_weights(w1, w2)
    w3p = native.swiglu_pack_down_weights(w2.t().contiguous())
    bad = [
        lambda: native.swiglu_backward(a.float(), wp, dy), lambda: native.swiglu_backward(a, wp, dy.cpu()),
        lambda: native.swiglu_backward(a[:, :32], wp, dy), lambda: native.swiglu_backward(a, wp, dy[:10]),
        lambda: native.swiglu_backward(a, wp[:100], dy), lambda: native.swiglu_backward(a, wp, dy.t()),
        lambda: native.swiglu_backward(a, wp, dy, dA=dy), lambda: native.swiglu_backward(a, wp, dy, dW1=w1.t()),
        lambda: native.swiglu_backward(a, wp, dy, workspace=torch.empty(1 << 22, dtype=torch.uint8)),
        lambda: native.swiglu_down_backward(a, w3p, dy[:10]), lambda: native.swiglu_down_backward(a, None, dy),
        lambda: native.swiglu_down_backward(a, w3p, None),
        lambda: native.swiglu_down_backward(a, w3p, None, need_weight=False),
        lambda: native.swiglu_down_backward(a, w3p, dy, N=64), lambda: native.swiglu_down_backward(a, w3p[:9], dy),
        lambda: native.swiglu_down_backward(a, w3p, dy.half()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


def _fields(plan):
    return {k: int(v) for k, _, v in (f.partition("=") for f in plan.split()) if v.isdigit()}


def test_plans_reach_every_form(native):
    # the tested shapes take sums in one part and in several, whole and half tiles of dG and
    # dU, and pairs that begin with weight tiles
    plans = [native.swiglu_backward_plan_string(*s) for s in SHAPES]
    assert all(p.startswith("backward grad whole=") for p in plans)
    parts = [[int(v) for v in p.replace("=", " ").split() if v.isdigit()] for p in plans]
    wholes, halves, _, in_parts, _, w_parts, early, _ = zip(*parts)
    assert max(in_parts) > 1 and min(in_parts) == 1 and max(w_parts) > 1 and min(w_parts) == 1
    assert max(halves) > 0 and max(early) > 0
    big = native.swiglu_backward_plan_string(4096, 3584, 18944)
    f = _fields(big)
    assert f["whole"] > 0 and f["early"] > 0 and f["pairs"] > 1, big
    assert max(wholes) > 0 or f["whole"] > 0
    assert native.swiglu_down_backward_plan_string(128, 4864, 896).startswith("down_backward input tiles=")
    assert native.swiglu_down_backward_workspace_bytes(4096, 18944, 3584) == 0


def _repeated(block, rows):
    """`block`'s rows repeated down to `rows` of them, on the GPU."""
    return block.cuda().repeat(-(-rows // block.shape[0]), 1)[:rows]


def _few_rows(block, M):
    """Tokens at both ends and in the middle of M, and a [M, cols] that is zero but for theirs."""
    rows = torch.cat([torch.arange(260), torch.tensor([(1 << 30) - 1, 1 << 30]), torch.arange(M - 260, M)])
    out = torch.zeros(M, block.shape[1], dtype=torch.bfloat16, device="cuda")
    out[rows.cuda()] = block[rows % block.shape[0]].cuda()
    return rows, out


def test_backward_largest_m(native):
    # 2^31 - 1 tokens, the largest M the ABI accepts: A repeats a block of rows, dY is zero but
    # for some tokens, whose sum the weight gradients are (about 172 GB on the device)
    M, K, N, blk = (1 << 31) - 1, 8, 8, 4096
    a, w1, w2, dy = inputs(blk, K, N, seed=74)
    ad = dyd = outs = None
    try:
        ad = _repeated(a, M)
        rows, dyd = _few_rows(dy, M)
        outs = native.swiglu_backward(ad, native.swiglu_pack_weights(w1.cuda(), w2.cuda()), dyd)
        native.swiglu_check_device_status()
        args = (f64(a[rows % blk]), f64(w1), f64(w2), f64(dy[rows % blk]))
        assert_within([outs[0][rows.cuda()], *outs[1:]], backward_values(*args), backward_bounds(*args))
    finally:
        ad = dyd = outs = None
        torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [(1 << 31) - 1, (1 << 31) - 15])
def test_down_backward_largest_m(native, M):
    # dOut is zero but for some tokens, Y repeats a block of rows (about 103 GB on the device)
    N, H, blk = 8, 8, 4096
    dout, w3, y = down_inputs(blk, N, H, seed=75)
    dod = yd = outs = None
    try:
        yd = _repeated(y, M)
        rows, dod = _few_rows(dout, M)
        outs = native.swiglu_down_backward(dod, native.swiglu_pack_down_weights(w3.cuda()), yd)
        native.swiglu_check_device_status()
        args = (f64(dout[rows % blk]), f64(w3), f64(y[rows % blk]))
        assert_within([outs[0][rows.cuda()], outs[1]], down_backward_values(*args), down_backward_bounds(*args))
    finally:
        dod = yd = outs = None
        torch.cuda.empty_cache()
