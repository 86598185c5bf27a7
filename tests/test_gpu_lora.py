"""Projections with low-rank adapters on the GPU against float64 (needs a GB300).

Every element is held to the worst-case bound of the roundings the kernels make
(oracle/lora_ref.py); no other tolerance is used.
"""
import numpy as np
import pytest
import torch

from oracle.lora_ref import down_forward_lora, forward_lora
from oracle.swiglu_ref import bf16_bits_to_f64
from swiglu_gated_mlp_gb300.workloads import bf16_bits, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def native(native_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return native_lib


def f64(t):
    if t.dtype == torch.bfloat16:
        return bf16_bits_to_f64(bf16_bits(t.cpu()))
    return t.cpu().double().numpy()


def table(L, halves, r, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (L, 2) if halves == 2 else (L,)
    la = (torch.randn(*shape, r, K, generator=g) / K ** 0.5).to(torch.bfloat16)
    lb = (torch.randn(*shape, N, r, generator=g) / r ** 0.5).to(torch.bfloat16)
    return la, lb, 0.5 + torch.rand(L, generator=g)


def indices(M, L, how, seed):
    g = torch.Generator().manual_seed(seed + 99)
    if how == "mixed":    # a request a token, none among them
        return torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)
    if how == "one":
        return torch.full((M,), L - 1, dtype=torch.int32)
    if how == "none":     # outside the table on both sides
        return torch.where(torch.arange(M) % 2 == 0, -1, L).to(torch.int32)
    runs = torch.randint(-1, L, (6,), generator=g, dtype=torch.int32)  # prompts
    return runs[(torch.arange(M) * 6) // M]


def assert_within(out, ref_bound):
    ref, bound = ref_bound
    d = np.abs(f64(out) - ref)
    worst = np.unravel_index(np.argmax(d / bound), d.shape)
    assert (d <= bound).all(), (worst, d[worst], bound[worst], ref[worst])


def run_gate_up(native, M, K, N, L, r, how, seed):
    a, w1, w2 = make_inputs(M, K, N, seed)
    la, lb, scale = table(L, 2, r, K, N, seed)
    index = indices(M, L, how, seed)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    y = native.swiglu_forward_lora(a.cuda(), wp, N, la.cuda(), lb.cuda(), index.cuda(), scale.cuda())
    native.swiglu_check_device_status()
    assert_within(y, forward_lora(*(f64(t) for t in (a, w1, w2, la, lb)), index.numpy(), f64(scale)))


def run_down(native, M, N, H, L, r, how, seed, residual=True):
    y, w3, _ = make_inputs(M, N, H, seed)
    res = make_inputs(M, H, 8, seed + 1)[0] if residual else None
    la, lb, scale = table(L, 1, r, N, H, seed)
    index = indices(M, L, how, seed)
    w3p = native.swiglu_pack_down_weights(w3.cuda())
    out = native.swiglu_down_forward_lora(y.cuda(), w3p, H, la.cuda(), lb.cuda(), index.cuda(),
                                          scale.cuda(), R=res.cuda() if residual else None)
    native.swiglu_check_device_status()
    assert_within(out, down_forward_lora(f64(y), f64(w3), f64(res) if residual else None, f64(la), f64(lb),
                                         index.numpy(), f64(scale)))


# single tokens, K split over clusters and not, several token groups, ragged
# columns and K; then one and several 256-token tiles, with one adapter, runs of
# prompts, a different one each token (many passes and slices), and none
SHAPES = [
    (1, 8, 8, 1, 8, "one"), (1, 896, 4864, 4, 8, "one"), (1, 200, 264, 3, 64, "none"),
    (2, 72, 136, 2, 24, "mixed"), (7, 1000, 520, 5, 16, "mixed"), (16, 896, 1000, 8, 16, "mixed"),
    (17, 264, 20000, 8, 8, "mixed"), (33, 512, 1032, 40, 40, "mixed"), (64, 256, 392, 3, 64, "runs"),
    (65, 1416, 1000, 20, 24, "mixed"), (100, 200, 264, 1, 56, "one"), (128, 896, 4864, 32, 16, "mixed"),
    (128, 64, 20000, 4, 64, "runs"),
    (129, 200, 264, 2, 8, "runs"), (130, 8, 8, 1, 8, "one"), (256, 512, 1000, 5, 16, "runs"),
    (257, 1000, 520, 3, 24, "mixed"), (300, 264, 392, 300, 8, "mixed"), (513, 1416, 1000, 20, 40, "mixed"),
    (700, 128, 136, 6, 64, "none"), (1025, 896, 520, 4, 64, "runs"), (2000, 72, 72, 2, 56, "one"),
]


@pytest.mark.parametrize("M,K,N,L,r,how", SHAPES)
def test_forward_lora_matches_the_formula(native, M, K, N, L, r, how):
    run_gate_up(native, M, K, N, L, r, how, seed=M + K + N + r)


@pytest.mark.parametrize("M,N,H,L,r,how", SHAPES)
def test_down_forward_lora_matches_the_formula(native, M, N, H, L, r, how):
    run_down(native, M, N, H, L, r, how, seed=M + N + H + r, residual=M % 2 == 0)


# a few tokens: every decode CTA makes V itself
@pytest.mark.parametrize("M,K,N,L,r,how", [
    (1, 64, 8, 2, 8, "mixed"), (1, 896, 4864, 3, 16, "one"), (2, 1016, 264, 2, 8, "one"),
    (1, 3584, 19000, 2, 32, "one"), (4, 2056, 19464, 3, 8, "mixed"), (3, 1032, 20000, 9, 16, "mixed"),
    (5, 2504, 19464, 5, 8, "none"), (16, 1000, 19464, 5, 8, "runs"),
])
@pytest.mark.parametrize("down", [False, True])
def test_tokens_whose_v_every_cta_makes(native, M, K, N, L, r, how, down):
    plan = (native.swiglu_down_lora_plan_string if down else native.swiglu_lora_plan_string)(M, K, N, r)
    assert "shrink inside" in plan or M == 16 or K == 1032, plan
    if down:
        run_down(native, M, K, N, L, r, how, seed=M + K + r, residual=M % 2 == 1)
    else:
        run_gate_up(native, M, K, N, L, r, how, seed=M + K + r)


def rows_of(M, count, seed):
    rng = np.random.default_rng(seed)
    return np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, count)]))


@pytest.mark.parametrize("M,L,r,how", [(16, 8, 16, "mixed"), (4096, 8, 64, "runs")])
def test_forward_lora_at_the_7b_shape(native, M, L, r, how):
    K, N = 3584, 18944
    a, w1, w2 = make_inputs(M, K, N, 3)
    la, lb, scale = table(L, 2, r, K, N, 3)
    index = indices(M, L, how, 3)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    y = native.swiglu_forward_lora(a.cuda(), wp, N, la.cuda(), lb.cuda(), index.cuda(), scale.cuda())
    native.swiglu_check_device_status()
    rows = rows_of(M, 24, 0)
    at = torch.from_numpy(rows)
    assert_within(y[at.cuda()], forward_lora(f64(a)[rows], f64(w1), f64(w2), f64(la), f64(lb),
                                             index.numpy()[rows], f64(scale)))


@pytest.mark.parametrize("M", [5, 300])
def test_adapters_of_no_token_and_an_empty_table(native, M):
    K, N = 264, 392
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 1))
    wp = native.swiglu_pack_weights(w1, w2)
    la, lb, scale = (t.cuda() for t in table(3, 2, 16, K, N, 1))
    none = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    # no token has an adapter: the table's values do not matter
    y = native.swiglu_forward_lora(a, wp, N, la * float("nan"), lb * float("nan"), none, scale)
    ref = forward_lora(f64(a), f64(w1), f64(w2), f64(la), f64(lb), none.cpu().numpy(), f64(scale))
    assert_within(y, ref)
    empty = native.swiglu_forward_lora(a, wp, N, la[:0], lb[:0], none, scale[:0])
    assert torch.equal(empty, native.swiglu_forward(a, wp, N))
    w3p = native.swiglu_pack_down_weights(w1)
    assert torch.equal(native.swiglu_down_forward_lora(a, w3p, N, la[:0, 0], lb[:0, 0], none, scale[:0]),
                       native.swiglu_down_forward(a, w3p, N))
    native.swiglu_check_device_status()


@pytest.mark.parametrize("M", [24, 300])
def test_another_adapters_values_do_not_reach_a_token(native, M):
    # adapter 1 holds a NaN in La and an infinite scale: only its own tokens see it
    K, N = 200, 264
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 2))
    wp = native.swiglu_pack_weights(w1, w2)
    la, lb, scale = (t.cuda() for t in table(3, 2, 16, K, N, 2))
    index = (torch.arange(M, dtype=torch.int32, device="cuda") * 7) % 4 - 1
    want = native.swiglu_forward_lora(a, wp, N, la, lb, index, scale)
    la[1, :, 3, 5] = float("nan")
    scale[1] = float("inf")
    got = native.swiglu_forward_lora(a, wp, N, la, lb, index, scale)
    native.swiglu_check_device_status()
    theirs = index != 1
    assert torch.equal(got[theirs], want[theirs])
    assert not got[~theirs].isfinite().any()


@pytest.mark.parametrize("M", [9, 300])
def test_down_lora_in_place_residual(native, M):
    N, H = 264, 520
    y, w3, _ = (t.cuda() for t in make_inputs(M, N, H, 4))
    res = make_inputs(M, H, 8, 5)[0].cuda()
    la, lb, scale = (t.cuda() for t in table(3, 1, 8, N, H, 4))
    index = indices(M, 3, "mixed", 4).cuda()
    w3p = native.swiglu_pack_down_weights(w3)
    want = native.swiglu_down_forward_lora(y, w3p, H, la, lb, index, scale, R=res)
    got = native.swiglu_down_forward_lora(y, w3p, H, la, lb, index, scale, R=res, Out=res)
    assert got is res and torch.equal(got, want)


@pytest.mark.parametrize("M,K,N,L,r", [(3, 136, 200, 2, 8), (128, 896, 1000, 9, 24), (300, 264, 392, 5, 40)])
def test_lora_writes_its_output_and_nothing_else(native, M, K, N, L, r):
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 6))
    wp = native.swiglu_pack_weights(w1, w2)
    la, lb, scale = (t.cuda() for t in table(L, 2, r, K, N, 6))
    index = indices(M, L, "mixed", 6).cuda()
    pad = 4096
    buf = torch.empty(M * N + 2 * pad, dtype=torch.bfloat16, device="cuda")
    buf.view(torch.int16).fill_(0x7FBF)
    n = native.swiglu_lora_workspace_bytes(M, K, N, r)
    ws = torch.full((n + 2048,), 0xA5, dtype=torch.uint8, device="cuda")
    y = native.swiglu_forward_lora(a, wp, N, la, lb, index, scale, Y=buf[pad:-pad].view(M, N),
                                   workspace=ws[1024:1024 + n])
    native.swiglu_check_device_status()
    assert torch.equal(y, native.swiglu_forward_lora(a, wp, N, la, lb, index, scale))
    for edge in (buf[:pad], buf[-pad:]):
        assert (edge.view(torch.int16) == 0x7FBF).all()
    assert (ws[:1024] == 0xA5).all() and (ws[-1024:] == 0xA5).all()


@pytest.mark.parametrize("M", [1, 16, 100, 300])
def test_back_to_back_calls_see_what_was_written_before_them(native, M):
    # the projection starts while V is made: tokens, weights, index and table that the
    # kernel just before the call wrote, with no synchronisation, on two streams
    K, N, L, r = 896, 4864, 4, 16
    base = [t.cuda() for t in make_inputs(M, K, N, 7)]
    la, lb, scale = (t.cuda() for t in table(L, 2, r, K, N, 7))
    index = indices(M, L, "mixed", 7).cuda()
    wp = native.swiglu_pack_weights(base[1], base[2])
    want = [native.swiglu_forward_lora(base[0] * f, wp, N, la * f, lb, index, scale) for f in (1.0, -2.0)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, stream in enumerate(streams):
        with torch.cuda.stream(stream):
            a, ta = torch.zeros_like(base[0]), torch.zeros_like(la)
            ws = native.swiglu_lora_workspace(M, K, N, r)
            wq = torch.zeros_like(wp)
            for i in range(10):
                f = (1.0, -2.0)[i % 2]
                torch.mul(base[0], f, out=a)
                torch.mul(la, f, out=ta)
                wq.copy_(wp)
                got.append((i % 2, native.swiglu_forward_lora(a, wq, N, ta, lb, index, scale, workspace=ws)))
                a.fill_(float("nan"))   # the next write may not pass the call either
                wq.fill_(float("nan"))
    torch.cuda.synchronize()
    native.swiglu_check_device_status()
    for which, y in got:
        assert torch.equal(y, want[which])


@pytest.mark.parametrize("M", [16, 300])
def test_lora_in_a_captured_graph_with_new_requests(native, M):
    K, N, L, r = 264, 520, 5, 16
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 8))
    wp = native.swiglu_pack_weights(w1, w2)
    la, lb, scale = (t.cuda() for t in table(L, 2, r, K, N, 8))
    index = indices(M, L, "one", 8).cuda()
    ws, y = native.swiglu_lora_workspace(M, K, N, r), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    native.swiglu_forward_lora(a, wp, N, la, lb, index, scale, Y=y, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        native.swiglu_forward_lora(a, wp, N, la, lb, index, scale, Y=y, workspace=ws)
    for how in ("mixed", "runs", "none", "one"):
        index.copy_(indices(M, L, how, 8))
        want = native.swiglu_forward_lora(a, wp, N, la, lb, index, scale)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), how


@pytest.mark.parametrize("M,K,N", [(100, 264, 392), (300, 896, 4864), (700, 1416, 20000)])
def test_lora_repeats_bit_for_bit(native, M, K, N):
    # many adapters in every tile, in a different order each time they are met
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 11))
    wp = native.swiglu_pack_weights(w1, w2)
    la, lb, scale = (t.cuda() for t in table(20, 2, 16, K, N, 11))
    index = indices(M, 20, "mixed", 11).cuda()
    want = native.swiglu_forward_lora(a, wp, N, la, lb, index, scale)
    for _ in range(8):
        assert torch.equal(native.swiglu_forward_lora(a, wp, N, la, lb, index, scale), want)


@pytest.mark.parametrize("M", [16, 300])
def test_lora_stalled_wait_is_reported(native, M):
    K, N, L, r = 512, 520, 3, 16
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 9))
    wp = native.swiglu_pack_weights(w1, w2)
    la, lb, scale = (t.cuda() for t in table(L, 2, r, K, N, 9))
    index = indices(M, L, "mixed", 9).cuda()
    want = native.swiglu_forward_lora(a, wp, N, la, lb, index, scale)
    native.swiglu_check_device_status()
    native.swiglu_testing_inject_stall(True, timeout_ms=200)
    try:
        native.swiglu_forward_lora(a, wp, N, la, lb, index, scale)
        with pytest.raises(native.SwigluError) as err:
            native.swiglu_check_device_status()
        assert err.value.code == native.SWIGLU_ERR_TIMEOUT
    finally:
        native.swiglu_testing_inject_stall(False, timeout_ms=1000)
    assert torch.equal(native.swiglu_forward_lora(a, wp, N, la, lb, index, scale), want)


def test_large_table_offsets(native):
    # an adapter whose La and Lb lie past 2^31 values of the table
    M, K, N, L, r = 3, 8192, 8192, 2100, 64
    a, w1, w2 = make_inputs(M, K, N, 10)
    la = torch.zeros(L, 2, r, K, dtype=torch.bfloat16, device="cuda")
    lb = torch.zeros(L, 2, N, r, dtype=torch.bfloat16, device="cuda")
    assert la[:-1].numel() > 1 << 31 and lb[:-1].numel() > 1 << 31
    last = table(1, 2, r, K, N, 10)
    la[-1], lb[-1] = last[0][0].cuda(), last[1][0].cuda()
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    for m in (M, 130):
        am = a.repeat(-(-m // M), 1)[:m]
        index = torch.full((m,), L - 1, dtype=torch.int32)
        y = native.swiglu_forward_lora(am.cuda(), wp, N, la, lb, index.cuda(),
                                       last[2].repeat(L).cuda())
        native.swiglu_check_device_status()
        ref = forward_lora(f64(a), f64(w1), f64(w2), f64(last[0]), f64(last[1]), np.zeros(M, int), f64(last[2]))
        assert_within(y[:M], ref)
        if m > M:
            assert torch.equal(y[m - 1], y[(m - 1) % M])


def test_binding_refuses_what_does_not_fit(native):
    M, K, N, L, r = 20, 64, 128, 3, 8
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 15))
    wp, w3p = native.swiglu_pack_weights(w1, w2), native.swiglu_pack_down_weights(w1)
    la, lb, scale = (t.cuda() for t in table(L, 2, r, K, N, 15))
    index = indices(M, L, "mixed", 15).cuda()
    good = dict(A=a, Wpacked=wp, N=N, La=la, Lb=lb, index=index, scale=scale)
    down = dict(Y=a, W3packed=w3p, H=N, La=la[:, 0].contiguous(), Lb=lb[:, 0].contiguous(), index=index,
                scale=scale)
    native.swiglu_forward_lora(**good)
    native.swiglu_down_forward_lora(**down)
    bad = [dict(A=a.float()), dict(A=a.cpu()), dict(A=a[:, :32]), dict(Wpacked=wp[:64]), dict(N=136),
           dict(La=la[:, :1]), dict(La=la[..., :32].contiguous()), dict(La=la[0]), dict(Lb=lb[:2]),
           dict(Lb=lb.transpose(2, 3)), dict(index=index.long()), dict(index=index[:5]), dict(index=index.cpu()),
           dict(scale=scale.half()), dict(scale=scale[:2]), dict(scale=scale.cpu()),
           dict(Y=torch.empty(M, K, dtype=torch.bfloat16, device="cuda")),
           dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))]
    for change in bad:
        with pytest.raises(ValueError):
            native.swiglu_forward_lora(**{**good, **change})
            pytest.fail(f"not refused: {list(change)}")
    for change in (dict(Y=a.half()), dict(W3packed=w3p[:9]), dict(H=256), dict(La=la), dict(R=a),
                   dict(index=index[::2]), dict(Out=a.float())):
        with pytest.raises(ValueError):
            native.swiglu_down_forward_lora(**{**down, **change})
            pytest.fail(f"not refused: {list(change)}")
    # a rank that is no multiple of 8 is a matter of the library
    with pytest.raises(native.SwigluError) as err:
        native.swiglu_forward_lora(**{**good, "La": la[:, :, :4].contiguous(), "Lb": lb[..., :4].contiguous()})
    assert err.value.code == native.SWIGLU_ERR_UNSUPPORTED


def test_plans_reach_every_form(native):
    # the tested shapes take both kernels, one and several token groups, K in one and several parts
    plans = [native.swiglu_lora_plan_string(M, K, N, r) for M, K, N, _, r, _ in SHAPES]
    assert any("large_m_pair" in p for p in plans) and any("groups=1 " in p for p in plans)
    assert any("small_m" in p and "groups=3" in p for p in plans)
    assert any("splits=8" in p for p in plans) and any("splits=1" in p for p in plans)
    assert any("shrink dots" in p for p in plans) and any("shrink tiles" in p for p in plans)
    assert any("shrink inside" in p for p in plans)
    down = [native.swiglu_down_lora_plan_string(M, N, H, r) for M, N, H, _, r, _ in SHAPES]
    assert all(p.startswith("down lora shrink") for p in down)
    assert "large_m_pair" in native.swiglu_lora_plan_string(4096, 3584, 18944, 64)
    assert "small_m mt=16" in native.swiglu_lora_plan_string(16, 3584, 18944, 16)


@pytest.mark.parametrize("rank", [8, 40])
@pytest.mark.parametrize("M, K, N", [
    (3, 712, 20000),    # decode kernel, V made by every CTA (rank 8)
    (24, 200, 264),     # decode kernel, K whole
    (24, 2048, 520),    # K over a cluster, adapters dealt to its CTAs
    (200, 712, 392),    # token groups
    (1200, 200, 1032),  # CTA pairs, ragged last tiles
])
def test_non_finite_lb_stays_with_its_tokens(native, M, K, N, rank):
    # some columns of adapter 1's Lb hold an infinity or NaN: exactly its tokens' outputs
    # there are not finite, every other output keeps its bits
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 2))
    wp = native.swiglu_pack_weights(w1, w2)
    la, lb, scale = (t.cuda() for t in table(3, 2, rank, K, N, 2))
    index = (torch.arange(M, dtype=torch.int32, device="cuda") * 7) % 4 - 1
    theirs = index == 1
    want = native.swiglu_forward_lora(a, wp, N, la, lb, index, scale)
    lb[1, 1, 0, 0] = float("nan")          # up
    lb[1, 1, 70, rank - 1] = float("inf")
    lb[1, 1, N - 1, 3] = float("-inf")
    lb[1, 0, 127, 5] = float("nan")        # gate
    lb[1, 0, 128, :] = float("nan")
    cols = torch.zeros(N, dtype=torch.bool, device="cuda")
    cols[[0, 70, 127, 128, N - 1]] = True
    got = native.swiglu_forward_lora(a, wp, N, la, lb, index, scale)
    native.swiglu_check_device_status()
    hit = theirs[:, None] & cols[None, :]
    assert torch.equal(got[~hit], want[~hit])
    assert not got[hit].isfinite().any()

    w3p = native.swiglu_pack_down_weights(w1)
    res = make_inputs(M, N, 8, 5)[0].cuda()
    la3, lb3, scale3 = (t.cuda() for t in table(3, 1, rank, K, N, 3))
    want = native.swiglu_down_forward_lora(a, w3p, N, la3, lb3, index, scale3, R=res)
    lb3[1, 0, 0] = float("nan")
    lb3[1, 70, rank - 1] = float("inf")
    lb3[1, N - 1, 3] = float("-inf")
    lb3[1, [127, 128], 5] = float("nan")
    got = res.clone()
    native.swiglu_down_forward_lora(a, w3p, N, la3, lb3, index, scale3, R=got, Out=got)
    native.swiglu_check_device_status()
    assert torch.equal(got[~hit], want[~hit])
    assert not got[hit].isfinite().any()
    # one infinity: its sign is that of the token's V, which one more call with a zero
    # weight and a one in its place shows
    only = torch.zeros_like(lb3)
    only[1, 70, rank - 1] = 1.0
    v = native.swiglu_down_forward_lora(a, torch.zeros_like(w3p), N, la3, only, index, scale3)[theirs, 70]
    assert torch.equal(got[theirs, 70], (v.float() * float("inf")).to(torch.bfloat16))


@pytest.mark.parametrize("M, K, N, r, L", [
    (1, 264, 1000, 8, 2), (16, 264, 1000, 16, 5), (100, 512, 2000, 64, 3), (200, 264, 2000, 24, 9),
    (600, 512, 1000, 40, 4),
])
def test_calls_one_after_another_see_each_others_outputs(native, M, K, N, r, L):
    # each call's kernels start while those before it run: what a call reads, the last one
    # wrote; a chain must give the bits that it gives with a synchronisation after each call
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 7))
    w3 = make_inputs(8, N, K, 8)[1].cuda() / 32  # small: the chain must not grow
    wp, w3p = native.swiglu_pack_weights(w1, w2), native.swiglu_pack_down_weights(w3)
    la, lb, scale = (t.cuda() for t in table(L, 2, r, K, N, 7))
    la3, lb3, scale3 = (t.cuda() for t in table(L, 1, r, N, K, 8))
    lb3 = lb3 / 32
    other = [make_inputs(M, K, 8, s)[0].cuda() for s in (11, 12, 13)]  # every step's x differs
    index = indices(M, L, "mixed", 3).cuda()
    ws = native.swiglu_lora_workspace(M, K, N, r)
    ws3 = native.swiglu_down_lora_workspace(M, N, K, r)

    def chain(sync, steps=12):
        x = a.clone()
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        for i in range(steps):
            native.swiglu_forward_lora(x, wp, N, la, lb, index, scale, Y=y, workspace=ws)
            if sync:
                torch.cuda.synchronize()
            native.swiglu_down_forward_lora(y, w3p, K, la3, lb3, index, scale3, R=other[i % 3], Out=x,
                                               workspace=ws3)
            if sync:
                torch.cuda.synchronize()
        return x

    want = chain(True)
    assert want.isfinite().all()
    for _ in range(5):
        assert torch.equal(chain(False), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(False)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    native.swiglu_check_device_status()


@pytest.mark.parametrize("down", [False, True])
def test_lora_largest_m(native, down):
    # 2^31 - 1 tokens, the largest M the ABI accepts: x, index and residual repeat a block of
    # rows, so each sampled row's reference is that of its row in the block (about 155 GB)
    M, K, N, L, r, blk = (1 << 31) - 1, 8, 8, 5, 8, 4096
    a, w1, w2 = make_inputs(blk, K, N, seed=76)
    la, lb, scale = table(L, 1 if down else 2, r, K, N, 76)
    index = indices(blk, L, "mixed", 76)
    res = make_inputs(blk, N, 8, 77)[0] if down else None
    reps = -(-M // blk)
    ad = idx = rd = y = None
    try:
        ad, idx = a.cuda().repeat(reps, 1)[:M], index.cuda().repeat(reps)[:M]
        if down:
            rd = res.cuda().repeat(reps, 1)[:M]
            y = native.swiglu_down_forward_lora(ad, native.swiglu_pack_down_weights(w1.cuda()), N, la.cuda(),
                                                lb.cuda(), idx, scale.cuda(), R=rd, Out=rd)
        else:
            y = native.swiglu_forward_lora(ad, native.swiglu_pack_weights(w1.cuda(), w2.cuda()), N, la.cuda(),
                                           lb.cuda(), idx, scale.cuda())
        native.swiglu_check_device_status()
        rows = np.array([0, 1, blk - 1, blk, (1 << 30) - 1, 1 << 30, M - 257, M - 256, M - 129, M - 2, M - 1])
        at = rows % blk
        got = y[torch.from_numpy(rows).cuda()]
        x, i, s = f64(a)[at], index.numpy()[at], f64(scale)
        assert_within(got, down_forward_lora(x, f64(w1), f64(res)[at], f64(la), f64(lb), i, s) if down else
                      forward_lora(x, f64(w1), f64(w2), f64(la), f64(lb), i, s))
    finally:
        ad = idx = rd = y = None
        torch.cuda.empty_cache()


@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("M, K, N", [(4096, 64, 2000), (700, 1416, 5000)])
def test_pairs_behind_a_kernel_of_many_blocks(native, M, K, N, down):
    # the projection's CTA pairs start while the kernel that makes V, and whatever ran before it,
    # still fill SMs: many calls in a row behind a kernel of thousands of small blocks
    L, r = 3, 16
    plan = (native.swiglu_down_lora_plan_string if down else native.swiglu_lora_plan_string)(M, K, N, r)
    assert "large_m_pair" in plan
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 5))
    la, lb, scale = (t.cuda() for t in table(L, 1 if down else 2, r, K, N, 5))
    index = indices(M, L, "mixed", 5).cuda()
    if down:
        wp, ws = native.swiglu_pack_down_weights(w1), native.swiglu_down_lora_workspace(M, K, N, r)
    else:
        wp, ws = native.swiglu_pack_weights(w1, w2), native.swiglu_lora_workspace(M, K, N, r)
    call = native.swiglu_down_forward_lora if down else native.swiglu_forward_lora
    b, v1, v2 = (t.cuda() for t in make_inputs(2048, 64, 18944, 7))
    kept = native.swiglu_forward_checkpoint(b, native.swiglu_pack_weights(v1, v2), 18944)[1:]
    first = call(a, wp, N, la, lb, index, scale, workspace=ws)
    torch.cuda.synchronize()
    for _ in range(20):
        for _ in range(50):
            native.swiglu_checkpoint_output(*kept)
            last = call(a, wp, N, la, lb, index, scale, workspace=ws)
        torch.cuda.synchronize()
    native.swiglu_check_device_status()
    assert torch.equal(first, last)
