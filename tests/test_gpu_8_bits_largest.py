"""The 8-bit calls at 2^31 - 1 tokens, the largest M the ABI accepts (needs a GB300, up to 250 GB of it).

Inputs repeat a block of rows, so each sampled row's reference is that of its row in the block.
"""
import gc

import numpy as np
import pytest
import torch

from oracle import int8_ref as ref
from oracle.backward_ref import FP32
from swiglu_gated_mlp_gb300.workloads import make_inputs
from test_gpu_int8 import assert_within, codes, f64, native, scales  # noqa: F401

pytestmark = pytest.mark.gpu

M, K, N, BLK = (1 << 31) - 1, 8, 8, 4096
ROWS = np.array([0, 1, BLK - 1, BLK, (1 << 30) - 1, 1 << 30, M - 257, M - 256, M - 193, M - 129, M - 128, M - 2, M - 1])
AT = ROWS % BLK


@pytest.fixture(autouse=True)
def all_memory():
    gc.collect()
    torch.cuda.empty_cache()
    yield
    gc.collect()
    torch.cuda.empty_cache()


def tiled(t):
    """[BLK, ...] as [M, ...]."""
    return t.cuda().repeat(-(-M // BLK), *[1] * (t.dim() - 1))[:M]


def rows(t):
    return t[torch.from_numpy(ROWS).cuda()]


def test_tokens(native):
    x = make_inputs(BLK, K, 8, 1)[0]
    q, s = native.swiglu_quantize_int8(tiled(x))
    want = ref.quantise(f64(x)[AT])
    assert (f64(rows(q)) == want[0]).all() and (f64(rows(s)) == want[1]).all()


@pytest.mark.parametrize("down", [False, True])
def test_projections(native, down):
    g = torch.Generator().manual_seed(1)
    a, w1, w2 = codes(g, BLK, K), codes(g, K, N), codes(g, K, N)
    sa, s1, s2 = scales(g, BLK, 0.02), scales(g, N, 0.01), scales(g, N, 0.01)
    gate = ref.product(f64(a)[AT], f64(sa)[AT], f64(w1), f64(s1))
    if down:
        r = make_inputs(BLK, N, 8, 3)[0]
        rd = tiled(r)
        out = native.swiglu_down_forward_int8(tiled(a), tiled(sa), native.swiglu_pack_down_weights_int8(w1.cuda()), N,
                                              s1.cuda(), R=rd, Out=rd)
        want = ref.added(*gate, f64(r)[AT])
    else:
        out = native.swiglu_forward_int8(tiled(a), tiled(sa), native.swiglu_pack_weights_int8(w1.cuda(), w2.cuda()), N,
                                         s1.cuda(), s2.cuda())
        want = ref.gated(*gate, *ref.product(f64(a)[AT], f64(sa)[AT], f64(w2), f64(s2)))
    native.swiglu_check_device_status()
    assert_within(rows(out), *want)


def test_checkpoint(native):
    a, w1, w2 = make_inputs(BLK, K, N, 2)
    wp = native.swiglu_pack_weights(w1.cuda(), w2.cuda())
    y, gate, up, scale = native.swiglu_forward_checkpoint(tiled(a), wp, N)
    native.swiglu_check_device_status()
    y = None
    dy = native.swiglu_checkpoint_output(gate, up, scale)
    at = torch.from_numpy(ROWS).cuda()
    kept = []
    for w, c, s in ((w1, gate, scale[0]), (w2, up, scale[1])):
        x, step = f64(a)[AT] @ f64(w), ref.wide(f64(s[:, at]), N)
        err = K * FP32 * (abs(f64(a)[AT]) @ abs(f64(w)))
        kept.append(f64(c[at]) * step)
        assert (abs(kept[-1] - x) <= (0.5 + 127 * 2 * FP32) * step + err).all()
    g, u = kept
    assert_within(rows(dy), *ref.gated(g, FP32 * abs(g), u, FP32 * abs(u)))
    q, sa = native.swiglu_quantize_int8(a.cuda())
    da, _, _ = native.swiglu_backward_checkpoint(tiled(q), wp, dy, gate, up, scale, scale_a=tiled(sa), need_weight=False)
    native.swiglu_check_device_status()
    args = (f64(a)[AT], f64(w1), f64(w2), g, u, f64(rows(dy)))
    assert_within(rows(da), ref.backward_values(*args)[0], ref.backward_bounds(*args)[0])
