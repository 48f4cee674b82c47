"""block_norm on the GPU against the 64-bit formula.

Bound: fp32 sums of H <= 16384 squares, one rsqrt and a few products keep y
and h to within 2^-18 of their terms, then one rounding to bf16 (8 significant
bits: 2^-8 of the value)."""
import pytest
import torch

import kv_reference as ref
from gpu_helpers import cuda_or_skip
from nvfp4_mixture_experts_top_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _case(T, H, a, gate, post, pre, seed, dev, pad=0):
    g = torch.Generator(device=dev).manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=g, device=dev)

    x = (rand(T, H + pad) * 2).to(BF)[:, :H]
    av = None if a is None else (rand(T, H + pad) * torch.exp2(3 * rand(T, 1))).to(a)[:, :H]
    shape = dict(none=None, channel=(H,), token=(T, 1), full=(T, H))[gate]
    gt = None if shape is None else rand(*shape).to(BF)
    wp = (1 + 0.2 * rand(H)).to(BF) if post else None
    wq = (1 + 0.2 * rand(H)).to(BF) if pre else None
    return x, av, gt, wp, wq


def _check(x, a, gate, wp, wq, alpha=1.0, eps=1e-6, inplace=False):
    want_y, want_h = ref.norm(x, a, gate, wp, wq, alpha, eps)
    mag = x.double().abs() + (0 if a is None else (want_y - x.double()).abs())
    y, h = B.block_norm(x, a, gate=gate, w_post=wp, w_pre=wq, alpha=alpha, eps=eps, y=x if inplace else None)
    if a is not None:
        assert bool(((y.double() - want_y).abs() <= 2.0 ** -8 * want_y.abs() + 2.0 ** -18 * mag).all())
    if wq is not None:
        r = 1 / torch.sqrt(want_y.square().mean(-1, keepdim=True) + eps)
        assert bool(((h.double() - want_h).abs() <= 2.0 ** -8 * want_h.abs() +
                     2.0 ** -17 * (mag * r * wq.double().abs() + want_h.abs())).all())
    return y, h


@pytest.mark.parametrize("T,H", [(1, 8), (3, 24), (16, 4096), (5, 6144), (2, 8192), (2, 8200), (3, 16384), (300, 1032),
                                 (1000, 256)])
@pytest.mark.parametrize("a", [None, BF, torch.float32])
def test_sizes_and_types(T, H, a):
    dev = cuda_or_skip()
    _check(*_case(T, H, a, "none", a is not None, True, T + H, dev))


@pytest.mark.parametrize("H", [264, 1032, 4096, 4104, 6152, 12288, 12296, 16384])
@pytest.mark.parametrize("a,gate", [(None, "none"), (BF, "channel"), (torch.float32, "full"), (BF, "token")])
def test_many_rows(H, a, gate):
    dev = cuda_or_skip()
    _check(*_case(333, H, a, gate, a is not None, True, H, dev), alpha=0.7)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("T", [1, 37])
def test_gates_and_weights(gate, post, pre, T):
    dev = cuda_or_skip()
    _check(*_case(T, 520, BF, gate, post, pre, 5, dev), alpha=-0.37, eps=1e-3)


@pytest.mark.parametrize("a", [BF, torch.float32])
def test_row_strides(a):
    dev = cuda_or_skip()
    _check(*_case(9, 264, a, "full", True, True, 9, dev, pad=40), alpha=0.5)


def test_residual_in_place():
    dev = cuda_or_skip()
    for T, H in ((4, 4096), (700, 1000)):
        x, a, gate, wp, wq = _case(T, H, torch.float32, "channel", True, True, 3, dev)
        y0, h0 = B.block_norm(x, a, gate=gate, w_post=wp, w_pre=wq)
        y1, h1 = B.block_norm(x, a, gate=gate, w_post=wp, w_pre=wq, y=x)
        assert y1 is x and torch.equal(x, y0) and torch.equal(h0, h1)


def test_zero_large_and_not_finite_rows():
    """A row of zeros, rows whose squares come near fp32's ends, and NaN / Inf that stay in their row."""
    dev = cuda_or_skip()
    x, a, _, wp, wq = _case(6, 512, torch.float32, "none", True, True, 21, dev)
    a[0] = 0
    x[0] = 0
    a[1] *= 1e15
    a[2] *= 1e-15
    y0, h0 = _check(x, a, None, wp, wq)
    assert bool((h0[0] == 0).all())
    x2, a2 = x.clone(), a.clone()
    a2[3, 7] = float("nan")
    x2[4, 9] = float("inf")
    y, h = B.block_norm(x2, a2, w_post=wp, w_pre=wq)
    assert bool(torch.isnan(h[3]).all()) and bool(torch.isnan(h[4, 9]))
    for r in (0, 1, 2, 5):
        assert torch.equal(h[r], h0[r]) and torch.equal(y[r], y0[r])


def test_repeats_bit_for_bit_and_on_another_stream():
    dev = cuda_or_skip()
    x, a, gate, wp, wq = _case(513, 4096, BF, "token", True, True, 2, dev)
    y, h = B.block_norm(x, a, gate=gate, w_post=wp, w_pre=wq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, h2 = B.block_norm(x, a, gate=gate, w_post=wp, w_pre=wq)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2) and torch.equal(h, h2)
