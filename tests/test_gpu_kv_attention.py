"""kv_attention on the GPU against the 64-bit definition over the same codes.

Error bound, by the arithmetic: the logits' operands are exact apart from the
query rows, carried to within 2^-18 of the row's largest element, and their
fp32 sums (128 terms); so a logit is off by at most
    d = scale * 2^-17 * max|q| * max_j sum_d |k_j[d]| + 2^-20 (1 + |lse|).
The weights carry at least 8 significant bits (2^-9) and fp32 sums, and out is
rounded to bf16 (2^-8 of its value): for W = sum_j p_j |v_j|
    |out - ref| <= 2^-8 * |ref| + (2^-9 + 2^-12 + 2 d) * W,   |lse - ref| <= d.
"""
import math
import random

import pytest
import torch

import kv_reference as ref
from gpu_helpers import cuda_or_skip
from nvfp4_mixture_experts_top_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _poison(codes, exps, table, kv):
    """NaN codes in every slot that no request holds, the NaN exponent in pages that none holds."""
    S = codes.shape[2]
    held = torch.zeros(codes.shape[0], S, dtype=torch.bool)
    for b, n in enumerate(kv):
        for j in range(-(-n // S)):
            held[int(table[b, j]), :min(S, n - j * S)] = True
    held = held.to(codes.device)
    codes.transpose(1, 2)[~held] = 0x7F
    exps[~held.any(1)] = 255


def _case(ctx, new, Hq, Hkv, D, S, seed, dev, spread=1.0, sharp=2.0):
    kv = [c + n for c, n in zip(ctx, new)]
    table, P = ref.make_tables(kv, S, seed, dev, junk=1 << 30)
    kc, ke = ref.make_cache(P, Hkv, S, D, seed + 1, dev, spread)
    vc, ve = ref.make_cache(P, Hkv, S, D, seed + 2, dev, spread)
    _poison(kc, ke, table, kv)
    _poison(vc, ve, table, kv)
    T = sum(new)
    g = torch.Generator(device=dev).manual_seed(seed)
    q = (torch.randn(T, Hq + 3, D, generator=g, device=dev) * sharp).to(torch.bfloat16)[:, :Hq]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return q, kc, ke, vc, ve, table, kv, start


def _check(case, scale=None, max_q=None, ws=None):
    q, kc, ke, vc, ve, table, kv, start = case
    dev = q.device
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    n = max([b - a for a, b in zip(start, start[1:])], default=0)
    out, lse = B.kv_attention(q, kc, ke, vc, ve, table, _i32(kv, dev), _i32(start, dev), n if max_q is None else max_q,
                              scale, want_lse=True, dev_status=st)
    o, z, W, slack = ref.attention(q, kc, ke, vc, ve, table, kv, start, scale)
    assert int(st.item()) == 0
    empty = torch.isinf(z)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert int((out[empty] != 0).sum()) == 0
    d = abs(scale) * 2.0 ** -17 * q.double().abs().amax(-1) * slack + 2.0 ** -20 * (1 + z.abs().masked_fill(empty, 0))
    err = (lse.double() - z).abs().masked_fill(empty, 0)
    assert bool((err <= d).all()), "lse off by %.3g of its bound" % float((err / d).max())
    bound = 2.0 ** -8 * o.abs() + (2.0 ** -9 + 2.0 ** -12 + 2 * d[..., None]) * W
    err = (out.double() - o).abs()
    assert bool((err <= bound).all()), "out off by %.3g of its bound" % float((err / bound.clamp(min=1e-300)).max())
    return out, lse


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,S", [
    ([0], [1], 1, 1, 64, 16),                               # one key
    ([332], [1], 32, 8, 128, 64),
    ([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129], [1] * 11, 8, 1, 128, 16),
    ([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129], [1] * 11, 5, 5, 64, 128),
    ([4095, 3, 2000, 700], [1] * 4, 12, 4, 128, 64),        # ragged, group 3
    ([1000, 37], [1, 1], 48, 8, 128, 32),                   # group 6
    ([250, 1, 999], [1] * 3, 16, 1, 64, 16),                # group 16
    ([250, 1, 999], [1] * 3, 71, 1, 128, 64),               # group 71: more than one row tile
    ([30000], [1], 8, 2, 128, 64),                          # one request over the whole GPU
    ([0, 5, 300, 64], [5, 2, 3, 7], 16, 4, 64, 16),         # drafted tokens
    ([31, 500], [16, 9], 7, 1, 128, 32),
])
def test_few_queries(ctx, new, Hq, Hkv, D, S):
    dev = cuda_or_skip()
    _check(_case(ctx, new, Hq, Hkv, D, S, 7, dev))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,S", [
    ([0], [128], 1, 1, 128, 64), ([0], [129], 2, 1, 64, 16), ([1], [257], 4, 2, 128, 128),
    ([300, 0], [211, 97], 6, 2, 128, 32), ([1000], [1000], 8, 1, 64, 64), ([5, 0, 77], [400, 1, 63], 5, 1, 128, 16),
    ([2048], [640], 8, 2, 128, 64), ([63, 64, 65], [65, 64, 63], 9, 3, 128, 64),
])
def test_prompts(ctx, new, Hq, Hkv, D, S):
    dev = cuda_or_skip()
    _check(_case(ctx, new, Hq, Hkv, D, S, 11, dev))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,S", [
    ([0], [1500], 7, 1, 128, 64), ([0, 600, 0], [900, 30, 1], 6, 2, 64, 16), ([100], [333], 71, 1, 64, 32),
    ([0, 0, 0], [300, 301, 302], 24, 2, 128, 16), ([1, 2500, 9], [700, 2, 17], 20, 4, 128, 128),
])
def test_prompts_cut_between_row_tiles_of_growing_length(ctx, new, Hq, Hkv, D, S):
    dev = cuda_or_skip()
    _check(_case(ctx, new, Hq, Hkv, D, S, 13, dev))


def test_prompts_next_to_single_tokens_and_absent_requests():
    dev = cuda_or_skip()
    ctx, new = [700, 0, 33, 5000, 0, 12, 64], [1, 300, 0, 1, 1, 40, 1]
    for D, S in ((128, 64), (64, 16)):
        _check(_case(ctx, new, 8, 2, D, S, 13, dev))


@pytest.mark.parametrize("new", [1, 3, 200])
def test_rows_without_keys(new):
    """No cached token, or more queries than keys: rows that see nothing give 0 and -inf."""
    dev = cuda_or_skip()
    q, kc, ke, vc, ve, table, kv, start = _case([5, 40, 0, 9], [new] * 4, 8, 2, 128, 16, 17, dev)
    kv = [0, new // 2, 0, kv[3]]
    _check((q, kc, ke, vc, ve, table, kv, start))


@pytest.mark.parametrize("new", [1, 6, 150])
@pytest.mark.parametrize("spread", [8.0, 20.0])
def test_blocks_of_very_different_scale(new, spread):
    """Values: the error stays relative to the largest value block of the request.  Keys: logits up to the
    thousands, so one key takes all."""
    dev = cuda_or_skip()
    q, kc, ke, vc, ve, table, kv, start = _case([700, 90], [new] * 2, 8, 2, 128, 16, 19, dev, spread=0.0)
    g = torch.Generator(device=dev).manual_seed(3)
    ve.copy_((ve.int() + (spread * torch.randn(ve.shape, generator=g, device=dev)).round().int()).clamp(10, 240))
    args = (q, kc, ke, vc, ve, table, _i32(kv, dev), _i32(start, dev), new)
    out = B.kv_attention(*args)
    o, z, W, slack = ref.attention(*args[:6], kv, start, 128 ** -0.5)
    d = 128 ** -0.5 * 2.0 ** -17 * q.double().abs().amax(-1) * slack + 2.0 ** -20 * (1 + z.abs())
    for b in range(2):
        t = slice(start[b], start[b + 1])
        pages = table[b, :-(-kv[b] // 16)].long()
        top = (448 * ref.two(ve[pages].long() - 127)).amax(0).repeat_interleave(4)  # largest value a head can hold
        bound = 2.0 ** -8 * o[t].abs() + (2.0 ** -9 + 2.0 ** -12 + 2 * d[t][..., None]) * W[t] + \
            2.0 ** -24 * top[None, :, None]
        assert bool(((out[t].double() - o[t]).abs() <= bound).all())
    ke.copy_((ke.int() + 6).clamp(max=240))
    q2 = (q.float() * 30).to(torch.bfloat16)
    out, lse = B.kv_attention(q2, *args[1:], want_lse=True)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())


def test_query_values_that_are_not_finite_stay_in_their_row():
    dev = cuda_or_skip()
    for new in (2, 130):
        case = _case([50, 300], [new, new], 8, 2, 128, 16, 23, dev)
        base, _ = _check(case)
        q = case[0].clone()
        q[1, 3, 5], q[new, 7, 0] = float("nan"), float("inf")
        out = B.kv_attention(q, *case[1:5], case[5], _i32(case[6], dev), _i32(case[7], dev), new)
        assert bool(torch.isnan(out[1, 3]).all()) and not bool(torch.isfinite(out[new, 7]).any())
        keep = torch.ones(q.shape[:2], dtype=torch.bool, device=dev)
        keep[1, 3] = keep[new, 7] = False
        assert torch.equal(out[keep], base[keep])


def test_query_rows_of_any_magnitude():
    dev = cuda_or_skip()
    for new in (1, 140):
        case = _case([200], [new], 4, 2, 128, 16, 29, dev)
        q = case[0].float()
        for mag in (2.0 ** -100, 2.0 ** 60):
            q2 = (q * mag).to(torch.bfloat16)
            _check((q2,) + case[1:], scale=128 ** -0.5 / mag)
        q2 = q.clone()
        q2[:, :, 3] *= 300  # one large channel
        _check((q2.to(torch.bfloat16),) + case[1:], scale=128 ** -0.5 / 100)
        q2[:] = 0
        _check((q2.to(torch.bfloat16),) + case[1:])


def test_scale_zero_and_negative():
    dev = cuda_or_skip()
    for new in (1, 135):
        case = _case([333], [new], 4, 2, 64, 16, 31, dev)
        _check(case, scale=0.0)
        _check(case, scale=-0.3)


def test_bounds_of_the_query_length_are_only_a_hint():
    dev = cuda_or_skip()
    case = _case([90, 300], [70, 1], 8, 2, 128, 16, 37, dev)
    for n in (0, 1, 70, 5000):
        _check(case, max_q=n)


def test_repeats_bit_for_bit_and_on_another_stream():
    dev = cuda_or_skip()
    for ctx, new in (([9000, 20], [1, 1]), ([700, 3000], [120, 200])):
        case = _case(ctx, new, 8, 2, 128, 64, 41, dev)
        args = case[:6] + (_i32(case[6], dev), _i32(case[7], dev), max(new))
        out = B.kv_attention(*args)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = [B.kv_attention(*args) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(s)
        for a in again:
            assert torch.equal(a, out)


def test_other_requests_do_not_matter():
    """A request alone and among others: the same result up to where partial sums are joined (2^-8 of the weight)."""
    dev = cuda_or_skip()
    case = _case([3000, 100, 800], [1, 1, 1], 8, 2, 128, 64, 43, dev)
    all3, _ = _check(case)
    q, kc, ke, vc, ve, table, kv, start = case
    for b in range(3):
        one, _ = _check((q[b:b + 1], kc, ke, vc, ve, table[b:b + 1], kv[b:b + 1], [0, 1]))
        _, _, W, _ = ref.attention(q[b:b + 1], kc, ke, vc, ve, table[b:b + 1], kv[b:b + 1], [0, 1], 128 ** -0.5)
        assert bool(((one.double() - all3[b:b + 1].double()).abs() <= 2.0 ** -8 * W).all())


def test_bad_pages_and_lengths_are_reported():
    """A page outside the cache counts as keys that are not there; a length past the table is cut."""
    dev = cuda_or_skip()
    for new in (1, 150):
        q, kc, ke, vc, ve, table, kv, start = _case([300, 200], [new, new], 8, 2, 128, 16, 47, dev)
        for bad in (-1, kc.shape[0], 1 << 30):
            t2 = table.clone()
            t2[0, 0] = bad
            st = torch.zeros(1, dtype=torch.int32, device=dev)
            out = B.kv_attention(q, kc, ke, vc, ve, t2, _i32(kv, dev), _i32(start, dev), new, dev_status=st)
            assert int(st.item()) == 10
            # the definition without the first page's keys
            o, _, W, _ = ref.attention(q[:new], kc, ke, vc, ve, table[:1, 1:], [kv[0] - 16], [0, new], 128 ** -0.5)
            assert bool(((out[:new].double() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -7 * W).all())
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        M = table.shape[1]
        full = table.clone().clamp(max=kc.shape[0] - 1)
        B.kv_attention(q, kc, ke, vc, ve, full, _i32([16 * M + 5, -7], dev), _i32(start, dev), new, dev_status=st)
        assert int(st.item()) == 10
        st.zero_()
        out = B.kv_attention(q, kc, ke, vc, ve, table, _i32(kv, dev), _i32([0, new, 2 * new + 50], dev), new,
                             dev_status=st)
        assert int(st.item()) == 10


def test_rows_of_no_request_are_not_written():
    dev = cuda_or_skip()
    for new in (1, 100):
        q, kc, ke, vc, ve, table, kv, start = _case([300, 200], [new, new], 8, 2, 64, 16, 53, dev)
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=dev)
        B.kv_attention(q, kc, ke, vc, ve, table[:1], _i32(kv[:1], dev), _i32(start[:2], dev), new, out=out)
        assert bool((out[new:] == 7).all()) and not bool((out[:new] == 7).all())


def test_past_32_bit_offsets():
    dev = cuda_or_skip()
    Hkv, D, S = 8, 128, 128
    P = (1 << 31) // (Hkv * D * S) + 40
    small = [ref.make_cache(40, Hkv, S, D, 3 + i, dev) for i in (0, 1)]
    big = []
    for c, e in small:
        C = torch.full((P, Hkv, S, D), 0x7F, dtype=torch.uint8, device=dev)
        E = torch.full((P, Hkv), 255, dtype=torch.uint8, device=dev)
        C[P - 40:], E[P - 40:] = c, e
        big += [C, E]
    g = torch.Generator(device=dev).manual_seed(1)
    for new in (1, 140):
        kv = [4000]
        table = torch.arange(39, 39 - 32, -1, dtype=torch.int32, device=dev)[None]
        q = torch.randn(new, 16, D, generator=g, device=dev).to(torch.bfloat16)
        out = B.kv_attention(q, *big, table + (P - 40), _i32(kv, dev), _i32([0, new], dev), new)
        same = B.kv_attention(q, *small[0], *small[1], table, _i32(kv, dev), _i32([0, new], dev), new)
        assert torch.equal(out, same)
        _check((q, *small[0], *small[1], table, kv, [0, new]))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,S", [
    ([3000 + 137 * i for i in range(24)], [1] * 24, 16, 8, 128, 64),
    ([70000, 300, 41000], [1, 1, 1], 8, 8, 128, 16),
    ([2000 + 311 * i for i in range(20)], [1 + i % 3 for i in range(20)], 24, 8, 64, 32),
    ([2000 + 311 * i for i in range(20)], [1 + i % 3 for i in range(20)], 24, 8, 128, 128),
])
def test_whole_gpu_many_times_over(ctx, new, Hq, Hkv, D, S):
    """Every CTA streams its share through its buffers many times, in calls that follow one another at once."""
    dev = cuda_or_skip()
    case = _case(ctx, new, Hq, Hkv, D, S, 61, dev)
    out, lse = _check(case)
    args = case[:6] + (_i32(case[6], dev), _i32(case[7], dev), max(new))
    ws = torch.empty(B.kv_attention_workspace_bytes(out.shape[0], len(ctx), Hq, Hkv, D), dtype=torch.uint8, device=dev)
    again = [B.kv_attention(*args, workspace=ws, want_lse=True) for _ in range(50)]
    for o, z in again:
        assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("seed", range(12))
def test_random_mixes(seed):
    dev = cuda_or_skip()
    r = random.Random(seed)
    n = r.randint(1, 9)
    D, S = r.choice((64, 128)), r.choice((16, 32, 64, 128))
    Hkv = r.choice((1, 2, 3, 8))
    Hq = Hkv * r.randint(1, 9)
    ctx = [int(math.exp(r.uniform(0, 8))) - 1 for _ in range(n)]
    top = r.choice((1, 4, 40, 300))
    new = [r.randint(0, top) for _ in range(n)]
    new[0] = max(new[0], 1)
    _check(_case(ctx, new, Hq, Hkv, D, S, 100 + seed, dev))


def test_no_tokens():
    dev = cuda_or_skip()
    q, kc, ke, vc, ve, table, kv, start = _case([20], [1], 4, 2, 64, 16, 59, dev)
    out = B.kv_attention(q[:0], kc, ke, vc, ve, table, _i32(kv, dev), _i32([0, 0], dev), 0)
    assert out.shape == (0, 4, 64)
    empty = torch.empty(0, 4, dtype=torch.int32, device=dev)
    out = B.kv_attention(q, kc, ke, vc, ve, empty, _i32([], dev), _i32([0], dev), 1)
    assert out.shape == (1, 4, 64)
