"""kv_plan and kv_append on the GPU against 64-bit / integer restatements.
Everything is compared exactly: both are integer or correctly rounded work."""
import random

import pytest
import torch

import kv_reference as ref
from gpu_helpers import cuda_or_skip
from nvfp4_mixture_experts_top_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _plan_case(seed, n, S, hi, new_hi, dev):
    r = random.Random(seed)
    ctx = [r.randint(0, hi) for _ in range(n)]
    new = [r.choice((0, 1, 1, r.randint(0, new_hi))) for _ in range(n)]
    table, P = ref.make_tables(ctx, S, seed, dev, width=max(1, -(-(hi + new_hi) // S)))
    used = set(table.flatten().tolist())
    free = [p for p in range(P + 40) if p not in used]
    r.shuffle(free)
    return ctx, new, table, free


def _run_plan(ctx, new, table, free, n_free, S, T, dev):
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    got = B.kv_plan(_i32(ctx, dev), _i32(new, dev), table, _i32(free, dev), _i32([n_free], dev), S, T, dev_status=st)
    return got, int(st.item())


@pytest.mark.parametrize("n,S,hi,new_hi", [(1, 16, 0, 1), (1, 64, 64, 1), (16, 64, 4096, 1), (33, 16, 100, 40),
                                           (511, 32, 300, 7), (700, 128, 1000, 300), (2000, 16, 50, 3)])
def test_plan_matches_the_restatement(n, S, hi, new_hi):
    dev = cuda_or_skip()
    ctx, new, table, free = _plan_case(n + S, n, S, hi, new_hi, dev)
    need = sum(-(-(c + m) // S) - -(-c // S) for c, m in zip(ctx, new))
    free = free + list(range(10 ** 6, 10 ** 6 + max(0, need - len(free) + 3)))
    T = sum(new) + 5  # five entries past the last token
    want = ref.plan(ctx, new, table.tolist(), free, len(free), S, T)
    for _ in range(2):  # the call can be repeated on its own result
        got, st = _run_plan(ctx, new, table, free, len(free), S, T, dev)
        assert table.tolist() == want[0]
        assert got["query_start"].tolist() == want[1] and got["kv_lens"].tolist() == want[2]
        assert got["slot_map"].tolist() == want[3] and got["free_left"].tolist() == [want[4]]
        assert st == 0


@pytest.mark.parametrize("n_free", [0, 1, 7, 20])
def test_plan_without_enough_pages(n_free):
    """Requests that do not fit keep their lengths and get no slot; the rest is served."""
    dev = cuda_or_skip()
    S = 16
    ctx, new, table, free = _plan_case(5, 40, S, 90, 30, dev)
    free = (free + list(range(10 ** 6, 10 ** 6 + 50)))[:50]
    T = sum(new)
    want = ref.plan(ctx, new, table.tolist(), free, n_free, S, T)
    got, st = _run_plan(ctx, new, table, free, n_free, S, T, dev)
    assert table.tolist() == want[0] and got["slot_map"].tolist() == want[3]
    assert got["kv_lens"].tolist() == want[2] and got["free_left"].tolist() == [want[4]]
    assert st == (9 if -1 in want[3] else 0)


def test_plan_table_too_narrow():
    dev = cuda_or_skip()
    table = _i32([[3, 4], [5, -1]], dev)
    got, st = _run_plan([32, 16], [1, 16], table, [9, 8, 7], 3, 16, 17, dev)
    assert got["kv_lens"].tolist() == [32, 32] and st == 9
    assert got["slot_map"].tolist() == [-1] + [8 * 16 + i for i in range(16)]  # the first request's page stays asked for
    assert table.tolist() == [[3, 4], [5, 8]] and got["free_left"].tolist() == [2]


def test_plan_bad_lengths_are_reported():
    dev = cuda_or_skip()
    for ctx, new in (([-3, 5], [1, 1]), ([0, 5], [-1, 1]), ([0, 5], [9, 1])):
        table = _i32([[0, 1], [2, 3]], dev)
        got, st = _run_plan(ctx, new, table, [7, 6], 2, 16, 2, dev)
        assert st == 10
        assert got["query_start"].tolist() == [0, 0, 1] and got["kv_lens"].tolist() == [0, 6]
        assert got["slot_map"].tolist() == [2 * 16 + 5, -1]


def test_plan_more_tokens_than_slots():
    dev = cuda_or_skip()
    table = _i32([[0], [1]], dev)
    got, st = _run_plan([0, 0], [3, 3], table, [5, 4], 2, 16, 4, dev)
    assert st == 10 and got["slot_map"].tolist() == [64, 65, 66, 80] and got["query_start"].tolist() == [0, 3, 6]


def test_plan_no_requests():
    dev = cuda_or_skip()
    got, st = _run_plan([], [], torch.empty(0, 4, dtype=torch.int32, device=dev), [5, 4], 2, 16, 3, dev)
    assert st == 0 and got["query_start"].tolist() == [0] and got["free_left"].tolist() == [2]
    assert got["slot_map"].tolist() == [-1] * 3


def _append_case(lens, new, Hkv, D, S, dtype, seed, dev):
    table, P = ref.make_tables([c + n for c, n in zip(lens, new)], S, seed, dev)
    g = torch.Generator(device=dev).manual_seed(seed)
    T = sum(new)
    x = torch.randn(T, 1 + 2 * Hkv, D, generator=g, device=dev) * torch.exp2(
        4 * torch.randn(T, 1, 1, generator=g, device=dev))
    x = x.to(dtype)
    slots = [int(table[b, p // S]) * S + p % S for b, (c, n) in enumerate(zip(lens, new)) for p in range(c, c + n)]
    return x[:, 1:1 + Hkv], x[:, 1 + Hkv:], slots, P


def _same_cache(got, want):
    """Equal codes (any NaN code for a NaN) and equal exponents."""
    nan = (want[0] & 127) == 127
    assert torch.equal((got[0] & 127) == 127, nan)
    assert torch.equal(got[0][~nan], want[0][~nan])
    assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,new,Hkv,D,S", [
    ([0], [1], 1, 64, 16), ([63, 64, 65, 0, 127], [1, 1, 1, 1, 1], 8, 128, 64), ([5, 0, 16], [40, 33, 1], 3, 64, 16),
    ([100, 1], [300, 0], 2, 128, 128), ([7] * 70, [1, 2, 0, 3, 1] * 14, 4, 128, 32), ([31, 15], [500, 1000], 8, 128, 64)])
def test_append_matches_the_restatement(dtype, lens, new, Hkv, D, S):
    dev = cuda_or_skip()
    k, v, slots, P = _append_case(lens, new, Hkv, D, S, dtype, len(lens) + D, dev)
    halves = [ref.make_cache(P, Hkv, S, D, 3 + i, dev, spread=4) for i in (0, 1)]
    want = [(c.clone(), e.clone()) for c, e in halves]
    for x, (c, e) in zip((k, v), want):
        ref.append(x.double(), slots, c, e)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    for _ in range(2):  # appending the same rows again changes nothing
        B.kv_append(k, v, _i32(slots, dev), *halves[0], *halves[1], dev_status=st)
        for g, w in zip(halves, want):
            _same_cache(g, w)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,new,Hkv,D,S", [
    ([0, 77, 3], [900, 1, 1200], 8, 128, 128), ([65, 0, 1], [700, 700, 70], 8, 64, 128),
    ([9, 0], [1000, 333], 8, 64, 16), ([0] * 9 + [40], [1] * 9 + [1500], 8, 128, 64), ([50], [2500], 4, 64, 32),
    ([200 + i for i in range(1300)], [1] * 1300, 4, 64, 16)])
def test_append_many_tokens(dtype, lens, new, Hkv, D, S):
    """Chunks of many tokens per CTA: runs that pass a chunk's end, whole pages, next to single tokens."""
    dev = cuda_or_skip()
    k, v, slots, P = _append_case(lens, new, Hkv, D, S, dtype, S + D, dev)
    halves = [ref.make_cache(P, Hkv, S, D, 3 + i, dev, spread=4) for i in (0, 1)]
    want = [(c.clone(), e.clone()) for c, e in halves]
    for x, (c, e) in zip((k, v), want):
        ref.append(x.double(), slots, c, e)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    B.kv_append(k, v, _i32(slots, dev), *halves[0], *halves[1], dev_status=st)
    for g, w in zip(halves, want):
        _same_cache(g, w)
    assert int(st.item()) == 0


def test_append_special_values():
    """Zeros, subnormals, infinities, NaN, the largest finite value, and 448 * 2^e exactly."""
    dev = cuda_or_skip()
    Hkv, D, S = 1, 64, 16
    rows = [[0.0], [-0.0], [1e-40], [3.4028234663852886e38], [float("inf"), -1.0], [float("nan"), 2.0], [448.0], [449.0],
            [448.0 * 2 ** 20], [447.9999 * 2.0 ** -60], [1.0, float("-inf")], [2.0 ** -118 * 1.75], [2.0 ** -119]]
    x = torch.zeros(len(rows), Hkv, D, device=dev)
    for i, r in enumerate(rows):
        x[i, 0, :len(r)] = torch.tensor(r)
    slots = [S * i for i in range(len(rows))]  # a fresh block each
    halves = [ref.make_cache(len(rows), Hkv, S, D, 3 + i, dev) for i in (0, 1)]
    want = [(c.clone(), e.clone()) for c, e in halves]
    for c, e in want:
        ref.append(x.double(), slots, c, e)
    B.kv_append(x, x, _i32(slots, dev), *halves[0], *halves[1])
    for g, w in zip(halves, want):
        _same_cache(g, w)


def test_append_moves_old_codes_to_a_larger_scale():
    dev = cuda_or_skip()
    Hkv, D, S = 2, 128, 64
    for jump in (1, 3, 9, 30, 200):
        halves = [ref.make_cache(1, Hkv, S, D, 3 + i, dev) for i in (0, 1)]
        for c, e in halves:
            e.fill_(20)  # 2^-107
        x = torch.full((1, Hkv, D), 300.0 * 2.0 ** -107, device=dev) * 2.0 ** min(jump, 100) * 2.0 ** max(0, jump - 100)
        want = [(c.clone(), e.clone()) for c, e in halves]
        for c, e in want:
            ref.append(x.double(), [37], c, e)
        B.kv_append(x, x, _i32([37], dev), *halves[0], *halves[1])
        for g, w in zip(halves, want):
            _same_cache(g, w)
            assert int(g[1][0, 0]) == 20 + jump


def test_append_skips_and_reports():
    """Negative slots are skipped; a slot past the cache is skipped and reported."""
    dev = cuda_or_skip()
    Hkv, D, S, P = 2, 64, 16, 4
    x = torch.randn(5, Hkv, D, device=dev)
    slots = [3, -1, 20, P * S, 40]
    halves = [ref.make_cache(P, Hkv, S, D, 3 + i, dev) for i in (0, 1)]
    want = [(c.clone(), e.clone()) for c, e in halves]
    for c, e in want:
        ref.append(x[[0, 2, 4]].double(), [3, 20, 40], c, e)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    B.kv_append(x, x, _i32(slots, dev), *halves[0], *halves[1], dev_status=st)
    for g, w in zip(halves, want):
        _same_cache(g, w)
    assert int(st.item()) == 10


def test_append_on_another_stream_and_past_32_bit_offsets():
    """A cache half of more than 2^31 bytes: its last pages are written where they belong."""
    dev = cuda_or_skip()
    Hkv, D, S = 8, 128, 128
    P = (1 << 31) // (Hkv * D * S) + 9
    codes = [torch.zeros(P, Hkv, S, D, dtype=torch.uint8, device=dev) for _ in (0, 1)]
    exps = [torch.zeros(P, Hkv, dtype=torch.uint8, device=dev) for _ in (0, 1)]
    x = torch.randn(3, Hkv, D, device=dev)
    slots = [(P - 1) * S + 126, (P - 1) * S + 127, (P - 3) * S]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sl = _i32(slots, dev)
    with torch.cuda.stream(s):
        B.kv_append(x, x, sl, codes[0], exps[0], codes[1], exps[1])
    torch.cuda.current_stream().wait_stream(s)
    small = torch.zeros(4, Hkv, S, D, dtype=torch.uint8, device=dev), torch.zeros(4, Hkv, dtype=torch.uint8, device=dev)
    ref.append(x.double(), [v - (P - 4) * S for v in slots], *small)
    for c, e in zip(codes, exps):
        assert torch.equal(c[P - 4:], small[0]) and torch.equal(e[P - 4:], small[1])
        assert int(c[:9].max()) == 0 and int(e[:P - 4].max()) == 0
