"""Plain 64-bit restatements of kv_plan, kv_append, kv_attention and
block_norm for the parity tests, and the builders of their inputs.  Nothing
here is shared with the library; E4M3 is decoded from its bit fields."""
import math

import numpy as np
import torch

# E4M3 FN by its fields: sign, 4 exponent bits (bias 7), 3 fraction bits
_E4M3 = np.array([(-1.0 if c & 128 else 1.0) * ((c & 7) / 8 * 2.0 ** -6 if (c >> 3) & 15 == 0 else
                                                (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7)) for c in range(256)])
_E4M3[[127, 255]] = np.nan


def e4m3_values(codes):
    t = torch.from_numpy(_E4M3).to(codes.device)
    return t[codes.long()]


def two(e):
    """2^e as float64, exactly."""
    t = torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device=e.device)
    return t[e.long() + 300]


def e4m3_codes(x):
    """Nearest E4M3 code of float64 x, ties to even, saturating; NaN -> 0x7F."""
    grid = torch.from_numpy(_E4M3[:127]).to(x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = x.abs().nan_to_num(nan=0.0)
    i = torch.searchsorted(mid, a)
    up = (i < 126) & (a == mid[i.clamp(max=125)]) & (i % 2 == 1)
    i = (i + up.long()).to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 7)
    return torch.where(torch.isnan(x), torch.full_like(i, 0x7F), i)


def plan(ctx, new, table, free, n_free, S, T):
    """kv_plan with Python integers; returns (table, query_start, kv, slots, free_left)."""
    table = [list(r) for r in table]
    start, kv, slots = [0], [], []
    asked = taken = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        held, want = -(-c // S), -(-(c + n) // S)
        need = want - held
        fits = (need == 0 or asked + need <= n_free) and want <= len(table[b])
        if fits:
            for j in range(need):
                table[b][held + j] = free[n_free - 1 - (asked + j)]
            taken += need
        asked += need
        kv.append(c + n if fits else c)
        slots += [table[b][p // S] * S + p % S if fits else -1 for p in range(c, c + n)]
        start.append(start[-1] + n)
    slots = (slots + [-1] * T)[:T]
    return table, start, kv, slots, n_free - taken


def append(x, slots, codes, exps):
    """kv_append on one half: x [T, Hkv, D] float64, codes and exps updated in place."""
    S = codes.shape[2]
    slots = [int(s) for s in slots]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        u = t + 1
        while u < len(slots) and slots[u] == slots[u - 1] + 1 and slots[u] % S:
            u += 1
        p, o = slots[t] // S, slots[t] % S
        rows = x[t:u]
        top = rows.abs().nan_to_num(nan=0.0, posinf=3.4028234663852886e38).amax((0, 2))
        e = torch.tensor([-127 if v == 0 else max(-127, math.frexp(v / 448)[1] - (math.frexp(v / 448)[0] == 0.5))
                          for v in top.tolist()], device=x.device)
        if o:
            old = exps[p].long() - 127
            grow = e > old
            moved = e4m3_codes(e4m3_values(codes[p, :, :o]) * two(old - e)[:, None, None])
            codes[p, :, :o] = torch.where(grow[:, None, None], moved, codes[p, :, :o])
            e = torch.maximum(e, old)
        codes[p, :, o:o + u - t] = e4m3_codes(rows.transpose(0, 1) * two(-e)[:, None, None])
        exps[p] = (e + 127).to(torch.uint8)
        t = u


def attention(q, kc, ke, vc, ve, table, kv, start, scale):
    """float64 (out, lse, weight, slack): weight = sum p |v| for every output,
    slack = largest sum_d |k_d| of the keys a row sees, for error bounds."""
    T, Hq, D = q.shape
    Hkv, S = kc.shape[1], kc.shape[2]
    dev = q.device
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=dev)
    wgt, slack = torch.zeros_like(out), torch.zeros(T, Hq, dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    for b in range(len(kv)):
        L, t0, t1 = int(kv[b]), int(start[b]), int(start[b + 1])
        if t1 == t0 or L == 0:
            continue
        pages = table[b, :-(-L // S)].long()

        def rows(c, e):
            x = e4m3_values(c[pages]) * two(e[pages].long() - 127)[..., None, None]
            return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :L].repeat_interleave(Hq // Hkv, 0)

        k, v = rows(kc, ke), rows(vc, ve)
        s = torch.einsum("thd,hkd->htk", q[t0:t1].double(), k) * scale
        limit = L - (t1 - t0) + 1 + torch.arange(t1 - t0, device=dev)
        seen = torch.arange(L, device=dev)[None, :] < limit[:, None]
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        z = torch.logsumexp(s, -1)
        p = torch.where(seen & (limit > 0)[:, None], torch.exp(s - z[..., None]), torch.zeros_like(s))
        o = torch.einsum("htk,hkd->thd", p, v)
        out[t0:t1] = o
        wgt[t0:t1] = torch.einsum("htk,hkd->thd", p, v.abs())
        lse[t0:t1] = z.T
        ks = torch.cummax(k.abs().sum(-1), -1).values  # [Hq, L]
        slack[t0:t1] = ks[:, (limit - 1).clamp(min=0)].T
    return out, lse, wgt, slack


def norm(x, a, gate, w_post, w_pre, alpha, eps):
    y = x.double()
    if a is not None:
        u = a.double()
        if w_post is not None:
            u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + eps) * w_post.double()
        y = y + alpha * (u if gate is None else u * gate.double())
    h = None
    if w_pre is not None:
        h = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w_pre.double()
    return y, h


def make_cache(P, Hkv, S, D, seed, dev, spread=1.0):
    """Random codes with block exponents about 1 (spread: width of the exponents, in powers of two)."""
    g = torch.Generator(device=dev).manual_seed(seed)
    codes = e4m3_codes((torch.randn(P, Hkv, S, D, generator=g, device=dev) * 64).double())
    exps = (121 + spread * torch.randn(P, Hkv, generator=g, device=dev)).round().clamp(1, 250).to(torch.uint8)
    return codes, exps


def make_tables(lens, S, seed, dev, spare=2, width=None, junk=-1):
    """A table of distinct random pages for lens cached tokens; junk behind each row's pages.  Returns (table, P)."""
    need = [-(-n // S) for n in lens]
    P = sum(need) + spare
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(P, generator=g).to(torch.int32).tolist()
    M = width or max(1, max(need, default=1))
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [junk] * (M - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32, device=dev).view(len(lens), M), P
