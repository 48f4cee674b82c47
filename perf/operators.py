"""Measured cases of the decoder-block operators: kv_plan, kv_append, kv_attention and block_norm.

A case is one call of one operator at one size.  ``prepare`` makes what a serving program holds before that call, ``run``
makes the call (``own``: through the binding; otherwise in plain 32-bit torch operations), ``exact`` restates it in 64 bits.
Request lengths follow from the case alone, values from the seed.
"""
import math
import random

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the page and slot bookkeeping of one decode step of 16 concurrent requests
        dict(name="plan_decode_16", op="plan", B=16, lo=1, hi=4096, new_hi=1, prompts=0, page=64, mix=1),
        # 509 requests in flight, a few of which bring a whole prompt chunk
        dict(name="plan_mixed_509", op="plan", B=509, lo=0, hi=16384, new_hi=4, prompts=6, page=16, mix=2),
        # the new tokens' K/V of that decode step, one token for each request
        dict(name="append_decode_16", op="append", B=16, lo=1, hi=4096, new_lo=1, new_hi=1, Hkv=8, D=128, page=64,
             dtype="bf16", mix=3),
        # the K/V of prompt chunks of odd lengths
        dict(name="append_prompt_7x1100", op="append", B=7, lo=0, hi=999, new_lo=900, new_hi=1300, Hkv=8, D=128, page=64,
             dtype="bf16", mix=4),
        # one request with a short context: latency
        dict(name="attn_decode_1x333", op="attn", B=1, lo=333, hi=333, new_lo=1, new_hi=1, Hq=32, Hkv=8, D=128, page=64,
             mix=5),
        # decode at 16 concurrent requests of ragged length
        dict(name="attn_decode_16x8k", op="attn", B=16, lo=2000, hi=8192, new_lo=1, new_hi=1, Hq=32, Hkv=8, D=128,
             page=64, mix=6),
        # decode at 512 concurrent requests, six query heads to a K/V head
        dict(name="attn_decode_512x2k", op="attn", B=512, lo=100, hi=4000, new_lo=1, new_hi=1, Hq=48, Hkv=8, D=128,
             page=64, mix=7),
        # one request with a long context: the keys are split over the whole GPU
        dict(name="attn_decode_1x131k", op="attn", B=1, lo=131035, hi=131035, new_lo=1, new_hi=1, Hq=64, Hkv=8, D=128,
             page=128, mix=8),
        # verification of a few drafted tokens, narrow heads, small pages
        dict(name="attn_verify_24x5", op="attn", B=24, lo=64, hi=5000, new_lo=2, new_hi=5, Hq=16, Hkv=4, D=64, page=16,
             mix=9),
        # prompt chunks after a cached prefix
        dict(name="attn_prompt_3x2k", op="attn", B=3, lo=500, hi=4000, new_lo=1500, new_hi=2100, Hq=32, Hkv=8, D=128,
             page=64, mix=10),
        # the norms around the MoE layer at 16 decode tokens (the layer's output is fp32)
        dict(name="norm_decode_16", op="norm", T=16, H=4096, a="f32", gate="none", post=True, mix=11),
        # the same for a prompt batch, bf16 block output, gate for every channel
        dict(name="norm_prompt_8191", op="norm", T=8191, H=6144, a="bf16", gate="channel", post=True, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "append", "append", "attn", "attn", "attn", "attn", "norm", "norm"))
    mix = rng.randrange(1 << 30)
    page = rng.choice((16, 32, 64, 128))
    if op == "plan":
        B = _log(rng, 1, 509)
        return dict(op=op, B=B, lo=0, hi=_log(rng, 1, 16384), new_hi=rng.randint(1, 8), prompts=rng.randint(0, min(B, 6)),
                    page=page, mix=mix)
    if op == "norm":
        T = _log(rng, 1, 8191)
        return dict(op=op, T=T, H=8 * rng.randint(16, 768), a=rng.choice(("f32", "bf16", "none")),
                    gate=rng.choice(("none", "channel", "token", "full")), post=rng.random() < 0.7, mix=mix)
    D = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    if op == "append":
        new = _log(rng, 1, 1300)
        B = _log(rng, 1, max(1, min(512, 7700 // new)))
        return dict(op=op, B=B, lo=0, hi=_log(rng, 1, 4096), new_lo=max(1, new // 2), new_hi=new, Hkv=Hkv, D=D,
                    page=page, dtype=rng.choice(("bf16", "f32")), mix=mix)
    Hq = Hkv * rng.randint(1, 8)
    kind = rng.choice(("decode", "decode", "verify", "prompt"))
    if kind == "prompt":
        new = _log(rng, 9, 2000)
        hi = _log(rng, 1, 4000)
        B = rng.randint(1, 3)
    else:
        new = 1 if kind == "decode" else rng.randint(2, 8)
        hi = _log(rng, 1, 131000)
        B = _log(rng, 1, max(1, min(512, 1000000 // (hi + new))))
    return dict(op=op, B=B, lo=hi // rng.choice((1, 2, 8)), hi=hi, new_lo=max(1, new // 2), new_hi=new, Hq=Hq, Hkv=Hkv,
                D=D, page=page, mix=mix)


def _spread(r, lo, hi):
    """A length in [lo, hi], uniform in the logarithm of 1 + length."""
    return min(hi, max(lo, int(round(math.exp(r.uniform(math.log(1 + lo), math.log(1 + hi))) - 1))))


def _lengths(c):
    """(cached tokens, new tokens) of every request of the case."""
    r = random.Random(c["mix"])
    ctx = [_spread(r, c["lo"], c["hi"]) for _ in range(c["B"])]
    if c["op"] == "plan":
        new = [r.randint(0, c["new_hi"]) if c["new_hi"] > 1 else 1 for _ in range(c["B"])]
        for b in r.sample(range(c["B"]), c["prompts"]):
            new[b] = r.randint(500, 2100)
    else:
        new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    return ctx, new


def _up(n, d):
    return -(-n // d)


# ---------------------------------------------------------------------------
# state
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(g, counts, spare, width=None):
    """Random page ids: a table [B, width] whose row b starts with counts[b] distinct pages (-1 behind them), and the unused
    pages."""
    total = sum(counts) + spare
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(counts), width or max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    n = torch.tensor(counts, device="cuda")
    used = torch.arange(table.shape[1], device="cuda")[None, :] < n[:, None]
    table[used] = ids[:sum(counts)]
    return table, ids[sum(counts):].contiguous(), total


def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127], exactly."""
    e = e.int()
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(F32)


def _rows_to_codes(x):
    """E4M3 codes and exponent bytes of whole blocks x [..., S, D]: the smallest power of two that covers each block."""
    amax = x.abs().amax((-2, -1)).float()
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1, and 448 = 0.875 * 2^9
    e = torch.where(amax > 0, (e - 9 + (m > 0.875).int()).clamp(-127, 127), torch.full_like(e, -127))
    codes = (x * _pow2(-e)[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _cache(g, P, Hkv, S, D):
    """A filled cache half: blocks of different magnitude, a few channels larger than the rest."""
    codes = torch.empty(P, Hkv, S, D, dtype=torch.uint8, device="cuda")
    exps = torch.empty(P, Hkv, dtype=torch.uint8, device="cuda")
    channel = 1 + 3 * (torch.rand(Hkv, 1, D, generator=g, device="cuda") > 0.95).float()
    step = max(1, (1 << 27) // (Hkv * S * D))
    for p in range(0, P, step):
        n = min(step, P - p)
        x = torch.randn(n, Hkv, S, D, generator=g, device="cuda") * channel
        x *= torch.exp2(torch.rand(n, Hkv, 1, 1, generator=g, device="cuda") - 0.5)
        codes[p:p + n], exps[p:p + n] = _rows_to_codes(x)
    return codes, exps


def prepare(case, seed):
    g = _gen(seed)
    c = case
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        s = dict(case=c, alpha=0.5 if c["gate"] != "none" else 1.0, eps=1e-6)
        s["x"] = (torch.randn(T, H, generator=g, device="cuda") * 2).to(BF16)
        s["a"] = None
        if c["a"] != "none":
            s["a"] = (torch.randn(T, H, generator=g, device="cuda") * torch.exp2(
                2 * torch.randn(T, 1, generator=g, device="cuda"))).to(F32 if c["a"] == "f32" else BF16)
        shape = dict(none=None, channel=(1, H), token=(T, 1), full=(T, H))[c["gate"]]
        s["gate"] = None if shape is None else torch.randn(*shape, generator=g, device="cuda").to(BF16)
        s["w_post"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF16) if c["post"] else None
        s["w_pre"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF16)
        return s
    ctx, new = _lengths(c)
    S = c["page"]
    if c["op"] == "plan":
        held = [_up(n, S) for n in ctx]
        want = [_up(n + m, S) for n, m in zip(ctx, new)]
        table, free, total = _tables(g, held, sum(want) - sum(held) + 5, max(1, max(want)))
        return dict(case=c, ctx=_ints(ctx), new=_ints(new), table=table, free=free, free_count=_ints([free.numel()]),
                    page=S, T=sum(new))
    kv = [n + m for n, m in zip(ctx, new)]
    table, _, P = _tables(g, [_up(n, S) for n in kv], 3)
    T, Hkv, D = sum(new), c["Hkv"], c["D"]
    start = [0]
    for m in new:
        start.append(start[-1] + m)
    if c["op"] == "append":
        # K and V are slices of one projection's output, after two query heads' columns
        dt = BF16 if c["dtype"] == "bf16" else F32
        x = (torch.randn(T, 2 + 2 * Hkv, D, generator=g, device="cuda") * torch.exp2(
            torch.randn(T, 1, 1, generator=g, device="cuda"))).to(dt)
        kc, ke = _cache(g, P, Hkv, S, D)
        vc, ve = _cache(g, P, Hkv, S, D)
        at = torch.cat([torch.arange(n, n + m) for n, m in zip(ctx, new)]).cuda()
        who = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(new)).cuda()
        slots = (table[who, at // S].long() * S + at % S).to(torch.int32)
        return dict(case=c, k=x[:, 2:2 + Hkv], v=x[:, 2 + Hkv:], slots=slots, kc=kc, ke=ke, vc=vc, ve=ve)
    Hq = c["Hq"]
    q = (3 * torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda")).to(BF16)[:, :Hq]
    kc, ke = _cache(g, P, Hkv, S, D)
    vc, ve = _cache(g, P, Hkv, S, D)
    s = dict(case=c, q=q, kc=kc, ke=ke, vc=vc, ve=ve, table=table, kv_lens=_ints(kv), start=_ints(start),
             max_q=max(new), scale=D ** -0.5)
    # the workspace that a serving program allocates once
    s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from nvfp4_mixture_experts_top_gb300 import binding as B
        if op == "plan":
            r = B.kv_plan(s["ctx"], s["new"], s["table"], s["free"], s["free_count"], s["page"], s["T"])
            return dict(table=s["table"], **r)
        if op == "append":
            B.kv_append(s["k"], s["v"], s["slots"], s["kc"], s["ke"], s["vc"], s["ve"])
            return _held(s)
        if op == "attn":
            out, lse = B.kv_attention(s["q"], s["kc"], s["ke"], s["vc"], s["ve"], s["table"], s["kv_lens"], s["start"],
                                      s["max_q"], s["scale"], want_lse=True, workspace=s["workspace"])
            return dict(out=out, lse=lse)
        y, h = B.block_norm(s["x"], s["a"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], alpha=s["alpha"],
                            eps=s["eps"])
        return dict(h=h) if s["a"] is None else dict(y=y, h=h)
    return dict(plan=_plan, append=_append, attn=_attn, norm=_norm)[op](s)


def _held(s):
    """The cache after an append: its 8-bit elements as the E4M3 values they stand for, and its exponent bytes."""
    return dict(k=s["kc"].view(torch.float8_e4m3fn), v=s["vc"].view(torch.float8_e4m3fn), ke=s["ke"], ve=s["ve"])


def _plan(s):
    S, table, T = s["page"], s["table"], s["T"]
    ctx, new = s["ctx"].long(), s["new"].long()
    B, M = table.shape
    held, want = (ctx + S - 1) // S, (ctx + new + S - 1) // S
    need = want - held
    first = torch.cumsum(need, 0) - need
    n = s["free_count"].long()
    fits = (need == 0) | ((first + need <= n) & (want <= M))
    j = torch.arange(M, device="cuda")[None, :]
    take = (j >= held[:, None]) & (j < want[:, None]) & fits[:, None]
    at = (n - 1 - (first[:, None] + j - held[:, None])).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(take, s["free"][at], table))
    start = torch.cat([torch.zeros_like(ctx[:1]), torch.cumsum(new, 0)])
    t = torch.arange(T, device="cuda")
    who = torch.searchsorted(start[1:], t, right=True)
    p = ctx[who] + t - start[who]
    slots = torch.where(fits[who], table[who, p // S].long() * S + p % S, torch.full_like(p, -1))
    return dict(table=table, query_start=start.int(), kv_lens=torch.where(fits, ctx + new, ctx).int(),
                slot_map=slots.int(), free_left=(n - (need * fits).sum()).int())


def _append(s):
    slots = s["slots"].long()
    S = s["kc"].shape[2]
    page, off = slots // S, slots % S
    P = s["kc"].shape[0]
    first = torch.full((P,), S, device="cuda").scatter_reduce(0, page, off, "amin")  # first new offset of each page
    for x, codes, exps in ((s["k"], s["kc"], s["ke"]), (s["v"], s["vc"], s["ve"])):
        x = x.float()
        top = torch.zeros(P, x.shape[1], device="cuda").scatter_reduce(
            0, page[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        m, e = torch.frexp(top)
        e = torch.where(top > 0, (e - 9 + (m > 0.875).int()).clamp(-127, 127), torch.full_like(e, -127))
        old = exps.int() - 127
        touched = (first < S)[:, None]
        e = torch.where(touched, torch.where((first > 0)[:, None], torch.maximum(e, old), e), old)
        # what the touched blocks hold already moves to the new exponent
        b = torch.unique_consecutive(page)
        was = codes[b].view(torch.float8_e4m3fn).float() * _pow2((old[b] - e[b]).clamp(min=-126))[..., None, None]
        keep = torch.arange(S, device="cuda")[None, :] < first[b][:, None]
        codes[b] = torch.where(keep[:, None, :, None], was.to(torch.float8_e4m3fn).view(torch.uint8), codes[b])
        y = (x * _pow2(-e[page])[..., None]).clamp(-448, 448)
        codes[page, :, off] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        exps.copy_((e + 127).to(torch.uint8))
    return _held(s)


def _attn(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G, S, B, n = Hq // Hkv, c["page"], c["B"], s["max_q"]
    T = s["q"].shape[0]
    start, kv = s["start"].long(), s["kv_lens"].long()
    ql = start[1:] - start[:-1]
    i = torch.arange(n, device="cuda")
    tok = (start[:-1, None] + i).clamp(max=T - 1)
    q = s["q"][tok].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    table = s["table"].long().clamp(min=0)
    L = table.shape[1] * S

    def read(codes, exps):
        x = codes[table].view(torch.float8_e4m3fn).float()  # [B, pages, Hkv, S, D]
        x *= _pow2(exps[table].int() - 127)[..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)

    x = torch.matmul(q, read(s["kc"], s["ke"]).transpose(-1, -2)) * s["scale"]
    limit = (kv - ql)[:, None] + i + 1  # keys that query i sees
    seen = torch.arange(L, device="cuda") < limit[..., None]  # [B, n, L]
    x = x.view(B, Hkv, G, n, L).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    del x
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)  # [B, Hkv, G, n]
    o = torch.matmul(p.view(B, Hkv, G * n, L), read(s["vc"], s["ve"])).view(B, Hkv, G, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    who = torch.repeat_interleave(torch.arange(B, device="cuda"), ql, output_size=T)
    at = torch.arange(T, device="cuda") - start[who]
    return dict(out=o.permute(0, 3, 1, 2, 4)[who, at].reshape(T, Hq, D).to(BF16),
                lse=lse.permute(0, 3, 1, 2)[who, at].reshape(T, Hq))


def _norm(s):
    y = s["x"].float()
    if s["a"] is not None:
        a = s["a"].float()
        if s["w_post"] is not None:
            a = a * torch.rsqrt(a.square().mean(-1, keepdim=True) + s["eps"]) * s["w_post"].float()
        if s["gate"] is not None:
            a = a * s["gate"].float()
        y = y + s["alpha"] * a
    h = (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * s["w_pre"].float()).to(BF16)
    return dict(h=h) if s["a"] is None else dict(y=y.to(BF16), h=h)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _two(e):
    """2^e in float64 for whole e in [-400, 400], from a table."""
    t = torch.tensor([2.0 ** i for i in range(-400, 401)], dtype=torch.float64, device=e.device)
    return t[e.long() + 400]


def _value(codes):
    """E4M3 (sign, 4 exponent bits of bias 7, 3 fraction bits) as float64."""
    c = codes.long()
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + f / 8) * _two(e - 7), f * 2.0 ** -9)
    return torch.where(c >= 128, -v, v)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    if op == "norm":
        x, wp = s["x"].double(), s["w_pre"].double()
        if s["a"] is None:
            return dict(h=x / torch.sqrt((x * x).mean(1, keepdim=True) + s["eps"]) * wp)
        a = s["a"].double()
        if s["w_post"] is not None:
            a = a / torch.sqrt((a * a).mean(1, keepdim=True) + s["eps"]) * s["w_post"].double()
        y = x + s["alpha"] * (a if s["gate"] is None else s["gate"].double() * a)
        return dict(y=y, h=y / torch.sqrt((y * y).mean(1, keepdim=True) + s["eps"]) * wp)
    ctx, new = _lengths(case)
    S = case["page"]
    if op == "append":
        if sum(new) > 20000 or len(new) > 600:
            return None
        grid = _value(torch.arange(127, device="cuda"))

        def nearest(v):  # to E4M3, ties to the even code, saturating
            at = torch.searchsorted((grid[1:] + grid[:-1]) / 2, v.abs())
            tie = v.abs() == ((grid[1:] + grid[:-1]) / 2)[at.clamp(max=125)]
            at = torch.where(tie & (at < 126) & (at % 2 == 1), at + 1, at)
            return torch.copysign(grid[at], v)

        res = {}
        slots = s["slots"].tolist()
        for name, x, codes, exps in (("k", s["k"], s["kc"], s["ke"]), ("v", s["v"], s["vc"], s["ve"])):
            held = _value(codes)
            t = 0
            while t < len(slots):
                u = t + 1
                while u < len(slots) and slots[u] == slots[u - 1] + 1 and slots[u] % S:
                    u += 1
                p, o = slots[t] // S, slots[t] % S
                rows = x[t:u].double()  # [n, Hkv, D]
                top = rows.abs().amax((0, 2))
                e = torch.ceil(torch.log2(top / 448)).clamp(-127, 127)
                e = torch.where(top > 448 * _two(e), e + 1, e)
                e = torch.where(top <= 448 * _two(e - 1), e - 1, e).clamp(-127, 127)
                if o:
                    old = exps[p].long() - 127
                    e = torch.maximum(e, old)
                    held[p, :, :o] = nearest(held[p, :, :o] * _two(old - e)[:, None, None])
                held[p, :, o:o + u - t] = nearest(rows.transpose(0, 1) * _two(-e)[:, None, None])
                t = u
            res[name] = held
        return dict(k=res["k"], v=res["v"], ke=None, ve=None)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    out, lse = [], []
    t = 0
    for b, (n, m) in enumerate(zip(ctx, new)):
        pages = s["table"][b, :_up(n + m, S)].long()

        def rows(codes, exps):
            x = _value(codes[pages]) * _two(exps[pages].long() - 127)[..., None, None]
            return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :n + m]

        k, v = rows(s["kc"], s["ke"]), rows(s["vc"], s["ve"])
        see = torch.arange(n + m, device="cuda")[None, :] <= torch.arange(n, n + m, device="cuda")[:, None]
        o, z = [], []
        for h in range(Hq):
            w = s["scale"] * (s["q"][t:t + m, h].double() @ k[h * Hkv // Hq].T)
            w = torch.where(see, w, torch.full_like(w, -math.inf))
            z.append(torch.logsumexp(w, 1))
            o.append(torch.exp(w - z[-1][:, None]) @ v[h * Hkv // Hq])
        out.append(torch.stack(o, 1))
        lse.append(torch.stack(z, 1))
        t += m
    return dict(out=torch.cat(out), lse=torch.cat(lse))


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        a = dict(none=0, bf16=2, f32=4)[c["a"]]
        gate = 0 if c["a"] == "none" else 2 * dict(none=0, channel=H, token=T, full=T * H)[c["gate"]]
        out = 2 if c["a"] == "none" else 4
        return dict(bytes=T * H * (a + 2 + out) + gate + 4 * H, flops=(10 if a else 4) * T * H)
    ctx, new = _lengths(c)
    T, S = sum(new), c["page"]
    if c["op"] == "plan":
        taken = sum(_up(n + m, S) - _up(n, S) for n, m in zip(ctx, new))
        held = sum(1 for n, m in zip(ctx, new) if m and n % S)  # pages that are begun already
        return dict(bytes=4 * (4 * c["B"] + 1 + T + 2 * taken + held + 2), flops=4 * T)
    Hkv, D = c["Hkv"], c["D"]
    if c["op"] == "append":
        size = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=2 * T * Hkv * D * (size + 1) + 4 * T, flops=4 * T * Hkv * D)
    Hq = c["Hq"]
    tokens = sum(ctx) + T
    pairs = sum(m * n + m * (m + 1) // 2 for n, m in zip(ctx, new))
    pages = sum(_up(n + m, S) for n, m in zip(ctx, new))
    return dict(bytes=2 * tokens * Hkv * D + pages * (4 + 2 * Hkv) + T * Hq * (4 * D + 4) + 8 * c["B"],
                flops=4 * pairs * Hq * D)
