"""The decoder block of examples/decoder_block.py: plan, cache, attention, norms and
experts one after another, each operator's output against its 64-bit definition on
the inputs that the block gave it, with the operators' own bounds."""
import importlib.util
import os

import pytest
import torch

import kv_reference as ref
from gpu_helpers import cuda_or_skip

pytestmark = pytest.mark.gpu
_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")
BF = torch.bfloat16


def _example():
    spec = importlib.util.spec_from_file_location("decoder_block", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _run(steps, seed, check):
    """Prompts of ragged lengths, then chunks; returns every step's x and h."""
    m, dev = _example(), cuda_or_skip()
    block = m.Block(device=dev)
    n = len(steps[0])
    total = [sum(s[b] for s in steps) for b in range(n)]
    pages = sum(-(-t // 32) for t in total)
    cache = m.Cache(n, pages, max(total), block.Hkv, block.D, 32, dev)
    copies = [t.clone().zero_() for t in cache.arrays()]
    for t, c in zip(cache.arrays(), copies):
        t.copy_(c)
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, outs = [0] * n, []
    for new in steps:
        T = sum(new)
        x = torch.randn(T, block.H, generator=g, device=dev).to(BF)
        x0 = x.clone()
        h = block.enter(x)
        x, h2, s = block.step(x, h, torch.tensor(new, dtype=torch.int32, device=dev), max(new), cache, block.norms[0])
        assert int(block.status) == 0
        lens = [a + b for a, b in zip(lens, new)]
        start = [sum(new[:b]) for b in range(n + 1)]
        assert s["kv_lens"].tolist() == lens and s["query_start"].tolist() == start
        outs += [x.clone(), h2]
        if not check:
            continue
        # the cache holds what the rows say (its blocks may carry a rescaling, which the restatement repeats)
        kc, ke, vc, ve = copies
        ref.append(s["k"].double(), s["slot_map"].tolist(), kc, ke)
        ref.append(s["v"].double(), s["slot_map"].tolist(), vc, ve)
        for got, want in zip(cache.arrays(), copies):
            assert torch.equal(got, want)
        scale = block.D ** -0.5
        o, z, W, slack = ref.attention(s["q"], *cache.arrays(), cache.table, lens, start, scale)
        d = scale * 2.0 ** -17 * s["q"].double().abs().amax(-1) * slack + 2.0 ** -20 * (1 + z.abs())
        bound = 2.0 ** -8 * o.abs() + (2.0 ** -9 + 2.0 ** -12 + 2 * d[..., None]) * W
        assert not bool(torch.isinf(z).any()) and bool(((s["a"].double() - o).abs() <= bound).all())
        # the residual stream: x0 + norm(a W_o) + norm(m), rounded to bf16 in between; fp32
        # sums and products keep h to 2^-17 of its terms, which 2^-15 of the largest covers
        y1, h1 = ref.norm(x0, s["a"].flatten(1) @ block.w_o, None, block.norms[1], block.norms[2], 1.0, 1e-6)
        assert bool(((s["h1"].double() - h1).abs() <= 2.0 ** -8 * h1.abs() + 2.0 ** -15 * (1 + h1.abs().amax())).all())
        y2, h = ref.norm(y1.to(BF), s["m"], None, block.norms[3], block.norms[0], 1.0, 1e-6)
        # y1 in 32 bits may round to the other neighbour: one step of bf16 of it, and one rounding
        assert bool(((x.double() - y2).abs() <= 2.0 ** -8 * y2.abs() + 2.0 ** -7 * y1.abs() + 2.0 ** -15).all())
        assert bool(torch.isfinite(s["m"]).all()) and bool(torch.isfinite(h2.float()).all())
    held = sum(-(-t // 32) for t in lens)
    assert int(cache.free_count) == pages - held
    used = cache.table.cpu()
    ids = [int(used[b, j]) for b in range(n) for j in range(-(-lens[b] // 32))]
    assert len(set(ids)) == held and all(0 <= i < pages for i in ids)
    return outs


def test_prompts_chunks_and_single_tokens():
    _run([[200, 1, 33, 64], [1, 1, 1, 1], [5, 40, 2, 1], [1, 1, 1, 1], [0, 3, 0, 130]], 3, True)


def test_repeats_bit_for_bit():
    steps = [[130, 7], [1, 1], [1, 1]]
    for a, b in zip(_run(steps, 5, False), _run(steps, 5, False)):
        assert torch.equal(a, b)


def test_the_command_runs(capsys, monkeypatch):
    cuda_or_skip()
    monkeypatch.setattr("sys.argv", ["decoder_block.py", "--requests", "3", "--prompt", "90", "--steps", "2"])
    _example().main()
    assert "2 steps of 3 requests" in capsys.readouterr().out
