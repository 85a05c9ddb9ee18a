"""The rotary append of prompts: blocks that go through many tokens, against 64 bits."""

import pytest

import memory_bound_gemv_gb300 as mbg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_decode import (BF16, F16, F32, HALF_STEP, TINY, close, make_cache, no_device_error,  # noqa: E402,F401
                             normal, rope_reference, same_bits)


# 400000 tokens of three heads are some 80 per block (64 threads, 32 blocks on an SM at most)
@pytest.mark.parametrize("tokens,hq,hk,dim,sections,pairs,shift", [
    (5003, 8, 2, 128, [16, 24, 24], True, 0), (5003, 8, 2, 128, [64], False, 1), (20000, 5, 1, 80, [13, 14, 13], False, 0),
    (400000, 1, 1, 16, [8], False, 0), (400000, 1, 1, 16, [3, 1, 1, 2, 1], True, 0), (400000, 1, 1, 10, [1, 1, 1, 1, 1], False, 0),
    (30000, 40, 8, 128, [16, 24, 24], False, 0)])
@pytest.mark.parametrize("src,dst", [(F32, F16), (BF16, BF16), (F16, BF16)])
def test_rope_prompt(tokens, hq, hk, dim, sections, pairs, shift, src, dst):
    starts = [3, 0, 17]
    counts = [tokens // 2, tokens // 3, tokens - tokens // 2 - tokens // 3]
    lengths = [a + n for a, n in zip(starts, counts)]
    cache = make_cache(101, lengths, hk, dim, 16, dst, shift=shift, fill=0.0, history=True)
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(counts)).to(torch.int32).cuda()
    slots = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, counts)]).to(torch.int32).cuda()
    mix = torch.randperm(tokens, device="cuda")  # neighbours in the call belong to different sequences
    seq, slots = seq[mix].contiguous(), slots[mix].contiguous()
    slots[::11] = -1  # padding, at every place among 32 tokens of a block
    qkv = normal(102, (tokens, hq + 2 * hk, dim), src, 1.3)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    positions = torch.randint(0, 10 ** 6, (len(sections), tokens), device="cuda", dtype=torch.int32)
    stamps = torch.randint(0, 10 ** 9, (tokens,), device="cuda", dtype=torch.int32)
    old = [cache.k.clone(), cache.v.clone(), cache.scores.clone(), cache.stamps.clone()]
    rope = mbg.RopeTable(2 * sum(sections), sections=sections, pairs=pairs)
    out = mbg.gemv_rope_append(cache, q, k, v, positions, slots, rope, seq=seq, stamps=stamps)
    args = (2 * sum(sections), sections, pairs)
    ref, mag = rope_reference(q, positions, args)
    close(out, ref, mag * 2.0 ** -20 + ref.abs() * HALF_STEP[dst] + TINY[dst], "q")
    del ref, mag
    put = (slots >= 0).nonzero()[:, 0]
    b, s = seq[put].long(), slots[put].long()
    pages, offs = cache.page_table[b, s // 16].long(), s % 16
    ref, mag = rope_reference(k[put], positions[:, put], args)
    close(cache.k[pages, offs], ref, mag * 2.0 ** -20 + ref.abs() * HALF_STEP[dst] + TINY[dst], "k")
    assert torch.equal(cache.v[pages, offs], v[put].float().to(dst))
    for now, was in zip((cache.k, cache.v), old):  # nothing else has changed
        was[pages, offs] = now[pages, offs]
        assert same_bits(now.contiguous(), was.contiguous())
    old[2][b, :, s] = 0.0
    old[3][b, :, s] = stamps[put][:, None]
    assert torch.equal(cache.scores, old[2]) and torch.equal(cache.stamps, old[3])
