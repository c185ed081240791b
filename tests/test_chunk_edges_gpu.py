"""The chunk operators on the GPU at the edges of what their documents allow: plans shared by caches of
different groups and capacities, many short prompts, against the plain 64-bit forms (chunk_testlib)."""
import random

import pytest
import torch

from bit_kv_cache_22_b200 import kvq

import chunk_testlib as ct

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

FP16, BF16 = torch.float16, torch.bfloat16


def pair(slots=4, hq=8, hkv=2, d=128, G=32, Gv=32, R=128, bits=2, sym=False, dtype=BF16, capacity=1024, page=128, seed=0):
    return ct.Pair(slots, hq, hkv, d, G, Gv, R, bits, sym, dtype, capacity, page, seed)


def check_prompt(got, q, k, v, lens, what=""):
    at = 0
    for n in lens:
        if n:
            rows = slice(at, at + n)
            plain = ct.attend(ct.wide(q[rows]), ct.wide(k[rows]).transpose(1, 0, 2), ct.wide(v[rows]).transpose(1, 0, 2), 0)
            ct.check_attention(got[rows], *plain, n, q.dtype, False, f"{what} rows {rows}")
        at += n


# ------------------------------------------------------------------ one plan, several caches

@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [1, 1, 0, 1]])
def test_a_decode_step_planned_for_other_groups(counts):
    """A plan of single tokens made for groups of 16 tokens, which no decode kernel on the tensor cores
    serves, reserves no scratch for one; groups of 32 have one."""
    maker, p = pair(G=16), pair()
    held = [300 * n for n in counts]
    p.append(held)
    p.append(counts)
    plan = maker.cache.plan_chunk(counts, held)
    assert plan.chunk.workspace == 0
    p.check_attention(plan)
    own = p.cache.plan_chunk(counts, held)
    assert own.chunk.workspace > 0
    p.check_attention(own)
    p.cache.check_device()
    maker.append(held)
    maker.append(counts)
    maker.check_attention(own)                      # and the other way: more room than needed
    maker.cache.check_device()


def test_a_decode_step_planned_for_a_smaller_capacity():
    """The decode kernel's splits follow from the cache, up to its capacity's."""
    maker, p = pair(slots=2, capacity=512), pair(slots=2, capacity=8192)
    held = [8000, 40]
    p.append(held)
    p.append([1, 1])
    plan, own = maker.cache.plan_chunk([1, 1], held), p.cache.plan_chunk([1, 1], held)
    assert plan.chunk.workspace < own.chunk.workspace
    q = p.new(2, 8)
    p.check_attention(plan, q)
    p.check_attention(own, q)
    p.cache.check_device()
    # a workspace of the caller's: what the plan asks for is enough, unaligned is refused
    lib, dq = kvq.load(), q.cuda()
    out = torch.empty_like(dq)
    rows = [kvq.Rows(t.data_ptr(), 8 * 128, 128) for t in (dq, out)]
    work = torch.empty(own.chunk.workspace + 16, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for use in (own, plan):
        room = use.chunk.workspace
        guard = work[room:room + 16].fill_(77)
        assert lib.kvq_paged_chunk_attention(p.cache._h, use.ref, *rows, work.data_ptr(), room, stream) == kvq.KVQ_OK
        p.check_attention(use, q, got=out)
        assert (guard == 77).all()
        assert lib.kvq_paged_chunk_attention(p.cache._h, use.ref, *rows, work.data_ptr() + 8, room, stream) == \
            kvq.KVQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ many short prompts

@pytest.mark.parametrize("hq,hkv,d,lo,hi", [(8, 2, 128, 33, 64), (8, 2, 64, 1, 127), (4, 4, 128, 1, 127), (6, 2, 128, 120, 260)])
def test_several_hundred_short_prompts(hq, hkv, d, lo, hi):
    """Many jobs a CTA, nearly each ending in a key tile that its prompt fills in part, of one query
    tile and of two."""
    rng = random.Random(hq + hi)
    lens = [rng.randint(lo, hi) for _ in range(500)]
    gen = torch.Generator().manual_seed(hi)
    q, k, v = (torch.randn(sum(lens), h, d, generator=gen).to(BF16) for h in (hq, hkv, hkv))
    plan = kvq.plan_prompt(lens, hq, hkv, d)
    assert plan.chunk.items * hkv > 3 * 148
    dev = [x.cuda() for x in (q, k, v)]
    got = [kvq.prompt_attention(plan, *dev) for _ in range(5)]
    plan.check_device()
    check_prompt(got[0], q, k, v, lens)
    assert all(torch.equal(got[0], x) for x in got[1:])
