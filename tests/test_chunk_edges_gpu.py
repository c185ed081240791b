"""The chunk operators on the GPU at the edges of what their documents allow: plans shared by caches of
different groups and capacities, many short prompts, plans and angles dropped while another stream still
reads them, large logits, large values, values of very different size; against the plain 64-bit forms
(chunk_testlib)."""
import math
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


def check_prompt(got, q, k, v, lens, what="", every=1):
    at = 0
    for i, n in enumerate(lens):
        if n and i % every == 0:
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
    check_prompt(got[0], q, k, v, lens, every=4)
    assert all(torch.equal(got[0], x) for x in got[1:])


# ------------------------------------------------------------------ memory that another stream still reads

def busy(ms=200):
    """Work on the current stream for about `ms`."""
    x = torch.zeros(1 << 28, dtype=torch.float32, device="cuda")           # 1 GiB: over 0.3 ms a pass
    for _ in range(3 * ms):
        x.add_(1.0)


@pytest.mark.parametrize("given", [False, True])
def test_a_plan_dropped_after_a_call_on_another_stream(given):
    """The plan is made on one stream and used on another, torch's current one or the call's own; its
    memory, and that of the angles' copies, is not handed out while calls wait there."""
    p, first = pair(), pair(seed=1)
    for x in (p, first):
        x.append([300, 10, 200, 1])
        x.cache.reserve(2, 260)
    cos, sin = (x.cuda() for x in ct.angles(512, 128))
    k, v, q = p.new(64, 2), p.new(64, 2), p.new(64, 8)
    dk, dv, dq = k.cuda(), v.cuda(), q.cuda()
    side = torch.cuda.Stream()

    def copies():                                   # not contiguous: Rope copies them
        return kvq.Rope(torch.stack([cos, cos], 2)[..., 0], torch.stack([sin, sin], 2)[..., 0])

    def plans(cache):
        return cache.plan_chunk([1, 2, 60, 1]), copies(), kvq.plan_prompt([40, 24], 8, 2, 128)

    def calls(cache, plan, rope, prompts, **on):
        turned = cache.append_chunk(plan, dk, dv, rope, dq, **on)
        return (turned, cache.chunk_attention(plan, turned, **on), cache.read_chunk(plan, **on)[0],
                kvq.prompt_attention(prompts, dq, dk, dv, **on))

    calls(first.cache, *plans(first.cache))         # (a kernel's first call may wait for the device)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy()
    plan, rope, prompts = plans(p.cache)
    torch.cuda.default_stream().synchronize()
    if given:
        got = calls(p.cache, plan, rope, prompts, stream=side)
    else:
        with torch.cuda.stream(side):
            got = calls(p.cache, plan, rope, prompts)
    lent = {t.data_ptr() for x in (plan, rope, prompts) for t in x._tensors}
    starts, offsets = plan.starts, plan.offsets
    positions = [s + i for s, n in zip(plan.starts, plan.counts) for i in range(n)]
    del plan, rope, prompts
    later = [x for _ in range(20) for x in (p.cache.plan_chunk([2, 1, 1, 60]), copies(),
                                            kvq.plan_prompt([24, 40], 8, 2, 128))]
    assert not side.query(), "the calls ended before the memory could be asked for again"
    assert not lent & {t.data_ptr() for x in later for t in x._tensors}
    side.synchronize()
    k, turned = (ct.rotate(x, positions, *ct.angles(512, 128), False) for x in (k, q))
    assert torch.equal(got[0].cpu(), turned)
    for b in range(4):
        rows = slice(offsets[b], offsets[b + 1])
        p.plain[b].append(starts[b], k[rows], v[rows])
    p.check_state()
    plan = p.cache.plan_chunk([1, 2, 60, 1], starts)
    p.check_attention(plan, turned, got=got[1])
    assert torch.equal(got[2], p.cache.read_chunk(plan)[0])
    check_prompt(got[3], q, dk.cpu(), v, [40, 24])


# ------------------------------------------------------------------ large logits

def one_hot_rows(q, k, first, margin):
    """(rows and heads whose largest logit leads by more than `margin`, which token that is): [n, Hq]."""
    n, hq, d = q.shape
    y = torch.einsum("nhd,hld->nhl", torch.from_numpy(q), torch.from_numpy(k).repeat_interleave(hq // k.shape[0], 0)) / d ** 0.5
    y[(torch.arange(k.shape[1])[None] > first + torch.arange(n)[:, None])[:, None].expand_as(y)] = -float("inf")
    top = torch.nn.functional.pad(y, (0, 1), value=-float("inf")).topk(2, -1)
    return top.values[..., 0] - top.values[..., 1] > margin, top.indices[..., 0]


def check_one_hot(got, q, k, v, first, dtype, what):
    """Logits of 2^30: their fp32 sums are off by many powers of two, so a row whose largest logit leads by
    more than that is one token's value, rounded once on the way (the cache's values to 11 bits) and
    once at the end, and the others lie among their tokens' values."""
    S = (abs(q).max(-1).max() * abs(k).max()) * q.shape[2] / q.shape[2] ** 0.5
    clear, token = one_hot_rows(q, k, first, 4 * (q.shape[2] + 8) * 2.0 ** -24 * S + 4 * 2.0 ** -11 * S)
    hg = q.shape[1] // k.shape[0]
    out = torch.from_numpy(ct.wide(got))
    assert torch.isfinite(out).all(), f"{what}: not finite"
    u = ct.half_step(dtype)
    vt = torch.from_numpy(v)
    assert (out.abs() <= vt.abs().max() * (1 + u) * (1 + 2.0 ** -10)).all(), what
    want = torch.stack([vt[h // hg][token[:, h]] for h in range(q.shape[1])], 1)
    off = (out - want).abs() <= want.abs() * (u + 2.0 ** -10) + 2.0 ** -24 * vt.abs().max()
    assert off[clear].all(), what
    return int(clear.sum())


@pytest.mark.parametrize("dtype,size", [(BF16, 2.0 ** 16), (FP16, 2.0 ** 13), (BF16, 2.0 ** 20)])
@pytest.mark.parametrize("counts", [[2, 1, 3, 0], [40, 130, 60, 0]])
def test_large_logits_over_the_cache(dtype, size, counts):
    p = pair(dtype=dtype, bits=4, capacity=4096)
    held = [3000, 10, 300, 50]
    for c in (held, counts):
        plan = p.cache.plan_chunk(c)
        k, v = p.new(plan.tokens, 2, size), p.new(plan.tokens, 2)
        p.cache.append_chunk(plan, k.cuda(), v.cuda())
        for b, (s, n) in enumerate(zip(plan.starts, plan.counts)):
            rows = slice(plan.offsets[b], plan.offsets[b + 1])
            p.plain[b].append(s, k[rows], v[rows])
    q = p.new(plan.tokens, 8, size)
    got = p.cache.chunk_attention(plan, q.cuda())
    p.cache.check_device()
    clear = 0
    for b in range(3):
        hk, hv = p.plain[b].held()
        rows = slice(plan.offsets[b], plan.offsets[b + 1])
        clear += check_one_hot(got[rows], ct.wide(q[rows]), hk, hv, plan.starts[b], dtype, f"slot {b}")
    assert clear > 0


@pytest.mark.parametrize("dtype,size", [(BF16, 2.0 ** 16), (FP16, 2.0 ** 13), (BF16, 2.0 ** 20), (BF16, 2.0 ** 56)])
def test_large_logits_of_prompts(dtype, size):
    lens, hq, hkv, d = [600, 1, 130], 4, 2, 128
    gen = torch.Generator().manual_seed(5)
    q, k, v = ((torch.randn(sum(lens), h, d, generator=gen) * s).to(dtype) for h, s in ((hq, size), (hkv, size), (hkv, 1.0)))
    got = kvq.prompt_attention(kvq.plan_prompt(lens, hq, hkv, d), q.cuda(), k.cuda(), v.cuda())
    at = clear = 0
    for n in lens:
        rows = slice(at, at + n)
        clear += check_one_hot(got[rows], ct.wide(q[rows]), ct.wide(k[rows]).transpose(1, 0, 2),
                               ct.wide(v[rows]).transpose(1, 0, 2), 0, dtype, f"rows {rows}")
        at += n
    assert clear > 0


def test_rows_whose_logits_all_lie_far_below_zero():
    """One token a prompt, attended by queries opposite to its key: logits of -2^113, weight 1."""
    gen = torch.Generator().manual_seed(9)
    k, v = ((torch.randn(20, 2, 128, generator=gen) * s).to(BF16) for s in (2.0 ** 55, 1.0))
    plan = kvq.plan_prompt([1] * 20, 2, 2, 128)
    got = kvq.prompt_attention(plan, -k.cuda(), k.cuda(), v.cuda())
    assert torch.equal(got.cpu(), v)


# ------------------------------------------------------------------ values of different size, large values

def largest_share(q, k, v, first):
    """max over 32 tokens of (the largest weight among them times the largest value among them), for each
    query row: the largest thing the row's sum is made of, [n, Hq, 1]."""
    n, hq, d = q.shape
    hkv, tokens, _ = k.shape
    out = torch.zeros(n, hq, 1, dtype=torch.float64).numpy()
    pad = -tokens % 32
    for h in range(hq):
        y = q[:, h] @ k[h // (hq // hkv)].T / d ** 0.5
        y[torch.arange(tokens)[None].numpy() > first + torch.arange(n)[:, None].numpy()] = -float("inf")
        p = torch.softmax(torch.from_numpy(y), 1)
        p = torch.nn.functional.pad(p, (0, pad)).view(n, -1, 32).amax(2)
        w = torch.nn.functional.pad(torch.from_numpy(abs(v[h // (hq // hkv)]).max(1)), (0, pad)).view(-1, 32).amax(1)
        out[:, h, 0] = (p * w).amax(1).numpy()
    return out


def check_by_what_rows_see(p, b, plan, q, got):
    """As Pair.check_attention, with the weights' absolute rounding measured by the row itself.  A weight
    meets its 32 tokens' values under a power of two; the products' scale is such that the largest
    of (weight x 2^e of its values) lies at 2^5 or above, and fp16 is off by at most 2^-25 below 2^-14: of a
    bound on the values, 2^e is at most 2^-11, a value at most 2^15 2^e, and a bound at most twice the
    largest value, so a token's share is off by 2^-25 2^-5 2^-11 2^15 2 = 2^-25 of the largest share."""
    k, v = p.plain[b].held()
    rows = slice(plan.offsets[b], plan.offsets[b + 1])
    qw = ct.wide(q[rows])
    o, A, S, _ = ct.attend(qw, k, v, plan.starts[b])
    share = largest_share(qw, k, v, plan.starts[b])
    ct.check_attention(got[rows], o, A, S, share, k.shape[1], p.dtype, True)

@pytest.mark.parametrize("held,count", [(6090, 2), (6050, 40), (245, 2), (210, 40)])
def test_large_values_in_the_residual(held, count):
    """bf16 values of 1e37 in the rows that are not quantized: their weighted sum before it is divided
    passes the range of fp32, their average does not.  Over a split cache and a short one, with few and
    with many rows."""
    p = pair(slots=1, capacity=8192)
    for n in (held, count):
        plan = p.cache.plan_chunk([n])
        start = plan.starts[0]
        k, v = p.new(n, 2, 0.1), (1.0 + p.new(n, 2, 0.25)).abs()
        first = max(0, (held + count) // 128 * 128 - start)          # of those that stay in the residual
        v[first:] *= 1e37
        p.cache.append_chunk(plan, k.cuda(), v.cuda())
        p.plain[0].append(start, k, v)
    q = p.new(count, 8)
    k, v = p.plain[0].held()
    assert k.shape[1] % 128 > 60
    check_by_what_rows_see(p, 0, plan, q, p.cache.chunk_attention(plan, q.cuda()))
    p.cache.check_device()


def test_large_values_of_prompts():
    """bf16 values up to 3e38, whose weighted sums before they are divided pass the range of fp32."""
    lens, hq, hkv, d = [700, 3, 150], 4, 2, 128
    gen = torch.Generator().manual_seed(6)
    q, k = (torch.randn(sum(lens), h, d, generator=gen).to(BF16) for h in (hq, hkv))
    v = ((2.5 + torch.rand(sum(lens), hkv, d, generator=gen) / 2) * 1e38).to(BF16)
    plan = kvq.plan_prompt(lens, hq, hkv, d)
    check_prompt(kvq.prompt_attention(plan, q.cuda(), k.cuda(), v.cuda()), q, k, v, lens)
    plan.check_device()


def test_a_hundred_thousand_small_weights():
    """fp16: a first token with nearly all the weight, and 100000 whose weights of 2^-26 are together a
    six-hundredth of it; the last rows, against their formula.  The weights' rounding (2^-11, and 2^-25 2^-7
    each below 2^-14) and the output's; logits are 0 but for the first."""
    n, d = 100000, 64
    q, k = torch.zeros(n, 1, d, dtype=FP16), torch.zeros(n, 1, d, dtype=FP16)
    q[..., 0], k[0, 0, 0] = 8.0, 26 * math.log(2)
    v = torch.ones(n, 1, d, dtype=FP16)
    v[0] = 0.0
    got = kvq.prompt_attention(kvq.plan_prompt([n], 1, 1, d), q.cuda(), k.cuda(), v.cuda())[-100:].cpu().double()
    seen = torch.arange(n - 100, n, dtype=torch.float64)
    w = torch.exp(-q[0, 0, 0].double() * k[0, 0, 0].double() / d ** 0.5)
    want = (seen * w / (1 + seen * w))[:, None, None].expand_as(got)
    assert ((got - want).abs() <= 2.0 ** -10 * want + 1e5 * 2.0 ** -32 + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype,bits", [(BF16, 2), (FP16, 4)])
@pytest.mark.parametrize("count", [3, 100])
@pytest.mark.parametrize("at", ["before", "between", "ahead"])
@pytest.mark.parametrize("power", [8, 18])
def test_large_values_that_hardly_weigh(dtype, bits, count, at, power):
    """One token with two fifths of the weight, thousands that share the rest, and a block of values 2^power
    times the others', of weight next to none, before them, among them or behind the queries.  All
    values are positive, so that what is lost of the many shows."""
    p = pair(slots=1, dtype=dtype, bits=bits, capacity=8192)
    n = 6000
    k, v = p.new(n, 2, 0.02), (1.0 + p.new(n, 2, 0.25)).abs() / 16
    big = {"before": slice(0, 96), "between": slice(2944, 3040), "ahead": slice(n - 100, n)}[at]
    k[..., 7] = 0.0
    k[150 if at == "ahead" else big.stop + 14, :, 7] = 23.5   # 8.3 nats, 12 powers of two, above the others
    k[big, :, 7] = -46.0                             # 23 powers of two below them
    v[big] *= 2.0 ** power
    plan = p.cache.plan_chunk([n])
    p.cache.append_chunk(plan, k.cuda(), v.cuda())
    p.plain[0].append(0, k, v)
    start = n - 130 - (0 if at == "ahead" else count - 30)
    plan = p.cache.plan_chunk([count], [start if at != "ahead" else n - 100 - count])
    q = p.new(count, 8, 0.05)
    q[..., 7] = 4.0
    check_by_what_rows_see(p, 0, plan, q, p.cache.chunk_attention(plan, q.cuda()))


@pytest.mark.parametrize("count", [2, 60])
def test_values_of_every_size(count):
    """Values that grow and shrink by 2^20 from block to block, weights that follow no order."""
    p = pair(slots=1, capacity=8192, seed=count)
    n = 5000
    k, v = p.new(n, 2, 1.5), (1.0 + p.new(n, 2, 0.25)).abs()
    for i in range(0, n, 128):
        v[i:i + 128] *= 2.0 ** ((i * 7 // 128) % 21 - 10)
    plan = p.cache.plan_chunk([n])
    p.cache.append_chunk(plan, k.cuda(), v.cuda())
    p.plain[0].append(0, k, v)
    plan = p.cache.plan_chunk([count], [n - count])
    q = p.new(count, 8, 1.5)
    check_by_what_rows_see(p, 0, plan, q, p.cache.chunk_attention(plan, q.cuda()))


# ------------------------------------------------------------------ refusals

def test_a_refused_append_gives_its_pages_back():
    """Angles that end before the tokens do: refused by the library, after the pages were looked for."""
    p = ct.Pair(4, 8, 2, 128, 32, 32, 128, 2, False, BF16, 1024, 128, num_pages=6)
    p.append([200, 10, 0, 0])
    free = list(p.cache.free_pages)
    short = kvq.Rope(*(x.cuda() for x in ct.angles(250, 128)))
    k = p.new(900, 2).cuda()
    for counts in ([100, 250, 0, 0], [100, 0, 300, 200], [0, 0, 0, 640]):
        n = sum(counts)
        with pytest.raises(kvq.KVQError) as e:
            p.cache.append_chunk(p.cache.plan_chunk(counts), k[:n], k[:n], short)
        assert e.value.status == kvq.KVQ_ERR_INVALID_ARG
        assert p.cache.free_pages == free and [len(x) for x in p.cache.pages] == [1, 0, 0, 0]
    plan, _, _ = p.append([0, 118, 512, 5])         # all that is left
    assert not p.cache.free_pages
    p.check_state()
    p.check_read(plan)
