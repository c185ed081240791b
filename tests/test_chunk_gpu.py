"""The chunk operators on the GPU against plain 64-bit forms (chunk_testlib)."""
import numpy as np
import pytest
import torch

from bit_kv_cache_22_b200 import kvq

import chunk_testlib as ct

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

FP16, BF16 = torch.float16, torch.bfloat16

# slots, hq, hkv, d, G, Gv, R, bits, sym, dtype, page
GEOMETRIES = {
    "gqa2": (4, 8, 2, 128, 32, 32, 128, 2, False, BF16, 128),
    "mha4": (4, 3, 3, 128, 128, 128, 128, 4, False, BF16, 256),
    "small": (5, 2, 2, 64, 32, 32, 32, 2, False, FP16, 64),
    "sym4": (3, 12, 4, 128, 32, 32, 96, 4, True, BF16, 192),
    "g16": (3, 5, 1, 64, 16, 16, 64, 4, False, FP16, 64),
    "g256": (2, 8, 1, 128, 256, 64, 256, 2, True, FP16, 256),
}


def make(name, capacity=1024, seed=0, **kw):
    slots, hq, hkv, d, G, Gv, R, bits, sym, dtype, page = GEOMETRIES[name]
    return ct.Pair(slots, hq, hkv, d, G, Gv, R, bits, sym, dtype, capacity, page, seed, **kw)


# ------------------------------------------------------------------ append and read

@pytest.mark.parametrize("name", GEOMETRIES)
def test_append_chunk_leaves_the_state_of_single_appends(name):
    """Chunks of 0, 1, a few and many tokens, from empty and mid-block: codes bit for bit."""
    p = make(name)
    R, B = p.g.residual, p.g.batch
    for step, counts in enumerate([[R + 5, 0, 1, 3, R][:B], [1, 2 * R + 1, R - 1, 0, 7][:B], [2, 0, R, 2 * R - 3, R + 1][:B],
                                   [0] * B, [1] * B]):
        plan, _, _ = p.append(counts, strided=step % 2 == 1)
        p.check_state(f"step {step}")
        p.check_read(plan, f"step {step}")


@pytest.mark.parametrize("name,rot,pairs", [("gqa2", 128, False), ("gqa2", 64, True), ("small", 64, False),
                                            ("small", 16, True), ("sym4", 32, False), ("g256", 128, True),
                                            ("g16", 48, False)])
def test_append_chunk_rotates_keys_and_queries(name, rot, pairs):
    p = make(name)
    R, B = p.g.residual, p.g.batch
    rope = ct.angles(1024, rot)
    for step, counts in enumerate([[R + 5, 1, 30, 0, 2][:B], [3, R, 1, 2 * R + 2, 1][:B]]):
        plan, got, want = p.append(counts, rope=rope, pairs=pairs, strided=step == 1, queries=True)
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
        p.check_state(f"step {step}")
        p.check_read(plan)


@pytest.mark.parametrize("name", ["small", "g16", "gqa2"])
def test_long_chunks_with_queries(name):
    """More tokens than all slots' residual rows: blocks, rests and queries of every slot."""
    p = make(name)
    R, B = p.g.residual, p.g.batch
    rope = ct.angles(1024, 32)
    p.append([3, 0, R - 1, 1, 2][:B], rope=rope)
    for counts in ([2 * R + 1, R + 5, 3 * R, 2 * R, 0][:B], [R, 3 * R, 1, 2 * R + 3, R][:B]):
        assert sum(counts) > R * B
        plan, got, want = p.append(counts, rope=rope, queries=True, strided=True)
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
        p.check_state(str(counts))
        p.check_read(plan)


def test_queries_rotate_in_place_and_into_a_strided_output():
    p = make("gqa2")
    rope = kvq.Rope(*(x.cuda() for x in ct.angles(512, 128)))
    plan = p.cache.plan_chunk([3, 1, 0, 40])
    k, v, q = (p.new(44, h).cuda() for h in (2, 2, 8))
    want = ct.rotate(q.cpu(), [0, 1, 2, 0] + list(range(40)), *ct.angles(512, 128), False)
    wide = torch.full((44, 10, 128), 7.0, dtype=BF16, device="cuda")
    p.cache.append_chunk(plan, k, v, rope, q, out=wide[:, 1:9])
    assert torch.equal(wide[:, 1:9].cpu(), want) and (wide[:, 0] == 7).all() and (wide[:, 9] == 7).all()
    got = p.cache.append_chunk(plan, k, v, rope, q, out=q)
    assert got is q and torch.equal(q.cpu(), want)


def test_rejected_tokens_are_dropped():
    p = make("gqa2")
    R = p.g.residual
    p.append([R + 20, 50, 3 * R, 0])
    p.append([6, 6, 6, 6])                                   # drafts
    p.append([4, 2, 9, 1], starts=[R + 22, 50, 3 * R + 5, 6])   # some accepted, then new ones
    p.check_state("drafts")
    p.append([R + 3, 0, 5, 1], starts=[R, 0, R, 0])          # back to block borders
    p.check_state("borders")
    plan = p.cache.plan_chunk([1, 0, 0, 0], [R - 1, 0, 0, 0])
    with pytest.raises(kvq.KVQError) as e:                   # inside a quantized block
        p.cache.append_chunk(plan, p.new(1, 2).cuda(), p.new(1, 2).cuda())
    assert e.value.status == kvq.KVQ_ERR_STATE
    p.check_state("refused")


def test_append_chunk_agrees_with_append_and_prefill():
    """The same tokens one at a time, by prefill, or as chunks: bit-identical decode outputs."""
    p, r = make("gqa2"), make("gqa2")
    total = [300, 17, 128, 64]
    k, v = [[p.new(n, 2, s) for n in total] for s in (1.0, 0.5)]
    for b, n in enumerate(total):
        r.cache.prefill(b, k[b].transpose(0, 1).contiguous().cuda(), v[b].transpose(0, 1).contiguous().cuda())
    at = [0] * 4
    for part in ([100, 17, 1, 0], [200, 0, 127, 63], [0, 0, 0, 1]):
        plan = p.cache.plan_chunk(part)
        cut = lambda x: torch.cat([x[b][at[b]:at[b] + part[b]] for b in range(4)]).cuda()  # noqa: E731
        p.cache.append_chunk(plan, cut(k), cut(v))
        at = [a + n for a, n in zip(at, part)]
    for _ in range(3):
        tk, tv, tq = p.new(4, 2).cuda(), p.new(4, 2).cuda(), p.new(4, 8).cuda()
        p.cache.append(tk, tv)
        r.cache.append(tk, tv)
        assert torch.equal(p.cache.decode_attention(tq), r.cache.decode_attention(tq))


# ------------------------------------------------------------------ attention over the cache

@pytest.mark.parametrize("name", GEOMETRIES)
@pytest.mark.parametrize("counts", ["ones", "few", "mixed", "many"])
def test_chunk_attention(name, counts):
    p = make(name, seed=len(counts))
    R, B = p.g.residual, p.g.batch
    p.append([2 * R + 3, 0, R - 1, 5, R][:B])
    if counts != "ones":
        p.append([1] * B)
    c = {"ones": [1] * B, "few": [4, 3, 2, 1, 0][:B], "mixed": [R, 1, 0, 37, 130][:B],
         "many": [260, 129, 2 * R + 1, 200, 64][:B]}[counts]
    plan, _, _ = p.append(c)
    p.check_attention(plan, what=f"{name} {counts}")
    p.cache.check_device()


def test_chunk_attention_over_a_long_cache():
    """One token and a ragged chunk over 6000 tokens: the work is split over the tokens."""
    p = make("gqa2", capacity=8192)
    p.append([6000, 3000, 0, 129])
    plan, _, _ = p.append([1, 50, 2, 1])
    p.check_attention(plan)
    plan, _, _ = p.append([1, 1, 1, 1])
    p.check_attention(plan)


def test_chunk_attention_of_older_tokens():
    """Queries before the newest tokens see only up to their own position."""
    p = make("mha4")
    p.append([300, 150, 1, 0])
    plan = p.cache.plan_chunk([5, 150, 1, 0], [100, 0, 0, 0])
    p.check_attention(plan)


def test_decode_and_chunk_attention_agree():
    p = make("gqa2")
    p.append([500, 129, 1, 77])
    q = p.new(4, 8)
    plan = p.cache.plan_chunk([1] * 4, [499, 128, 0, 76])
    got = p.check_attention(plan, q)
    ref = p.cache.decode_attention(q.cuda())
    assert (got.float() - ref).abs().max() <= 0.02 * ref.abs().max()


@pytest.mark.parametrize("scale_k,scale_v", [(1e-6, 1e-6), (1e6, 1e4), (1e-3, 1e7), (30.0, 1e-9)])
def test_chunk_attention_magnitudes(scale_k, scale_v):
    """bf16 keys and values far from 1, queries scaled so that the logits stay ordinary."""
    p = make("gqa2")
    plan = p.cache.plan_chunk([200, 3, 131, 1])
    k, v = p.new(335, 2, scale_k), p.new(335, 2, scale_v)
    p.cache.append_chunk(plan, k.cuda(), v.cuda())
    for b in range(4):
        rows = slice(plan.offsets[b], plan.offsets[b + 1])
        p.plain[b].append(0, k[rows], v[rows])
    p.check_attention(plan, p.new(335, 8, 1 / scale_k))


def test_values_of_very_different_size_in_one_cache():
    """A block of large values early in the sequence does not coarsen what later rows see of it."""
    p = make("gqa2")
    plan = p.cache.plan_chunk([400, 0, 0, 0])
    k, v = p.new(400, 2), p.new(400, 2)
    v[:100] *= 1000.0
    v[300:] *= 0.001
    k[:100, :, 7] = -40.0                                   # the large ones hardly weigh
    q = p.new(400, 8)
    q[..., 7] = 4.0
    p.cache.append_chunk(plan, k.cuda(), v.cuda())
    p.plain[0].append(0, k, v)
    p.check_attention(plan, q)


def test_extreme_logits_and_equal_rows():
    p = make("gqa2")
    plan = p.cache.plan_chunk([150, 20, 0, 0])
    k, v, q = p.new(170, 2, 6.0), p.new(170, 2), p.new(170, 8, 20.0)
    q[5], q[160] = 0.0, 0.0                                 # equal weights
    p.cache.append_chunk(plan, k.cuda(), v.cuda())
    p.plain[0].append(0, k[:150], v[:150])
    p.plain[1].append(0, k[150:], v[150:])
    p.check_attention(plan, q)


# ------------------------------------------------------------------ prompts

def prompt_reference(q, k, v, lens):
    at = 0
    for n in lens:
        if n:
            yield slice(at, at + n), ct.attend(ct.wide(q[at:at + n]), ct.wide(k[at:at + n]).transpose(1, 0, 2),
                                               ct.wide(v[at:at + n]).transpose(1, 0, 2), 0)
        at += n


def check_prompt(got, q, k, v, lens, what=""):
    for rows, plain in prompt_reference(q, k, v, lens):
        ct.check_attention(got[rows], *plain, rows.stop - rows.start, q.dtype, False, f"{what} rows {rows}")


@pytest.mark.parametrize("hq,hkv,d,dtype", [(2, 2, 64, FP16), (8, 2, 128, BF16), (3, 1, 128, FP16), (5, 1, 64, BF16),
                                            (4, 4, 128, BF16), (32, 4, 64, BF16), (40, 1, 128, BF16), (130, 1, 64, FP16)])
@pytest.mark.parametrize("lens", [[1], [2, 0, 1, 33], [127, 128, 129], [0, 300, 0, 70, 0], [520, 1]])
def test_prompt_attention(hq, hkv, d, dtype, lens):
    if hq // hkv > 128:
        with pytest.raises(kvq.KVQError) as e:
            kvq.plan_prompt(lens, hq, hkv, d)
        assert e.value.status == kvq.KVQ_ERR_UNSUPPORTED
        return
    gen = torch.Generator().manual_seed(sum(lens) + hq)
    total = sum(lens)
    q, k, v = (torch.randn(total, h, d, generator=gen).to(dtype) for h in (hq, hkv, hkv))
    k[..., 1] *= 6
    plan = kvq.plan_prompt(lens, hq, hkv, d)
    got = kvq.prompt_attention(plan, q.cuda(), k.cuda(), v.cuda())
    check_prompt(got, q, k, v, lens)


def test_prompt_attention_views_and_neighbours():
    """Fused-projection views inside a larger buffer whose other rows are NaN; a strided output
    whose other elements stay."""
    lens, hq, hkv, d = [100, 0, 37, 200], 8, 2, 128
    total = sum(lens)
    gen = torch.Generator().manual_seed(1)
    buf = torch.full((total + 300, hq + 2 * hkv, d), float("nan"), dtype=BF16)
    qkv = torch.randn(total, hq + 2 * hkv, d, generator=gen).to(BF16)
    buf[100:100 + total] = qkv
    dev = buf.cuda()[100:100 + total]
    out = torch.full((total + 9, hq + 3, d), 5.0, dtype=BF16, device="cuda")
    plan = kvq.plan_prompt(lens, hq, hkv, d)
    kvq.prompt_attention(plan, dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], out=out[4:4 + total, 2:2 + hq])
    check_prompt(out[4:4 + total, 2:2 + hq], qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], lens)
    out[4:4 + total, 2:2 + hq] = 5.0
    assert (out == 5.0).all()
    # head-major storage (strides swapped) and a broadcast kv head
    q, k, v = (qkv[:, a:b].transpose(0, 1).contiguous().transpose(0, 1) for a, b in ((0, 8), (8, 10), (10, 12)))
    got = kvq.prompt_attention(plan, q.cuda(), k.cuda(), v.cuda())
    check_prompt(got, q, k, v, lens, "head-major")
    one = k[:, :1].cuda().expand(total, hkv, d)
    got = kvq.prompt_attention(plan, q.cuda(), one, v.cuda())
    check_prompt(got, q, k[:, :1].expand(total, hkv, d), v, lens, "broadcast")


def test_a_sequence_with_infinities_leaves_the_others_alone():
    lens, hq, hkv, d = [70, 60, 90], 4, 2, 128
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(220, h, d, generator=gen).to(BF16) for h in (hq, hkv, hkv))
    v[70:130], k[70:130] = float("inf"), float("nan")
    plan = kvq.plan_prompt(lens, hq, hkv, d)
    got = kvq.prompt_attention(plan, q.cuda(), k.cuda(), v.cuda())
    for rows in (slice(0, 70), slice(130, 220)):
        n = rows.stop - rows.start
        check_prompt(got[rows], q[rows], k[rows], v[rows], [n])


@pytest.mark.parametrize("dtype,scale", [(BF16, 1e-18), (BF16, 1e15), (FP16, 3e-4), (FP16, 60.0)])
def test_prompt_attention_magnitudes(dtype, scale):
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(150, 4, 64, generator=gen) for _ in range(3))
    q, k, v = (q / scale).to(dtype), (k * scale).to(dtype), (v * scale).to(dtype)
    got = kvq.prompt_attention(kvq.plan_prompt([150], 4, 4, 64), q.cuda(), k.cuda(), v.cuda())
    check_prompt(got, q, k, v, [150])


def test_prompt_attention_long_and_peaked():
    """One prompt of 3001 tokens whose logits spread widely: the running maximum moves often."""
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(3001, h, 128, generator=gen) for h in (4, 1, 1))
    q = (q * torch.linspace(0.1, 6, 3001)[:, None, None]).to(BF16)
    k = (k * torch.linspace(0.5, 2, 3001)[:, None, None]).to(BF16)
    v = v.to(BF16)
    got = kvq.prompt_attention(kvq.plan_prompt([3001], 4, 1, 128), q.cuda(), k.cuda(), v.cuda())
    check_prompt(got, q, k, v, [3001])


# ------------------------------------------------------------------ together, streams, graphs

def test_prompt_then_chunks_then_decode():
    """A serving run: prompts attended exactly and stored, a mixed chunk step, a draft rejected, a
    decode step."""
    p = make("gqa2")
    rope = ct.angles(1024, 128)
    lens = [200, 1, 0, 129]
    plan, q_dev, q = p.append(lens, rope=rope, queries=True, strided=True)
    k_rot = torch.cat([p.plain[b].K.transpose(0, 1) for b in range(4)])
    v_all = torch.cat([p.plain[b].V.transpose(0, 1) for b in range(4)])
    got = kvq.prompt_attention(kvq.plan_prompt(lens, 8, 2, 128), q_dev, k_rot.cuda(), v_all.cuda())
    check_prompt(got, q, k_rot, v_all, lens)
    plan, q_dev, q = p.append([1, 140, 60, 5], rope=rope, queries=True)
    p.check_attention(plan, q, got=p.cache.chunk_attention(plan, q_dev))
    starts = [p.cache.seq_len(b) - d for b, d in enumerate((0, 0, 0, 3))]
    plan, q_dev, q = p.append([2, 1, 1, 4], starts=starts, rope=rope, queries=True)
    p.check_attention(plan, q, got=p.cache.chunk_attention(plan, q_dev))
    p.check_state()


def test_other_stream_and_reused_memory():
    p = make("gqa2")
    p.append([300, 10, 200, 1])
    q = p.new(4, 8)
    plan = p.cache.plan_chunk([1] * 4, [299, 9, 199, 0])
    dq = q.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = p.cache.chunk_attention(plan, dq, stream=side)
    side.synchronize()
    p.check_attention(plan, q, got=got)
    k, v = p.cache.read_chunk(plan, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    k2, v2 = p.cache.read_chunk(plan)
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_captured_steps_replay():
    """append + attention + prompt attention captured once; replays follow the inputs' contents."""
    p = make("gqa2")
    p.append([300, 10, 200, 1])
    plan = p.cache.plan_chunk([2, 3, 60, 1])
    k, v, q = (torch.zeros(66, h, 128, dtype=BF16, device="cuda") for h in (2, 2, 8))
    pp = kvq.plan_prompt([40, 26], 8, 2, 128)
    p.cache.reserve(2, 260)                                  # slot 2 fills a block
    kvq.prompt_attention(pp, q, k, v)
    kept = p.cache.k_residual.clone(), p.cache.v_residual.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.cache.append_chunk(plan, k, v)
        o = p.cache.chunk_attention(plan, q)
        op = kvq.prompt_attention(pp, q, k, v)
    for _ in range(3):
        hk, hv, hq = p.new(66, 2), p.new(66, 2), p.new(66, 8)
        k.copy_(hk), v.copy_(hv), q.copy_(hq)
        p.cache.k_residual.copy_(kept[0]), p.cache.v_residual.copy_(kept[1])   # as at the capture
        graph.replay()
        torch.cuda.synchronize()
        for b in range(4):
            rows = slice(plan.offsets[b], plan.offsets[b + 1])
            p.plain[b].append(plan.starts[b], hk[rows], hv[rows])
        p.check_state()
        p.check_attention(plan, hq, got=o)
        check_prompt(op, hq, hk, hv, [40, 26])


def test_repeated_calls_give_the_same_bits():
    p = make("gqa2", capacity=4096)
    p.append([3000, 700, 200, 1])
    plan = p.cache.plan_chunk([1, 4, 100, 1], [2999, 696, 100, 0])
    q = p.new(106, 8).cuda()
    a = [p.cache.chunk_attention(plan, q) for _ in range(4)]
    assert all(torch.equal(a[0], x) for x in a[1:])


# ------------------------------------------------------------------ sizes and values at the variants' edges

def fill(p, counts, make_rows):
    """Slots of tokens from make_rows(total, kv heads) -> (k, v), on both sides."""
    plan = p.cache.plan_chunk(counts)
    k, v = make_rows(plan.tokens, p.g.kv_heads)
    p.cache.append_chunk(plan, k.cuda(), v.cuda())
    for b, (s, n) in enumerate(zip(plan.starts, plan.counts)):
        if n:
            rows = slice(plan.offsets[b], plan.offsets[b + 1])
            p.plain[b].append(s, k[rows], v[rows])
    return plan


@pytest.mark.parametrize("name", ["g16", "small"])
def test_zeros_beyond_eleven_bits(name):
    """Keys and values far from 0 with little spread: code minus zero no longer fits in fp16.  Chunks
    that are unpacked in the attention kernel and chunks that are unpacked before it."""
    p = make(name)

    def rows(n, heads):
        step = torch.randint(0, 2, (2, n, heads, p.g.head_dim), generator=p.gen) * 2.0 ** -5
        k, v = (48.0 + step).to(FP16)
        k[..., ::2] *= -1                                    # logits of both signs
        return k, v

    R = p.g.residual
    fill(p, [3 * R + 5, 2 * R, R + 1] + [0] * (p.g.batch - 3), rows)
    rest = [0] * (p.g.batch - 3)
    plan = p.cache.plan_chunk([2, R, R] + rest, [3 * R + 3, R, 1] + rest)
    zeros = p.cache.k_zeros
    assert zeros.abs().max() > 1024
    p.check_attention(plan, p.new(plan.tokens, p.g.q_heads, 2.0 ** -6))
    p.cache.check_device()


@pytest.mark.parametrize("name,rows", [("gqa2", 4), ("mha4", 1), ("sym4", 3)])
def test_chunk_sizes_around_the_tiles(name, rows):
    """Chunks of one token more and less than what a tile, two tiles and the narrow form hold."""
    p = make(name, capacity=2048)
    sizes = sorted({n + e for n in (32 // rows, 128 // rows, 256 // rows) for e in (0, 1)})
    p.append([150, 7, 131, 0][:p.g.batch])
    for i in range(0, len(sizes), 2):
        plan, _, _ = p.append(([0] + sizes[i:i + 2] + [0])[:p.g.batch])
        p.check_attention(plan, what=f"{sizes[i:i + 2]}")
    p.cache.check_device()


@pytest.mark.parametrize("hq,hkv", [(128, 1), (33, 1), (66, 2), (7, 7)])
def test_chunk_attention_head_counts(hq, hkv):
    p = ct.Pair(2, hq, hkv, 64, 32, 32, 64, 2, False, BF16, 512, 64, seed=hq)
    p.append([150, 64])
    for counts in ([1, 0], [3, 1], [5, 40]):
        plan, _, _ = p.append(counts)
        p.check_attention(plan, what=str(counts))


def test_decode_steps_as_chunks():
    """Every slot's newest token: slots that hold nothing, strided queries and outputs, then slots
    that keep still, which leave the decode kernel's form."""
    p = make("gqa2")
    p.append([500, 0, 1, 127])
    fused = torch.zeros(3, 13, 128, dtype=BF16, device="cuda")
    out = torch.full((5, 11, 128), 7.0, dtype=BF16, device="cuda")
    for _ in range(3):                                       # slot 3 fills a block
        plan, _, _ = p.append([1, 0, 1, 1])
        q = p.new(3, 8)
        fused[:, 2:10] = q.cuda()
        got = p.cache.chunk_attention(plan, fused[:, 2:10], out=out[1:4, 3:])
        p.check_attention(plan, q, got=got)
    keep = out.clone()
    keep[1:4, 3:] = 7.0
    assert (keep == 7.0).all()
    plan, _, _ = p.append([1, 0, 0, 1])                      # slot 2 holds tokens and brings none
    p.check_attention(plan)
    p.cache.release(0)
    p.plain[0] = ct.PlainSlot(p.g, BF16)
    plan, _, _ = p.append([0, 0, 1, 1])
    p.check_attention(plan)
    p.cache.check_device()


def test_many_slots():
    """More slots than a warp has lanes, most without tokens."""
    p = ct.Pair(150, 2, 1, 64, 16, 16, 32, 4, False, BF16, 128, 64, seed=5)
    counts = [(b * 7) % 45 if b % 3 else 0 for b in range(150)]
    plan, _, _ = p.append(counts)
    p.check_read(plan)
    p.check_attention(plan)
    plan, _, _ = p.append([1 if b % 5 else 0 for b in range(150)])
    p.check_attention(plan)
    p.check_state()


@pytest.mark.parametrize("counts", [[2, 2, 2, 0], [20, 60, 20, 0]])
def test_a_slot_with_infinities_leaves_the_others_alone(counts):
    p = make("gqa2")
    p.append([200, 0, 50, 0])
    plan = p.cache.plan_chunk(counts)
    k, v, q = p.new(plan.tokens, 2), p.new(plan.tokens, 2), p.new(plan.tokens, 8)
    bad = slice(plan.offsets[1], plan.offsets[2])
    k[bad], v[bad], q[bad] = float("nan"), float("inf"), float("nan")
    p.cache.append_chunk(plan, k.cuda(), v.cuda())
    got = p.cache.chunk_attention(plan, q.cuda())
    for b in (0, 2):
        rows = slice(plan.offsets[b], plan.offsets[b + 1])
        p.plain[b].append(plan.starts[b], k[rows], v[rows])
        hk, hv = p.plain[b].held()
        ct.check_attention(got[rows], *ct.attend(ct.wide(q[rows]), hk, hv, plan.starts[b]), hk.shape[1], BF16, True)


def test_captured_wide_chunk_and_decode_step_replay():
    """Two graphs captured on one cache, a long chunk over a split cache and a decode step, replayed in
    turn and back to back: each keeps scratch of its own."""
    p = make("gqa2", capacity=4096)
    p.append([3000, 700, 200, 1])
    wide = p.cache.plan_chunk([100, 300, 9, 0], [2900, 400, 191, 0])
    step = p.cache.plan_chunk([1] * 4, [2999, 699, 199, 0])
    qw, qs = (torch.zeros(n, 8, 128, dtype=BF16, device="cuda") for n in (wide.tokens, 4))
    p.cache.chunk_attention(wide, qw), p.cache.chunk_attention(step, qs)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for plan, q in ((wide, qw), (step, qs)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(p.cache.chunk_attention(plan, q))
    for _ in range(2):
        hw, hs = p.new(wide.tokens, 8), p.new(4, 8)
        qw.copy_(hw), qs.copy_(hs)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        p.check_attention(wide, hw, got=outs[0])
        p.check_attention(step, hs, got=outs[1])
    eager = p.cache.chunk_attention(wide, qw)
    assert torch.equal(eager, outs[0])


def test_wide_chunks_on_two_streams():
    """Attention calls of two caches that may run at once."""
    pairs = [make("gqa2", capacity=2048, seed=s) for s in (1, 2)]
    jobs = []
    for p in pairs:
        p.append([900, 300, 40, 0])
        plan, _, _ = p.append([200, 90, 1, 3])
        q = p.new(plan.tokens, 8)
        jobs.append((p, plan, q, q.cuda(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[p.cache.chunk_attention(plan, dq, stream=s) for p, plan, _, dq, s in jobs] for _ in range(4)]
    torch.cuda.synchronize()
    for got in outs:
        for (p, plan, q, _, _), o in zip(jobs, got):
            p.check_attention(plan, q, got=o)


def test_repeated_wide_calls_give_the_same_bits():
    p = make("gqa2", capacity=4096)
    p.append([3500, 700, 200, 1])
    plan = p.cache.plan_chunk([500, 90, 1, 0], [3000, 600, 199, 0])
    q = p.new(plan.tokens, 8).cuda()
    a = [p.cache.chunk_attention(plan, q) for _ in range(4)]
    assert all(torch.equal(a[0], x) for x in a[1:])


def test_status_of_prompts_and_plans():
    plan = kvq.plan_prompt([40, 9], 8, 2, 128)
    q, k, v = (torch.randn(49, h, 128, device="cuda").to(BF16) for h in (8, 2, 2))
    kvq.prompt_attention(plan, q, k, v)
    plan.check_device()
    items = plan.table.clone()
    plan.table[-4] = 7                                       # the last piece's slot: there are two
    kvq.prompt_attention(plan, q, k, v)
    with pytest.raises(kvq.KVQError) as e:
        plan.check_device()
    assert e.value.status == kvq.KVQ_ERR_DEVICE_CHECK
    plan.check_device()                                      # cleared
    plan.table.copy_(items)
    p = make("gqa2")
    p.append([70, 0, 3, 0])
    chunk = p.cache.plan_chunk([2, 0, 3, 0], [68, 0, 0, 0])
    with pytest.raises(ValueError):
        chunk.check_device()
    with pytest.raises(kvq.KVQError):
        kvq.prompt_attention(chunk, q[:5], k[:5], v[:5])
    with pytest.raises(kvq.KVQError):
        p.cache.chunk_attention(plan, q)
    keep, chunk.device = chunk.device, torch.device("cuda", 99)
    for call in (lambda: p.cache.chunk_attention(chunk, q[:5]), lambda: p.cache.read_chunk(chunk),
                 lambda: p.cache.append_chunk(chunk, k[:5], v[:5])):
        with pytest.raises(ValueError):
            call()
    chunk.device = keep
    p.check_attention(chunk)


# ------------------------------------------------------------------ refusals and bad tables

def test_refused_calls_change_nothing():
    p = make("gqa2", capacity=256)
    p.append([200, 10, 0, 1])
    lib = kvq.load()
    k = p.new(100, 2).cuda()

    def refused(status, counts, starts=None, **kw):
        plan = p.cache.plan_chunk(counts, starts)
        n = plan.tokens
        with pytest.raises(kvq.KVQError) as e:
            p.cache.append_chunk(plan, k[:n], k[:n], **kw)
        assert e.value.status == status and lib.kvq_last_error()

    refused(kvq.KVQ_ERR_STATE, [1, 0, 0, 0], [201, 0, 0, 0])
    refused(kvq.KVQ_ERR_STATE, [0, 0, 2, 0], [0, 0, 1, 0])            # a gap before an empty slot's tokens
    big = p.new(256, 2).cuda()
    plan = p.cache.plan_chunk([200, 0, 0, 0])
    with pytest.raises(kvq.KVQError) as e:
        p.cache.append_chunk(plan, big[:200], big[:200])
    assert e.value.status == kvq.KVQ_ERR_CAPACITY
    short = kvq.Rope(*(x.cuda() for x in ct.angles(50, 128)))
    refused(kvq.KVQ_ERR_INVALID_ARG, [0, 50, 0, 0], rope=short)
    plan = p.cache.plan_chunk([1, 0, 0, 0], [200, 0, 0, 0])          # not appended yet
    with pytest.raises(kvq.KVQError) as e:
        p.cache.chunk_attention(plan, p.new(1, 8).cuda())
    assert e.value.status == kvq.KVQ_ERR_STATE
    with pytest.raises(kvq.KVQError) as e:
        p.cache.read_chunk(plan)
    assert e.value.status == kvq.KVQ_ERR_STATE
    other = make("mha4").cache.plan_chunk([1, 0, 0, 0])
    with pytest.raises((kvq.KVQError, ValueError)):
        p.cache.append_chunk(other, k[:1], k[:1])
    with pytest.raises(TypeError):
        p.cache.append_chunk(p.cache.plan_chunk([1, 0, 0, 0]), k[:1].half(), k[:1].half())
    with pytest.raises(ValueError):
        p.cache.chunk_attention(plan, p.new(2, 8).cuda())
    p.check_state("after refusals")


def test_an_exhausted_pool_refuses_and_keeps_the_state():
    p = make("gqa2", num_pages=2)
    p.append([128, 0, 0, 0])
    k = p.new(300, 2).cuda()
    with pytest.raises(kvq.KVQError) as e:
        p.cache.append_chunk(p.cache.plan_chunk([0, 256, 0, 0]), k[:256], k[:256])
    assert e.value.status == kvq.KVQ_ERR_CAPACITY
    assert len(p.cache.free_pages) == 1
    with pytest.raises(kvq.KVQError) as e:
        p.cache.reserve(1, 256)
    assert e.value.status == kvq.KVQ_ERR_CAPACITY and len(p.cache.free_pages) == 1
    p.append([100, 0, 0, 0])
    p.check_state()


def test_a_bad_page_is_reported_and_not_followed():
    p = make("gqa2")
    p.append([300, 200, 0, 0])
    keep = p.cache.page_table.clone()
    p.cache.page_table[0, 0], p.cache.page_table[1, 0] = 10 ** 6, -5
    plan = p.cache.plan_chunk([5, 7, 0, 0], [295, 193, 0, 0])
    p.cache.chunk_attention(plan, p.new(12, 8).cuda())
    with pytest.raises(kvq.KVQError) as e:
        p.cache.check_device()
    assert e.value.status == kvq.KVQ_ERR_DEVICE_CHECK
    p.cache.page_table.copy_(keep)
    p.check_attention(plan)
    p.cache.check_device()
