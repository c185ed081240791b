"""The chunk planner and its refusals on the host, without a device."""
import ctypes
import random

import pytest

from bit_kv_cache_22_b200 import kvq


def config(batch=3, hq=8, hkv=2, R=128, page=128, capacity=1024):
    geom = kvq.make_config(batch, hq, hkv, 128, 32, 32, R, 2, False, kvq.KVQ_BF16, capacity)
    return kvq.PagedConfig(geom, page, 16)


def plan(cfg, counts, starts, room=None, sms=148):
    n = len(counts)
    c, s = (ctypes.c_int32 * n)(*counts), (ctypes.c_int32 * n)(*starts)
    out = kvq.Chunk()
    lib = kvq.load()
    st = lib.kvq_plan_chunk(ctypes.byref(cfg), c, s, sms, ctypes.byref(out), None, 0)
    if st != kvq.KVQ_OK:
        return st, None, None
    words = out.table_bytes // 4
    table = (ctypes.c_int32 * (words + 1))(*([77] * (words + 1)))
    st = lib.kvq_plan_chunk(ctypes.byref(cfg), c, s, sms, ctypes.byref(out), table,
                            out.table_bytes if room is None else room)
    assert table[words] == 77                       # nothing past the end
    return st, out, list(table)


def test_table_of_random_plans():
    rng = random.Random(1)
    for _ in range(200):
        B, R = rng.randint(1, 9), rng.choice([32, 128, 256])
        cfg = config(batch=B, R=R, page=256, capacity=1024)
        counts = [rng.choice([0, 1, rng.randint(0, 700)]) for _ in range(B)]
        starts = [rng.randint(0, 500) for _ in range(B)]
        st, out, t = plan(cfg, counts, starts)
        assert st == kvq.KVQ_OK and out.tokens == sum(counts)
        assert t[:B + 1] == [sum(counts[:b]) for b in range(B + 1)]
        assert t[B + 1:2 * B + 1] == starts
        tiles = [(s + n + 15) // 16 - s // 16 if n else 0 for s, n in zip(starts, counts)]
        assert t[2 * B + 1:3 * B + 2] == [sum(tiles[:b]) for b in range(B + 1)] and out.read_tiles == sum(tiles)
        blocks = [(b, i) for b in range(B) if counts[b]
                  for i in range(starts[b] // R, (starts[b] + counts[b]) // R)]
        wide = [4 * n > 32 for n in counts]         # 4 query heads a kv head: more than 32 query rows
        kv = [-(-(s + n) // 128) * w for s, n, w in zip(starts, counts, wide)]
        q = [-(-n // 32) * w for n, w in zip(counts, wide)]
        assert t[3 * B + 2:4 * B + 3] == [sum(kv[:b]) for b in range(B + 1)] and out.kv_tiles == sum(kv)
        assert t[4 * B + 3:5 * B + 4] == [sum(q[:b]) for b in range(B + 1)] and out.q_tiles == sum(q)
        at = 5 * B + 4
        assert [tuple(t[at + 2 * i:at + 2 * i + 2]) for i in range(out.blocks)] == blocks and out.blocks == len(blocks)
        at = -(-(at + 2 * out.blocks) // 4) * 4
        items = [tuple(t[i:i + 4]) for i in range(at, at + 4 * out.items, 4)]
        merges = [tuple(t[i:i + 4]) for i in range(at + 4 * out.items, len(t) - 1, 4)]
        pieces = {}
        for b, i, z, part in items:                 # every piece whole, its splits numbered from 0
            assert z >> 16 >= 1 and z & 0xffff == len(pieces.setdefault((b, i, z >> 16, part), []))
            pieces[b, i, z >> 16, part].append(z & 0xffff)
        assert sorted(k[:2] for k in pieces) == [(b, i) for b in range(B) for i in range(0, counts[b], 64)]
        assert all(len(v) == k[2] for k, v in pieces.items())
        assert merges == [k for k in pieces if k[2] > 1] and len(merges) == out.merges
        part = 0                                    # partial results laid end to end
        for b, i, n, at_part in merges:
            assert at_part == part
            part += n * (1 if counts[b] - i <= 32 else 2)
        assert part == out.part_tiles
        room = 2 * (part * 128 * 130 * 4 + sum(kv) * (2 * 32768 + 32) + sum(q) * (32768 + 512))
        if max(counts) <= 1:                        # single tokens may take the decode kernel
            assert out.workspace >= room
        else:
            assert out.workspace == room
        n_wide = sum(n for b, _, n, _ in pieces if wide[b])
        assert out.wide_items == n_wide and all(wide[i[0]] == (k < n_wide) for k, i in enumerate(items))
        share = [-(-(starts[b] + min(i + 64, counts[b])) // 128) / n for b, i, n, _ in pieces]
        of_wide = [wide[b] for b, _, _, _ in pieces]
        for w in (True, False):                     # the longest first, the wide slots' before the others
            part = [x for x, y in zip(share, of_wide) if y == w]
            assert part == sorted(part, reverse=True)


def test_a_long_sequence_is_split_over_the_gpu():
    cfg = config(batch=1, hq=8, hkv=2, capacity=131072)
    st, out, _ = plan(cfg, [1], [130000])
    assert st == kvq.KVQ_OK and out.merges == 1 and out.items * 2 > 100
    st, out, _ = plan(cfg, [1], [130000], sms=1)
    assert st == kvq.KVQ_OK and out.items * 2 <= 4 * 2
    assert plan(cfg, [1], [5], sms=0)[0] == kvq.KVQ_ERR_INVALID_ARG


@pytest.mark.parametrize("counts,starts", [([-1, 0, 0], [0, 0, 0]), ([1, 0, 0], [-1, 0, 0]),
                                           ([2, 0, 0], [2 ** 31 - 2, 0, 0]), ([2 ** 30] * 3, [0] * 3)])
def test_refused_plans(counts, starts):
    assert plan(config(), counts, starts)[0] == kvq.KVQ_ERR_INVALID_ARG
    assert kvq.load().kvq_last_error()


def test_a_short_table_is_refused():
    assert plan(config(), [5, 1, 300], [0, 0, 0], room=8)[0] == kvq.KVQ_ERR_INVALID_ARG


def test_prompt_plans():
    lib = kvq.load()
    out = kvq.Chunk()
    c = (ctypes.c_int32 * 2)(5, 7)
    ok = [2, 8, 2, 128]
    assert lib.kvq_plan_prompt(*ok, c, ctypes.byref(out), None, 0) == kvq.KVQ_OK
    assert out.tokens == 12 and out.residual == 0 and out.blocks == 0
    for bad, status in (([0, 8, 2, 128], kvq.KVQ_ERR_INVALID_ARG), ([2, 8, 3, 128], kvq.KVQ_ERR_INVALID_ARG),
                        ([2, 8, 2, 96], kvq.KVQ_ERR_UNSUPPORTED), ([2, 129, 1, 128], kvq.KVQ_ERR_UNSUPPORTED)):
        assert lib.kvq_plan_prompt(*bad, c, ctypes.byref(out), None, 0) == status, bad
    assert lib.kvq_plan_prompt(*ok, None, ctypes.byref(out), None, 0) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_plan_chunk(None, c, c, 148, ctypes.byref(out), None, 0) == kvq.KVQ_ERR_INVALID_ARG


def test_calls_refuse_bad_arguments_before_any_launch():
    lib = kvq.load()
    c = (ctypes.c_int32 * 1)(4)
    out = kvq.Chunk()
    assert lib.kvq_plan_prompt(1, 4, 2, 128, c, ctypes.byref(out), None, 0) == kvq.KVQ_OK
    fake = 1 << 20                                  # aligned, never followed: every call below is refused
    good = kvq.Rows(fake, 512, 128)
    r = ctypes.byref

    def attend(p, dtype=kvq.KVQ_BF16, q=good, o=good):
        return lib.kvq_prompt_attention(r(p), dtype, r(q), r(good), r(good), r(o), None, None)

    assert attend(out) == kvq.KVQ_ERR_INVALID_ARG and b"table" in lib.kvq_last_error()
    out.table = fake
    assert attend(out, dtype=9) == kvq.KVQ_ERR_INVALID_ARG
    for bad in (kvq.Rows(None, 512, 128), kvq.Rows(fake + 2, 512, 128), kvq.Rows(fake, 500, 128),
                kvq.Rows(fake, 512, -128), kvq.Rows(fake, 512, 4), kvq.Rows(fake, 0, 128), kvq.Rows(fake, 512, 0)):
        assert attend(out, q=bad) == kvq.KVQ_ERR_INVALID_ARG
        assert attend(out, o=bad) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_prompt_attention(None, 0, r(good), r(good), r(good), r(good), None, None) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_paged_append_chunk(None, r(out), r(good), r(good), None, None, None, None) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_paged_read_chunk(None, r(out), r(good), r(good), None) == kvq.KVQ_ERR_INVALID_ARG
    assert lib.kvq_paged_chunk_attention(None, r(out), r(good), r(good), None, 0, None) == kvq.KVQ_ERR_INVALID_ARG
    none = (ctypes.c_int32 * 1)(0)                  # nothing to do: no launch, no device
    assert lib.kvq_plan_prompt(1, 4, 2, 128, none, r(out), None, 0) == kvq.KVQ_OK
    out.table = fake
    assert attend(out) == kvq.KVQ_OK
