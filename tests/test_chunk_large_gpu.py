"""The chunk operators at lengths and sizes beyond the other tests', against the plain 64-bit forms
(chunk_testlib) on some of their rows; and the two kernels that answer single tokens, compared."""
import pytest
import torch

from bit_kv_cache_22_b200 import kvq

import chunk_testlib as ct

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

FP16, BF16 = torch.float16, torch.bfloat16


def rows_of_prompt(got, q, k, v, first, count, dtype, what):
    """Rows first .. first + count - 1 of a prompt whose keys and values are k, v [tokens, Hkv, d]."""
    end = first + count
    plain = ct.attend(ct.wide(q[first:end]), ct.wide(k[:end]).transpose(1, 0, 2), ct.wide(v[:end]).transpose(1, 0, 2), first)
    ct.check_attention(got[first:end], *plain, end, dtype, False, what)


@pytest.mark.parametrize("hq,hkv,d,dtype", [(4, 1, 128, BF16), (2, 2, 64, FP16)])
def test_a_prompt_of_40000_tokens(hq, hkv, d, dtype):
    n = 40001
    gen = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(n, h, d, generator=gen).to(dtype) for h in (hq, hkv, hkv))
    plan = kvq.plan_prompt([n], hq, hkv, d)
    got = kvq.prompt_attention(plan, q.cuda(), k.cuda(), v.cuda())
    plan.check_device()
    for first in (0, 127, 16380, 32760, n - 20):
        rows_of_prompt(got, q, k, v, first, 20, dtype, f"from {first}")


@pytest.mark.parametrize("dtype,bits", [(BF16, 2), (FP16, 4)])
def test_a_cache_of_100000_tokens(dtype, bits):
    """Single tokens, drafts and a long chunk at its end, and queries in its middle."""
    p = ct.Pair(2, 4, 1, 128, 32, 32, 128, bits, False, dtype, 101 * 1024, 128)
    p.append([100000, 70])
    for counts in ([1, 1], [3, 2], [300, 40]):
        plan, _, _ = p.append(counts)
        p.check_attention(plan, what=str(counts))
    p.check_read(p.cache.plan_chunk([500, 0], [99700, 0]))
    p.check_attention(p.cache.plan_chunk([40, 0], [65520, 0]))
    p.check_attention(p.cache.plan_chunk([4, 0], [65534, 0]))
    p.cache.check_device()


def test_packed_rows_beyond_31_bits_of_elements():
    """540 sequences of 1000 tokens, 32 query heads: 2.2e9 elements of queries, and more bytes of operand
    tiles.  The first and the last sequences against their formulas."""
    slots, n, hq, hkv, d = 540, 1000, 32, 8, 128
    total = slots * n
    assert total * hq * d > 2 ** 31
    gen = torch.Generator("cuda").manual_seed(8)

    def new(heads):
        x = torch.empty(total, heads, d, dtype=BF16, device="cuda")
        for i in range(0, total, 1 << 16):
            part = x[i:i + (1 << 16)]
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
        return x

    q, k, v = new(hq), new(hkv), new(hkv)
    plan = kvq.plan_prompt([n] * slots, hq, hkv, d)
    got = kvq.prompt_attention(plan, q, k, v)
    plan.check_device()
    for b in (0, slots - 1):
        rows = slice(b * n, b * n + n)
        x = [t[rows].cpu() for t in (q, k, v)]
        rows_of_prompt(got[rows].cpu(), *x, n - 30, 30, BF16, f"prompt {b}")
    del got
    cache = kvq.PagedKVQCache(slots, hq, hkv, d, 32, 32, 128, 2, False, BF16, 1024, 128)
    cos, sin = ct.angles(1024, 128)
    plan = cache.plan_chunk([n] * slots)
    turned = cache.append_chunk(plan, k, v, kvq.Rope(cos.cuda(), sin.cuda()), q)
    k_read, v_read = cache.read_chunk(plan)
    out = cache.chunk_attention(plan, turned)
    cache.check_device()
    for b in (0, slots - 1):
        rows = slice(b * n, b * n + n)
        kr, qr = (ct.rotate(t[rows].cpu(), list(range(n)), cos, sin, False) for t in (k, q))
        assert torch.equal(turned[rows].cpu(), qr)
        plain = ct.PlainSlot(cache.geom, BF16)
        plain.append(0, kr, v[rows].cpu())
        hk, hv = plain.held()
        for have, want in ((k_read, hk), (v_read, hv)):
            assert torch.equal(have[rows].cpu(), torch.from_numpy(want.transpose(1, 0, 2).copy()).float().to(BF16))
        last = slice(b * n + n - 30, b * n + n)
        ct.check_attention(out[last], *ct.attend(ct.wide(qr[n - 30:]), hk, hv, n - 30), n, BF16, True, f"slot {b}")


@pytest.mark.parametrize("name", ["G32", "G128"])
def test_decode_kernel_and_narrow_kernel_agree(name):
    """A step of single newest tokens takes the decode kernel; the same rows in a chunk that a slot sits
    out take the narrow attention kernel.  Both within the bound of their own roundings."""
    group = {"G32": 32, "G128": 128}[name]
    p = ct.Pair(4, 8, 2, 128, group, 32, 128, 2, False, BF16, 2048, 128, seed=group)
    p.append([1500, 129, 1, 77])
    q = p.new(4, 8)
    step = p.cache.plan_chunk([1] * 4, [1499, 128, 0, 76])
    launches = kvq.kernel_launches()
    a = p.check_attention(step, q)
    decode = kvq.kernel_launches() - launches
    part = p.cache.plan_chunk([1, 1, 0, 1], [1499, 128, 0, 76])
    keep = [0, 1, 3]
    launches = kvq.kernel_launches()
    b = p.check_attention(part, q[keep])
    assert (decode, kvq.kernel_launches() - launches) == (2, 1 + (part.chunk.merges > 0))
    assert not torch.equal(a[keep], b)              # kernels of their own
    k, v = zip(*(p.plain[s].held() for s in keep))
    for i, s in enumerate(keep):
        o, A, S, vmax = ct.attend(ct.wide(q[s:s + 1]), k[i], v[i], step.starts[s])
        lim = 2 * ct.attention_bound(o, A, S, vmax, k[i].shape[1], 128, BF16, True)
        assert (abs(ct.wide(a[s:s + 1]) - ct.wide(b[i:i + 1])) <= lim).all()
