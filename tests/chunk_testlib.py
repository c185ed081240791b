"""Plain 64-bit forms of the chunk operators (prompt attention, rotated append, read-back, chunk
attention), written from the formulas on the oracle's quantiser, and how far a result may be off."""
from __future__ import annotations

import numpy as np
import torch

from bit_kv_cache_22_b200 import kvq
from bit_kv_cache_22_b200 import workloads as wl


def code_of(dtype):
    return wl.FP16 if dtype == torch.float16 else wl.BF16


def bits_of(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def wide(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def rotate(x: torch.Tensor, positions, cos, sin, pairs: bool) -> torch.Tensor:
    """x [n, h, d] e on the CPU, turned by its rows' positions: fp32, one rounding an operation."""
    half = cos.shape[1]
    c, s = cos.cpu()[positions][:, None], sin.cpu()[positions][:, None]
    y = x.float().clone()
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if pairs else (y[..., :half], y[..., half:2 * half])
    a0, b0 = a.clone(), b.clone()
    a.copy_((a0 * c) - (b0 * s))
    b.copy_((b0 * c) + (a0 * s))
    return y.to(x.dtype)


def angles(positions: int, rot: int, device="cpu"):
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return a.cos().float().to(device), a.sin().float().to(device)


class PlainSlot:
    """One slot's tokens as elements [Hkv, n, d]; what the cache holds of them follows from n."""

    def __init__(self, geom, dtype):
        self.g, self.dtype = geom, dtype
        self.K = torch.empty(geom.kv_heads, 0, geom.head_dim, dtype=dtype)
        self.V = self.K.clone()

    def append(self, start, k, v):
        """k, v [n, Hkv, d] (CPU, rotated) become tokens start ...; tokens from start on are dropped."""
        self.K = torch.cat([self.K[:, :start], k.transpose(0, 1)], 1)
        self.V = torch.cat([self.V[:, :start], v.transpose(0, 1)], 1)

    def quantized(self):
        import oracle
        g = self.g
        tq = self.K.shape[1] // g.residual * g.residual
        return tq, oracle.quantize_kv(bits_of(self.K[:, :tq]), bits_of(self.V[:, :tq]), code_of(self.dtype),
                                      g.group_k, g.group_v, g.bits, bool(g.symmetric))

    def packed(self):
        import oracle
        tq, q = self.quantized()
        g = self.g
        return tq, dict(Kc=oracle.pack(q["Kq"], g.bits, False), Vc=oracle.pack(q["Vq"], g.bits, True), Ks=q["Ks"],
                        Kz=q["Kz"], Vs=q["Vs"], Vz=q["Vz"])

    def held(self):
        """[Hkv, n, d] keys and values as the cache holds them, fp64."""
        tq, q = self.quantized()
        g = self.g
        off = 1 << (g.bits - 1)

        def deq(code, s, z, token_group, channel_group):
            s = np.repeat(np.repeat(s.astype(np.float64), token_group, 1), channel_group, 2)
            z = off if g.symmetric else np.repeat(np.repeat(z.astype(np.float64), token_group, 1), channel_group, 2)
            return (code.astype(np.float64) - z) * s

        k, v = wide(self.K), wide(self.V)
        if tq:
            k[:, :tq] = deq(q["Kq"], q["Ks"], q["Kz"], g.group_k, 1)
            v[:, :tq] = deq(q["Vq"], q["Vs"], q["Vz"], 1, g.group_v)
        return k, v


def attend(q, k, v, first: int):
    """q [n, Hq, d], k, v [Hkv, L, d] fp64; row i sees tokens 0 .. first + i.  Returns o [n, Hq, d],
    A = sum_j p_j |v_j| of the same shape, S = max_j sum_c |q_c k_jc| / sqrt(d) [n, Hq, 1] and max |v|."""
    n, hq, d = q.shape
    hkv = k.shape[0]
    o, A, S = np.zeros_like(q), np.zeros_like(q), np.zeros((n, hq, 1))
    seen = np.arange(k.shape[1])[None] <= first + np.arange(n)[:, None]
    for h in range(hq):
        kh, vh = k[h // (hq // hkv)], v[h // (hq // hkv)]
        y = np.where(seen, q[:, h] @ kh.T / np.sqrt(d), -np.inf)
        p = np.exp(y - y.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        o[:, h], A[:, h] = p @ vh, p @ np.abs(vh)
        S[:, h] = np.where(seen, np.abs(q[:, h]) @ np.abs(kh).T, 0).max(1, keepdims=True) / np.sqrt(d)
    return o, A, S, np.abs(v).max()


def attention_bound(o, A, S, vmax, tokens, d, dtype, cache: bool):
    """How far an output may be off, elementwise (u = half a step).

    The output is rounded once: u(e) |o|, and in fp16 below 2^-14 by up to 2^-25 whatever its size.
    Weights are rounded to 16 bits before they meet the values: u A (prompt: e; cache: fp16,
    u = 2^-11); an fp16 weight below 2^-14 by up to 2^-25, for each token: tokens 2^-25 max|v| (the
    weights' sum is at least 1 before they are normalised).  Over the cache, keys and values are
    rounded to fp16 too: the values' rounding moves the sum by u A, the keys' moves each logit by at
    most u S, so each weight by a factor within exp(2 u S): the numerator and the sum of weights,
    2 u S A.  fp32: a logit's d products and sums and its scaling are off by at most (d + 4) 2^-24 S
    and the subtraction of the maximum by 2^-24 (2 S), again twice; exp2 by 2^-21 relative; sums over
    the tokens by tokens 2^-24, numerator and denominator."""
    u = half_step(dtype)
    w = 2.0 ** -11 if cache else u
    rel = w + 2 * (d + 8) * 2.0 ** -24 * S + 2.0 ** -20 + 2 * tokens * 2.0 ** -24
    if cache:
        rel = rel + w + 2 * w * S
    small = 0.0
    if cache or dtype == torch.float16:
        small += tokens * 2.0 ** -25 * vmax
    if dtype == torch.float16:
        small += 2.0 ** -25
    return u * np.abs(o) + (1 + u) * A * rel + small


def check_attention(got, o, A, S, vmax, tokens, dtype, cache, what=""):
    got = wide(got)
    assert got.shape == o.shape
    assert np.isfinite(got).all(), f"{what}: not finite"
    err, lim = np.abs(got - o), attention_bound(o, A, S, vmax, tokens, o.shape[-1], dtype, cache)
    bad = err > lim
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}, "
                           f"worst {np.max(err / lim):.2f} of the bound")
    # and as a whole: the roundings are independent, so the norm is far inside the worst case
    if np.linalg.norm(o) > 0:
        rel = np.linalg.norm(got - o) / np.linalg.norm(A)
        assert rel < 4 * half_step(dtype) + (2.0 ** -11 * (4 + 4 * S.max()) if cache else 0) + \
            (2.0 ** -25 * np.sqrt(o.size) / np.linalg.norm(A) if dtype == torch.float16 else 0), f"{what}: rel {rel:.2e}"


def gather_packed(cache: kvq.PagedKVQCache, b: int, tq: int) -> dict:
    """Slot b's quantized tokens gathered from its pages, in the oracle's array shapes."""
    g = cache.geom
    n = -(-tq // cache.page_tokens)
    rows = [pg * g.kv_heads + h for h in range(g.kv_heads) for pg in cache.pages[b][:n]]

    def gather(t, keep):
        x = t[rows].reshape(g.kv_heads, n, *t.shape[1:])
        return x.reshape(g.kv_heads, n * t.shape[1], *t.shape[2:])[:, :keep].cpu().numpy()

    words = tq * g.head_dim * g.bits // 32
    out = dict(Kc=gather(cache.k_codes, words).view(np.uint32), Vc=gather(cache.v_codes, words).view(np.uint32),
               Ks=gather(cache.k_scales, tq // g.group_k), Vs=gather(cache.v_scales, tq))
    if cache.k_zeros is not None:
        out["Kz"], out["Vz"] = gather(cache.k_zeros, tq // g.group_k), gather(cache.v_zeros, tq)
    return out


class Pair:
    """A paged cache on the GPU and its plain slots, fed the same chunks."""

    def __init__(self, slots, hq, hkv, d, G, Gv, R, bits, sym=False, dtype=torch.bfloat16, capacity=1024, page=128,
                 seed=0, num_pages=None):
        self.cache = kvq.PagedKVQCache(slots, hq, hkv, d, G, Gv, R, bits, sym, dtype, capacity, page, num_pages)
        np.random.default_rng(seed).shuffle(self.cache.free_pages)
        self.g, self.dtype = self.cache.geom, dtype
        self.plain = [PlainSlot(self.g, dtype) for _ in range(slots)]
        self.gen = torch.Generator().manual_seed(seed)

    def new(self, tokens, heads, scale=1.0):
        return (torch.randn(tokens, heads, self.g.head_dim, generator=self.gen) * scale).to(self.dtype)

    def append(self, counts, starts=None, rope=None, pairs=False, strided=False, queries=False, stream=None):
        """rope: (cos, sin) on the CPU.  Returns (plan, rotated queries on the GPU, what they should be)."""
        plan = self.cache.plan_chunk(counts, starts)
        g = self.g
        k, v, q = (self.new(plan.tokens, g.kv_heads), self.new(plan.tokens, g.kv_heads, 0.5),
                   self.new(plan.tokens, g.q_heads))
        k[..., 3] *= 8
        if strided:                                  # views of one fused projection
            fused = torch.cat([q, k, v], 1).cuda()
            dq, dk, dv = fused[:, :g.q_heads], fused[:, g.q_heads:g.q_heads + g.kv_heads], fused[:, g.q_heads + g.kv_heads:]
        else:
            dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
        positions = [s + i for s, n in zip(plan.starts, plan.counts) for i in range(n)]
        handle = None
        if rope is not None:
            handle = kvq.Rope(rope[0].cuda(), rope[1].cuda(), interleaved=pairs)
            k, q = rotate(k, positions, *rope, pairs), rotate(q, positions, *rope, pairs)
        got = self.cache.append_chunk(plan, dk, dv, handle, dq if queries else None, stream=stream)
        for b, (s, n) in enumerate(zip(plan.starts, plan.counts)):
            if n:
                self.plain[b].append(s, k[plan.offsets[b]:plan.offsets[b + 1]], v[plan.offsets[b]:plan.offsets[b + 1]])
        return plan, got, q

    def check_state(self, what=""):
        import kvq_testlib as tl
        g, c = self.g, self.cache
        for b, p in enumerate(self.plain):
            n = p.K.shape[1]
            assert c.seq_len(b) in (n, -1 if n == 0 else n), f"{what} slot {b}"
            tq, packed = p.packed() if n >= g.residual else (0, None)
            if tq:
                tl.assert_codes_equal(gather_packed(c, b, tq), packed, bool(g.symmetric))
            for res, x in ((c.k_residual, p.K), (c.v_residual, p.V)):
                rows = res.view(g.batch, g.kv_heads, g.residual, g.head_dim)[b, :, :n - tq].cpu()
                assert torch.equal(rows.view(torch.int16), x[:, tq:].contiguous().view(torch.int16)), f"{what} slot {b}"
        c.check_device()

    def check_read(self, plan, what=""):
        k, v = self.cache.read_chunk(plan)
        for b, (s, n) in enumerate(zip(plan.starts, plan.counts)):
            if n:
                hk, hv = self.plain[b].held()
                for got, want in ((k, hk), (v, hv)):
                    x = torch.from_numpy(want[:, s:s + n].transpose(1, 0, 2).copy()).float().to(self.dtype)
                    assert torch.equal(got[plan.offsets[b]:plan.offsets[b + 1]].cpu(), x), f"{what} slot {b}"

    def check_attention(self, plan, q=None, what="", out=None, got=None):
        if q is None:
            q = self.new(plan.tokens, self.g.q_heads)
        if got is None:
            got = self.cache.chunk_attention(plan, q.cuda(), out=out)
        for b, (s, n) in enumerate(zip(plan.starts, plan.counts)):
            if n:
                k, v = self.plain[b].held()
                rows = slice(plan.offsets[b], plan.offsets[b + 1])
                check_attention(got[rows], *attend(wide(q[rows]), k, v, s), k.shape[1], self.dtype, True,
                                f"{what} slot {b}")
        return got
