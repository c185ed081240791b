"""The serving operators on new tokens, as cases that can be timed and checked.

Three operators on `counts[b]` new tokens of each of B sequences (packed one after the
other, token-major, the way a projection's output arrives):

* ``prompt``: causal attention over whole prompts of different lengths, grouped heads, keys
  and values in fp16 / bf16;
* ``chunk``: attention of the newest tokens of every slot over the paged low-bit cache that
  already holds them (a token at position p sees tokens 0 .. p);
* ``store``: the new tokens' keys rotated by position and stored, with the values, in the
  paged cache (whole blocks of R tokens quantized, the rest kept as they are), the queries
  rotated on the way; then what the cache holds for those tokens, read back.

Every case names its geometry, its quantiser and the ranges its lengths are drawn from; the
lengths follow from the case alone, the tensors from the seed.  The plain forms are
elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

_QUANT = {   # bits, symmetric, G, Gv, R of the workloads this library is measured on
    "tiny": (2, False, 32, 32, 32),
    "llama7b": (4, False, 128, 128, 128),
    "gqa8b": (2, False, 32, 32, 128),
    "stream4sym": (4, True, 32, 32, 128),
}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a handful of short prompts, one empty and one of a single token: launch latency counts
        dict(name="prompt_short", op="prompt", dtype="fp16", hq=2, hkv=2, d=64, slots=5, clo=0, chi=160, mix=3),
        # a serving batch's prompts of mixed lengths, packed
        dict(name="prompt_mixed", op="prompt", dtype="bf16", hq=32, hkv=8, d=128, slots=12, clo=32, chi=2048, mix=1),
        # one long prompt, grouped heads
        dict(name="prompt_8192", op="prompt", dtype="bf16", hq=32, hkv=8, d=128, slots=1, clo=8192, chi=8192, mix=0),
        # two prompts, as many kv heads as query heads, fp16
        dict(name="prompt_mha_4096", op="prompt", dtype="fp16", hq=32, hkv=32, d=128, slots=2, clo=4096, chi=4096,
             mix=0),
        # a few drafted tokens verified on a short cache: the smallest call
        dict(name="chunk_draft", op="chunk", dtype="fp16", quant="tiny", hq=2, hkv=2, d=64, slots=3, page=64, lo=100,
             hi=400, clo=1, chi=6, mix=1),
        # one new token for each of 32 sequences of very different lengths (a decode step)
        dict(name="chunk_decode", op="chunk", dtype="bf16", quant="gqa8b", hq=32, hkv=8, d=128, slots=32, page=128,
             lo=512, hi=15872, clo=1, chi=1, mix=5),
        # chunked prefill of a mixed batch, one kv head per query head, 4-bit groups of 128
        dict(name="chunk_mixed", op="chunk", dtype="bf16", quant="llama7b", hq=32, hkv=32, d=128, slots=6, page=256,
             lo=300, hi=4096, clo=17, chi=700, mix=7),
        # a 2048-token chunk of one very long sequence
        dict(name="chunk_long", op="chunk", dtype="bf16", quant="gqa8b", hq=32, hkv=8, d=128, slots=1, page=128,
             lo=126976, hi=126976, clo=2048, chi=2048, mix=0),
        # one new token for each of 32 sequences, between two flushes
        dict(name="store_token", op="store", dtype="bf16", quant="gqa8b", hq=32, hkv=8, d=128, slots=32, page=128,
             lo=512, hi=8192, clo=1, chi=1, rot=128, pairs=False, mix=4),
        # four whole prompts into empty slots, 2-bit
        dict(name="store_prompt", op="store", dtype="bf16", quant="gqa8b", hq=32, hkv=8, d=128, slots=4, page=128,
             lo=0, hi=0, clo=8192, chi=8192, rot=128, pairs=False, mix=0),
        # the next chunks of a mixed batch, symmetric 4-bit, neighbouring channels rotated together, half of them
        dict(name="store_mixed", op="store", dtype="bf16", quant="stream4sym", hq=32, hkv=8, d=128, slots=16, page=256,
             lo=0, hi=2048, clo=1, chi=900, rot=64, pairs=True, mix=6),
        # fp16, 64 channels, one kv head per query head, blocks of 32 tokens
        dict(name="store_fp16", op="store", dtype="fp16", quant="tiny", hq=8, hkv=8, d=64, slots=3, page=128, lo=0,
             hi=900, clo=200, chi=2000, rot=64, pairs=False, mix=9),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["prompt", "chunk", "store"])
        hkv = rng.choice([1, 2, 4, 8, 8, 32])
        group = rng.choice([1, 1, 2, 3, 4, 4, 5, 8]) if hkv <= 8 else 1
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), hq=hkv * group, hkv=hkv, d=rng.choice([64, 128, 128]),
                 slots=_spread(rng, 1, 32), mix=rng.randrange(1 << 20))
        if op != "prompt":
            c["quant"] = rng.choice(sorted(_QUANT))
            if c["d"] < _QUANT[c["quant"]][3]:
                c["d"] = 128
            c["page"] = rng.choice([128, 256])
        a, b = sorted((_spread(rng, 1, 8192), _spread(rng, 1, 8192)))
        c["clo"], c["chi"] = a, b
        if op == "chunk":
            a, b = sorted((_spread(rng, 1, 65536), _spread(rng, 1, 65536)))
            c["lo"], c["hi"] = a, b
            if rng.random() < 0.4:
                c["clo"], c["chi"] = 1, rng.choice([1, 1, 4, 16])
        if op == "store":
            c["lo"], c["hi"] = 0, _spread(rng, 1, 8192)
            c["rot"] = rng.choice([c["d"], c["d"] // 2])
            c["pairs"] = rng.random() < 0.3
        starts, counts = _lengths(c)
        if sum(starts) + sum(counts) > 300000 or sum(counts) * c["hq"] > 32 * 65536:
            continue
        if 2e4 < _cost(c) <= top:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 200)


def _lengths(c):
    """(starts, counts): tokens each slot holds before its new ones, and its new tokens."""
    rng = random.Random(c["mix"])
    counts = [rng.randint(c["clo"], c["chi"]) if rng.random() < 0.9 else c["clo"] for _ in range(c["slots"])]
    starts = [rng.randint(c["lo"], c["hi"]) if "lo" in c else 0 for _ in range(c["slots"])]
    if c["op"] == "store":
        # tokens behind `starts` are dropped first, which the full-precision rows and whole blocks allow: a single
        # token goes between two flushes, longer chunks start on a block's border
        r = _QUANT[c["quant"]][4]
        starts = [s if n == 1 and (s + 1) % r else s // r * r for s, n in zip(starts, counts)]
    return starts, counts


# ------------------------------------------------------------------ inputs

def _dtype(c):
    return torch.float16 if c["dtype"] == "fp16" else torch.bfloat16


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys(gen, c, h, n):
    """[h, n, d] keys: N(0, 1) with one channel per head ten times larger, as trained models show."""
    x = _normal(gen, h, n, c["d"])
    x[torch.arange(h, device="cuda"), :, torch.randint(c["d"], (h,), generator=gen, device="cuda")] *= 10.0
    return x.to(_dtype(c))


def _rope_table(c, n):
    half = c["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator("cuda").manual_seed(int(seed))
    starts, counts = _lengths(c)
    hq, hkv, d, total = c["hq"], c["hkv"], c["d"], sum(counts)
    st = dict(case=c, starts=starts, counts=counts)
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    st["offsets"] = offsets
    if own:
        from bit_kv_cache_22_b200 import kvq
    if c["op"] == "prompt":
        # one projection's output: queries, keys and values of a token side by side
        qkv = _normal(gen, total, hq + 2 * hkv, d)
        qkv[:, hq:hq + hkv, 5] *= 10.0
        qkv[:, hq + hkv:] *= 0.5
        qkv = qkv.to(_dtype(c))
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        if own:
            st["plan"] = kvq.plan_prompt(counts, hq, hkv, d)
        return st
    bits, sym, G, Gv, R = _QUANT[c["quant"]]
    cap = -(-max(s + n for s, n in zip(starts, counts)) // c["page"]) * c["page"]
    held = [s + n for s, n in zip(starts, counts)] if c["op"] == "chunk" else starts
    if own:
        cache = kvq.PagedKVQCache(c["slots"], hq, hkv, d, G, Gv, R, bits, sym, _dtype(c), cap, c["page"])
        random.Random(seed).shuffle(cache.free_pages)   # a serving system's pages are in no order
        st["cache"] = cache
    else:
        st["slots"] = []
        st["k_res"] = torch.zeros(c["slots"], hkv, R, d, dtype=_dtype(c), device="cuda")
        st["v_res"] = torch.zeros_like(st["k_res"])
    for b, n in enumerate(held):
        k, v = _keys(gen, c, hkv, n), (0.5 * _normal(gen, hkv, n, d)).to(_dtype(c))
        if own:
            cache.prefill(b, k, v)
        else:
            tq = n // R * R
            st["k_res"][b, :, :n - tq], st["v_res"][b, :, :n - tq] = k[:, tq:], v[:, tq:]
            st["slots"].append((_quantize(k[:, :tq].float(), G, 1, bits, sym),
                                _quantize(v[:, :tq].float(), 1, Gv, bits, sym)) if c["op"] == "chunk" else None)
    st["q"] = _normal(gen, total, hq, d).to(_dtype(c))
    if c["op"] == "store":
        st["k"] = _keys(gen, c, hkv, total).transpose(0, 1).contiguous()
        st["v"] = (0.5 * _normal(gen, total, hkv, d)).to(_dtype(c))
        st["cos"], st["sin"] = _rope_table(c, cap)
        if own:
            st["rope"] = kvq.Rope(st["cos"], st["sin"], interleaved=c["pairs"])
    if own:
        st["plan"] = cache.plan_chunk(counts, starts)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        if op == "prompt":
            from bit_kv_cache_22_b200 import kvq
            return kvq.prompt_attention(st["plan"], st["q"], st["k"], st["v"])
        cache = st["cache"]
        if op == "chunk":
            return cache.chunk_attention(st["plan"], st["q"])
        q = cache.append_chunk(st["plan"], st["k"], st["v"], rope=st["rope"], t_Q=st["q"])
        k, v = cache.read_chunk(st["plan"])
        c = st["case"]
        shape = (c["slots"], c["hkv"], -1, c["d"])
        return dict(q=q, k=k, v=v, k_res=cache.k_residual.view(shape), v_res=cache.v_residual.view(shape))
    return _plain_store(st) if op == "store" else _plain_attention(st)


def _quantize(x, gt, gc, bits, sym):
    """x [h, t, d] float: codes, scales and zeros over groups of gt tokens x gc channels (one of them is 1), in fp32."""
    h, t, d = x.shape
    g = x.reshape(h, t // gt, gt, d // gc, gc)
    levels = torch.full((), float(2 ** bits - 1), device=x.device)
    if sym:
        s = 2.0 * g.abs().amax((2, 4), keepdim=True) / levels
        half = 2 ** (bits - 1)
        code = torch.where(s > 0, torch.round(g / s), torch.zeros_like(g)).clamp(-half, half - 1) + half
        z = torch.full_like(s, half)
    else:
        lo, hi = g.amin((2, 4), keepdim=True), g.amax((2, 4), keepdim=True)
        s = torch.where(hi > lo, (hi - lo) / levels, torch.where(lo != 0, lo.abs(), torch.ones_like(lo)))
        z = torch.round(-lo / s)
        code = (torch.round(g / s) + z).clamp(0, 2 ** bits - 1)
    return code.to(torch.uint8), s, z.to(torch.int16)


def _dequantize(held):
    code, s, z = held
    x = (code.float() - z.float()) * s
    return x.reshape(x.shape[0], x.shape[1] * x.shape[2], x.shape[3] * x.shape[4])


def _plain_attention(st):
    c = st["case"]
    hq, hkv, d, R = c["hq"], c["hkv"], c["d"], _QUANT[c["quant"]][4] if "quant" in c else 0
    out = torch.empty(st["q"].shape, dtype=_dtype(c), device="cuda")
    for b, (start, n) in enumerate(zip(st["starts"], st["counts"])):
        if n == 0:
            continue
        at, to = st["offsets"][b], st["offsets"][b + 1]
        if c["op"] == "prompt":
            k, v = (st[x][at:to].float().transpose(0, 1) for x in "kv")
        else:
            r = (start + n) % R
            k, v = (torch.cat([_dequantize(held), st[res][b, :, :r].float()], 1)
                    for held, res in zip(st["slots"][b], ("k_res", "v_res")))
        q = st["q"][at:to].float().reshape(n, hkv, hq // hkv, d).permute(1, 2, 0, 3)     # [hkv, g, n, d]
        step = max(1, (1 << 29) // (hq * (start + n)))
        for i in range(0, n, step):
            m = min(n, i + step)
            seen = start + m
            y = q[:, :, i:m].reshape(hkv, -1, d) @ k[:, :seen].transpose(1, 2) * (1.0 / math.sqrt(d))
            y = y.view(hkv, hq // hkv, m - i, seen)
            ahead = torch.arange(seen, device="cuda") > start + torch.arange(i, m, device="cuda")[:, None]
            y.masked_fill_(ahead, -math.inf)
            y -= y.amax(-1, keepdim=True)
            y.exp_()
            o = (y.view(hkv, -1, seen) @ v[:, :seen]).view(hkv, hq // hkv, m - i, d) / y.sum(-1, keepdim=True)
            out[at + i:at + m] = o.permute(2, 0, 1, 3).reshape(m - i, hq, d).to(out.dtype)
    return out


def _rotate(x, cos, sin, pairs):
    """x [n, h, d] float: channels (i, i + rot/2), or (2i, 2i + 1) for pairs, rotated by the row's angle i."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    x1, x2 = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs else (x[..., :half], x[..., half:2 * half])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack([y1, y2], -1).flatten(-2) if pairs else torch.cat([y1, y2], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _plain_store(st):
    c = st["case"]
    bits, sym, G, Gv, R = _QUANT[c["quant"]]
    t = _dtype(c)
    at = torch.cat([torch.arange(s, s + n, device="cuda") for s, n in zip(st["starts"], st["counts"])])
    cos, sin = st["cos"][at], st["sin"][at]
    q = _rotate(st["q"].float(), cos, sin, c["pairs"]).to(t)
    k = _rotate(st["k"].float(), cos, sin, c["pairs"]).to(t)
    k_out, v_out = k.clone(), st["v"].clone()
    k_res, v_res = st["k_res"].clone(), st["v_res"].clone()
    for b, (start, n) in enumerate(zip(st["starts"], st["counts"])):
        o, end = st["offsets"][b], start + n
        full = max(0, end // R * R - start) if start % R == 0 else 0      # new tokens in whole blocks
        if full:
            x = _dequantize(_quantize(k[o:o + full].float().transpose(0, 1), G, 1, bits, sym))
            k_out[o:o + full] = x.transpose(0, 1).to(t)
            x = _dequantize(_quantize(st["v"][o:o + full].float().transpose(0, 1), 1, Gv, bits, sym))
            v_out[o:o + full] = x.transpose(0, 1).to(t)
        row = (start + full) % R
        k_res[b, :, row:row + n - full] = k[o + full:o + n].transpose(0, 1)
        v_res[b, :, row:row + n - full] = st["v"][o + full:o + n].transpose(0, 1)
    return dict(q=q, k=k_out, v=v_out, k_res=k_res, v_res=v_res)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    starts, counts = _lengths(c)
    hq, hkv, d, total = c["hq"], c["hkv"], c["d"], sum(counts)
    pairs = sum(n * s + n * (n + 1) // 2 for s, n in zip(starts, counts))
    if c["op"] == "prompt":
        return {"bytes": 4 * total * d * (hq + hkv), "flops": 4 * d * hq * pairs}
    bits, sym, G, Gv, R = _QUANT[c["quant"]]
    meta = 4 if sym else 6
    token = hkv * (2 * d * bits // 8 + d * meta / G + d // Gv * meta)      # a quantized token's bytes
    if c["op"] == "chunk":
        live = [s + n for s, n in zip(starts, counts) if n]
        held = sum(n // R * R * token + n % R * hkv * d * 4 for n in live)
        return {"bytes": held + 4 * total * hq * d, "flops": 4 * d * hq * pairs}
    full = sum((s + n) // R * R - s if s % R == 0 else 0 for s, n in zip(starts, counts))
    kept = full * token + (total - full) * hkv * d * 4
    return {"bytes": 4 * total * d * (hq + hkv) + total * c["rot"] * 4 + 2 * kept + total * hkv * d * 4,
            "flops": 3 * total * c["rot"] * (hq + hkv) + 8 * full * hkv * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_held(x, bits, sym, axis_groups):
    """What is kept of x [n, h, d] (as the element type holds it): quotients are 32-bit, as the format defines them."""
    x = x.double()
    token_group, channel_group = axis_groups
    n, h, d = x.shape
    g = x.view(n // token_group, token_group, h, d // channel_group, channel_group)
    top = 2 ** bits - 1
    if sym:
        s = (2 * g.abs().amax(4, True).amax(1, True) / top).float().double()
        u = torch.nan_to_num((g / s).float().double().round(), nan=0.0).clamp(-(top + 1) // 2, top // 2)
        return (u * s).view(n, h, d)
    small, large = g.amin(4, True).amin(1, True), g.amax(4, True).amax(1, True)
    s = ((large - small).float().double() / top).float().double()
    s = torch.where(large > small, s, torch.where(small == 0, 1.0, small.abs()))
    z = (-small / s).float().double().round()
    u = ((g / s).float().double().round() + z).clamp(0, top)
    return ((u - z) * s).view(n, h, d)


def exact(case, seed):
    global own
    before, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = before
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "store":
        return _exact_store(st)
    res = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["counts"]):
        first, start = st["offsets"][b], st["starts"][b]
        if c["op"] == "prompt":
            k, v = st["k"][first:first + n].double(), st["v"][first:first + n].double()
        else:
            r = (start + n) % _QUANT[c["quant"]][4]
            k, v = (torch.cat([((code.double() - z.double()) * s.double()).flatten(3).flatten(1, 2),
                               rows[b, :, :r].double()], 1).transpose(0, 1)
                    for (code, s, z), rows in zip(st["slots"][b], (st["k_res"], st["v_res"])))
        for h in range(hq):
            kh, vh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
            for i in range(0, n, 1024):
                m = min(n, i + 1024)
                see = start + m
                y = torch.einsum("id,jd->ij", st["q"][first + i:first + m, h].double(), kh[:see]) / math.sqrt(d)
                y = y + torch.full_like(y, -math.inf).triu(start + i + 1)
                res[first + i:first + m, h] = torch.einsum("ij,jd->id", torch.softmax(y, -1), vh[:see])
    return res


def _exact_store(st):
    c = st["case"]
    bits, sym, G, Gv, R = _QUANT[c["quant"]]
    half, t = c["rot"] // 2, _dtype(c)
    position = torch.tensor([s + i for s, n in zip(st["starts"], st["counts"]) for i in range(n)], device="cuda")
    turn = torch.complex(st["cos"].double(), st["sin"].double())[position][:, None]

    def turned(x):
        x = x.double()
        if c["pairs"]:
            y = torch.view_as_real(torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:2], half, 2)) * turn)
            return torch.cat([y.reshape(*x.shape[:2], 2 * half), x[..., 2 * half:]], -1)
        y = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
        return torch.cat([y.real, y.imag, x[..., 2 * half:]], -1)

    q, k, v = turned(st["q"]), turned(st["k"]), st["v"].double()
    k_kept, v_kept, k_res, v_res = k.clone(), v.clone(), st["k_res"].double(), st["v_res"].double()
    for b, (start, n) in enumerate(zip(st["starts"], st["counts"])):
        o = st["offsets"][b]
        whole = (start + n) // R * R - start if start % R == 0 else 0
        if whole:
            k_kept[o:o + whole] = _exact_held(k[o:o + whole].to(t), bits, sym, (G, 1))
            v_kept[o:o + whole] = _exact_held(v[o:o + whole], bits, sym, (1, Gv))
        for i in range(whole, n):
            k_res[b, :, (start + i) % R] = k[o + i]
            v_res[b, :, (start + i) % R] = v[o + i]
    return dict(q=q, k=k_kept, v=v_kept, k_res=k_res, v_res=v_res)
