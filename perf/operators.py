"""The cache operators, measured: 4-bit (MXFP4) paged keys and values of a language model, the attention that
reads them, the norm and rotation of queries and keys before them, and the moving of pages.

Each case is one operator call (the append cases read back what they wrote).  ``own = False`` computes it in its
plain form: elementary torch operations in fp32, rounded once at the end.  ``own = True`` makes the calls that a
user of the library makes.

The cache is a uint8 tensor [pages, page_bytes].  A page holds ``page`` tokens of every key/value head:
[head][group of 16 tokens][record], a record being 17 * dim bytes: key codes (8 * dim), value codes (8 * dim), key
exponents (dim / 2), value exponents (dim / 2).  Codes are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives),
each block of 32 elements along the head dimension has one UE8M0 exponent e, a value is code * 2^(e - 127).
``pack_records`` and ``unpack_records`` below say where each code stands.
"""
import math
import random

import torch

own = False

DEV = "cuda"
# E2M1 codes 0..15
CODE_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases

def listed():
    llama = {"q_heads": 32, "kv_heads": 8, "dim": 128}  # the 6144 columns of a fused 4096 -> 6144 projection
    return [
        # one decode step of 64 requests, between the QKV projection and the cache: latency
        {"name": "norm_decode", "op": "norm", "tokens": 64, **llama, "rot": 128, "interleaved": False, "max_pos": 32768},
        # a prefill of 8192 tokens, far positions
        {"name": "norm_prefill", "op": "norm", "tokens": 8192, **llama, "rot": 128, "interleaved": False, "max_pos": 1048576},
        # the new token of each of 64 decoding requests enters the cache
        {"name": "append_decode", "op": "append", "batch": 64, "new_lo": 1, "new_hi": 1, "old_lo": 1, "old_hi": 2000,
         "kv_heads": 8, "dim": 128, "page": 64},
        # prompts of odd lengths enter it, some behind a prefix that ends inside a 16-token group
        {"name": "append_prefill", "op": "append", "batch": 8, "new_lo": 1, "new_hi": 2047, "old_lo": 0, "old_hi": 301,
         "kv_heads": 8, "dim": 128, "page": 64},
        # short prefixes read back as bf16 (a prefill of another length against them)
        {"name": "gather_short", "op": "gather", "batch": 8, "len_lo": 100, "len_hi": 1500, "kv_heads": 8, "dim": 128, "page": 64},
        # long contexts read back
        {"name": "gather_long", "op": "gather", "batch": 2, "len_lo": 65001, "len_hi": 65536, "kv_heads": 8, "dim": 128, "page": 64},
        # one request's decode step over a short context: latency
        {"name": "attn_one", "op": "attn", "batch": 1, "q_lo": 1, "q_hi": 1, "len_lo": 1000, "len_hi": 1000, **llama, "page": 64},
        # a decode batch of 64 requests of every length up to 8192
        {"name": "attn_decode", "op": "attn", "batch": 64, "q_lo": 1, "q_hi": 1, "len_lo": 1, "len_hi": 8192, **llama, "page": 64},
        # a few very long contexts
        {"name": "attn_long", "op": "attn", "batch": 4, "q_lo": 1, "q_hi": 1, "len_lo": 100003, "len_hi": 131072, **llama, "page": 64},
        # two chunks of prompts behind cached prefixes (chunked prefill)
        {"name": "attn_chunk", "op": "attn", "batch": 2, "q_lo": 1025, "q_hi": 2048, "len_lo": 2048, "len_hi": 16384, **llama, "page": 64},
        # a request is forked: one partly filled page, in each of 32 layers
        {"name": "pages_fork", "op": "pages", "layers": 32, "pool": 64, "moves": 1, "kv_heads": 8, "dim": 128, "page": 64},
        # a pool is compacted
        {"name": "pages_compact", "op": "pages", "layers": 16, "pool": 1024, "moves": 400, "kv_heads": 8, "dim": 128, "page": 64},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over their logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "gather", "attn", "attn", "attn", "pages"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        return {"op": op, "tokens": _spread(rng, 1, 8192), "q_heads": min(40, kv * group), "kv_heads": kv, "dim": dim,
                "rot": rng.choice([dim, dim // 2]), "interleaved": rng.random() < 0.5, "max_pos": _spread(rng, 1024, 1048576)}
    if op == "append":
        batch = _spread(rng, 1, 64)
        hi = _spread(rng, 1, max(1, 8192 // batch))
        return {"op": op, "batch": batch, "new_lo": rng.choice([1, hi]), "new_hi": hi, "old_lo": 0, "old_hi": _spread(rng, 1, 2000),
                "kv_heads": kv, "dim": dim, "page": page}
    if op == "gather":
        batch = _spread(rng, 1, 32)
        hi = _spread(rng, 2, 65536 // batch)
        return {"op": op, "batch": batch, "len_lo": rng.randint(1, hi), "len_hi": hi, "kv_heads": kv, "dim": dim, "page": page}
    if op == "pages":
        pool = _spread(rng, 8, 1024)
        return {"op": op, "layers": rng.choice([1, 2, 5, 16]), "pool": pool, "moves": _spread(rng, 1, pool // 3 + 1), "kv_heads": kv,
                "dim": dim, "page": page}
    heads = {"q_heads": kv * group, "kv_heads": kv, "dim": dim, "page": page}
    kind = rng.choice(["decode", "decode", "spec", "chunk"])
    if kind == "chunk":
        q = _spread(rng, 9, 1024)
        ln = q + _spread(rng, 1, 6000)
        return {"op": op, "batch": rng.randint(1, 2), "q_lo": rng.randint(1, q), "q_hi": q, "len_lo": ln - rng.randint(0, ln - q), "len_hi": ln, **heads}
    batch = _spread(rng, 1, 64)
    hi = _spread(rng, 16, 131072 // batch)
    q = 1 if kind == "decode" else rng.randint(2, 8)
    return {"op": op, "batch": batch, "q_lo": 1, "q_hi": q, "len_lo": rng.randint(q, hi), "len_hi": hi, **heads}


def _lengths(n, lo, hi):
    """n lengths from lo to hi in even steps (in this order; prepare() shuffles the sequences)."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _sequences(case):
    """[(new tokens or queries, length with them)] of the case's sequences."""
    b = case["batch"]
    if case["op"] == "append":
        new = _lengths(b, case["new_lo"], case["new_hi"])
        old = _lengths(b, case["old_lo"], case["old_hi"])
        return [(n, n + o) for n, o in zip(new, reversed(old))]
    if case["op"] == "gather":
        return [(n, n) for n in _lengths(b, case["len_lo"], case["len_hi"])]
    return list(zip(_lengths(b, case["q_lo"], case["q_hi"]), _lengths(b, case["len_lo"], case["len_hi"])))


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        return {"bytes": 4 * n * case["dim"] + case["tokens"] * (4 * case["rot"] + 4), "flops": 10 * n * case["dim"]}
    per_token = case["kv_heads"] * case["dim"] * 17 // 16  # K and V of one token in the cache, in bytes
    if op == "pages":
        return {"bytes": 2 * case["layers"] * case["moves"] * case["page"] * per_token, "flops": 0}
    seqs = _sequences(case)
    rows = case["kv_heads"] * case["dim"] * 4  # K and V of one token as bf16, in bytes
    if op == "append":
        new = sum(n for n, _ in seqs)
        back = sum(ln - (ln - n) // 16 * 16 for n, ln in seqs)
        return {"bytes": new * (rows + per_token) + back * (per_token + rows), "flops": 0}
    if op == "gather":
        n = sum(ln for _, ln in seqs)
        return {"bytes": n * (per_token + rows), "flops": 0}
    width = case["q_heads"] * case["dim"]
    pairs = sum(n * (ln - n) + n * (n + 1) // 2 for n, ln in seqs)  # a query sees itself and all before it
    return {"bytes": sum(ln for _, ln in seqs) * per_token + 4 * sum(n for n, _ in seqs) * width, "flops": 4 * pairs * width}


# ------------------------------------------------------------------ the format, in elementary operations

def quantize(x):
    """bf16 [..., dim] -> E2M1 codes uint8 [..., dim] and exponents uint8 [..., dim / 32]: the smallest power of two
    that brings a block's largest magnitude to 6 or less, round to nearest even; exponent 0 for a block of zeros."""
    blocks = x.float().unflatten(-1, (-1, 32))
    mant, ex = torch.frexp(blocks.abs().amax(-1))
    e = ex - 3 + (mant > 0.75).int()
    e = torch.where(mant == 0, -127, e).clamp(-127, 127)
    y = torch.ldexp(blocks, -e.unsqueeze(-1))
    a = y.abs()
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte()
    return (code + 8 * torch.signbit(y).byte()).flatten(-2), (e + 127).byte()


def dequantize(codes, e):
    """Codes [..., dim] and exponents [..., dim / 32] -> fp32 values."""
    v = torch.tensor(CODE_VALUES, device=codes.device)[codes.int()].unflatten(-1, (-1, 32))
    return torch.ldexp(v, (e.int() - 127).unsqueeze(-1)).flatten(-2)


def pack_records(kc, ke, vc, ve):
    """Codes [..., 16, dim] and exponents [..., 16, dim / 32] of 16 tokens -> records [..., 17 * dim]."""
    lead, dim, nb = kc.shape[:-2], kc.shape[-1], ke.shape[-1]
    z = len(lead)
    k = kc.reshape(*lead, 16, nb, 4, 4, 2)  # token, block, quarter of the block, byte, nibble
    k = (k[..., 0] | (k[..., 1] << 4)).movedim(z + 2, z + 1).reshape(*lead, -1)  # token, quarter, block, byte
    v = vc.reshape(*lead, 2, 4, 2, dim // 64, 4, 2, 8)  # tokens: half, pair, odd; dim: 64s, 16s, 8s, 1s
    v = v.select(z + 2, 0) | (v.select(z + 2, 1) << 4)  # half, pair, 64s, 16s, 8s, 1s
    v = v.permute(*range(z), z + 2, z + 5, z + 1, z + 3, z + 0, z + 4).reshape(*lead, -1)
    return torch.cat([k, v, ke.reshape(*lead, -1), ve.reshape(*lead, -1)], -1)


def unpack_records(rec):
    """Records [..., 17 * dim] -> fp32 keys and values [..., 16, dim]."""
    lead, dim = rec.shape[:-1], rec.shape[-1] // 17
    z, nb = len(lead), dim // 32
    k, v, ke, ve = rec.split([8 * dim, 8 * dim, dim // 2, dim // 2], -1)
    k = k.reshape(*lead, 16, 4, nb, 4).movedim(z + 1, z + 2)
    k = torch.stack([k & 15, k >> 4], -1).reshape(*lead, 16, dim)
    v = v.reshape(*lead, dim // 64, 8, 4, 4, 2, 2).permute(*range(z), z + 4, z + 2, z + 0, z + 3, z + 5, z + 1)  # half, pair, 64s, 16s, 8s, 1s
    v = torch.stack([v & 15, v >> 4], z + 2).reshape(*lead, 16, dim)
    return dequantize(k, ke.reshape(*lead, 16, nb)), dequantize(v, ve.reshape(*lead, 16, nb))


def read_cache(cache, table, kv_heads, dim, page):
    """The cached keys and values of every slot of a page table: fp32 [sequences, slots, kv_heads, dim] each."""
    rec = cache[table.clamp(min=0).long()].reshape(*table.shape, kv_heads, page // 16, 17 * dim)
    k, v = unpack_records(rec)  # sequence, page, head, group, token, dim
    return tuple(t.permute(0, 1, 3, 4, 2, 5).reshape(table.shape[0], -1, kv_heads, dim) for t in (k, v))


# ------------------------------------------------------------------ inputs

def _kv_values(g, n, kv_heads, dim):
    """bf16 keys and values as a projection gives them: keys with a few strong channels, values smaller."""
    chan = torch.exp(0.7 * torch.randn(kv_heads, dim, generator=g, device=DEV))
    k = torch.randn(n, kv_heads, dim, generator=g, device=DEV) * chan
    v = torch.randn(n, kv_heads, dim, generator=g, device=DEV) * 0.5
    return k.bfloat16(), v.bfloat16()


def _cached(g, rng, case, lengths, room):
    """A cache that holds ``lengths`` tokens of each sequence, in pages for ``room`` tokens.  Slots behind a
    sequence hold whatever a page held before: any bytes."""
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    pages = [-(-r // page) for r in room]
    used, spare = sum(pages), 3
    ids = list(range(used + spare))
    rng.shuffle(ids)
    table = torch.full((len(room), max(1, max(pages))), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    cache = torch.randint(0, 256, (used + spare, page * kv * dim * 17 // 16), generator=g, device=DEV, dtype=torch.uint8)
    for s, n in enumerate(lengths):  # tokens of one sequence at a time, so that a long cache needs little memory beside it
        slots = pages[s] * page
        if slots == 0:
            continue
        k, v = _kv_values(g, slots, kv, dim)
        (kc, ke), (vc, ve) = quantize(k), quantize(v)
        stale = (torch.arange(slots, device=DEV) >= n).view(-1, 1, 1)
        parts = []
        for t, top in ((kc, 16), (ke, 256), (vc, 16), (ve, 256)):
            t = torch.where(stale, torch.randint(0, top, t.shape, generator=g, device=DEV, dtype=torch.uint8), t)
            parts.append(t.reshape(pages[s], page // 16, 16, kv, -1).permute(0, 3, 1, 2, 4))
        cache[table[s, :pages[s]].long().to(DEV)] = pack_records(*parts).reshape(pages[s], -1)
    return cache, table.to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    op, dim = case["op"], case["dim"]
    st = {"case": case}
    if op == "norm":
        t, hq, hk, rot = case["tokens"], case["q_heads"], case["kv_heads"], case["rot"]
        # the projection's output, whose V part stays as it is
        qkv = (torch.randn(t, (hq + 2 * hk) * dim, generator=g, device=DEV) * 1.5).bfloat16()
        st["q"] = qkv[:, :hq * dim].unflatten(1, (hq, dim))
        st["k"] = qkv[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
        st["wq"], st["wk"] = ((1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).bfloat16() for _ in range(2))
        # the table that a program keeps: angles in 64 bits
        inv = 500000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        ang = torch.arange(case["max_pos"], device=DEV, dtype=torch.float64).unsqueeze(1) * inv
        st["cos_sin"] = torch.cat([ang.cos().float(), ang.sin().float()], 1)
        st["pos"] = torch.randint(0, case["max_pos"], (t,), generator=g, device=DEV).int()
        return st
    if op == "pages":
        width = case["page"] * case["kv_heads"] * dim * 17 // 16
        st["cache"] = torch.randint(0, 256, (case["layers"], case["pool"], width), generator=g, device=DEV, dtype=torch.uint8)
        ids = rng.sample(range(case["pool"]), 2 * case["moves"])  # what a pool's bookkeeping on the host gives
        st["src"], st["dst"] = ids[:case["moves"]], ids[case["moves"]:]
        return st
    seqs = _sequences(case)
    rng.shuffle(seqs)
    lengths = [ln for _, ln in seqs]
    cu = [0]
    for n, _ in seqs:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    st["lens"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    st["total"] = cu[-1]
    old = [ln - n for n, ln in seqs] if op == "append" else lengths
    st["cache"], st["table"] = _cached(g, rng, case, old, lengths)
    if op == "append":
        st["k"], st["v"] = _kv_values(g, cu[-1], case["kv_heads"], dim)
        starts = [o // 16 * 16 for o in old]  # read back from the first group that the call writes into
        back = [0]
        for s, ln in zip(starts, lengths):
            back.append(back[-1] + ln - s)
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        st["back"] = torch.tensor(back, dtype=torch.int32, device=DEV)
        st["back_total"] = back[-1]
    elif op == "attn":
        st["q"] = torch.randn(cu[-1], case["q_heads"], dim, generator=g, device=DEV).bfloat16()
        st["scale"] = dim ** -0.5
        st["ws"] = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)  # scratch that a serving program zeroes once and keeps
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        return _run_own(case["op"], case, st)
    return {"norm": _norm, "append": _append, "gather": _gather, "attn": _attention, "pages": _pages}[case["op"]](case, st)


def _run_own(op, case, st):
    import mxfp8_block_scaled_fp8_b200 as fp8mm
    if op == "norm":
        return fp8mm.qk_norm_rope(st["q"], st["k"], st["cos_sin"], st["pos"], q_weight=st["wq"], k_weight=st["wk"], eps=1e-6,
                                  interleaved=case["interleaved"])
    if op == "pages":
        return fp8mm.kv_copy_pages(st["cache"], st["src"], st["dst"])
    page, dim = case["page"], case["dim"]
    if op == "append":
        fp8mm.mxfp4_kv_append(st["k"], st["v"], st["cache"], st["table"], st["lens"], page, cu_seqlens=st["cu"])
        return fp8mm.mxfp4_kv_gather(st["cache"], st["table"], st["back"], page, dim, st["back_total"], starts=st["starts"])
    if op == "gather":
        return fp8mm.mxfp4_kv_gather(st["cache"], st["table"], st["cu"], page, dim, st["total"])
    cu = st["cu"] if case["q_hi"] > 1 else None
    return fp8mm.mxfp4_kv_attention(st["q"], st["cache"], st["table"], st["lens"], page, cu_seqlens=cu, scale=st["scale"],
                                    workspace=st["ws"])


def _norm(case, st):
    half = case["rot"] // 2
    cos, sin = st["cos_sin"][st["pos"].long()].unsqueeze(1).split(half, -1)
    outs = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        r, rest = x[..., :case["rot"]], x[..., case["rot"]:]
        a, b = (r[..., 0::2], r[..., 1::2]) if case["interleaved"] else (r[..., :half], r[..., half:])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        r = torch.stack([ra, rb], -1).flatten(-2) if case["interleaved"] else torch.cat([ra, rb], -1)
        outs.append(torch.cat([r, rest], -1).bfloat16())
    return tuple(outs)


def _spans(cu, starts, total):
    """Sequence and position of each row of a ragged batch."""
    row = torch.arange(total, device=DEV)
    seq = torch.searchsorted(cu[1:].long(), row, right=True)
    pos = row - cu.long()[seq]
    return seq, pos if starts is None else pos + starts.long()[seq]


def _append(case, st):
    page = case["page"]
    old = (st["lens"] - st["cu"][1:] + st["cu"][:-1]).long()
    at = st["table"].gather(1, (old // page).clamp(max=st["table"].shape[1] - 1).view(-1, 1))  # the page that the new tokens begin in
    seq, pos = _spans(st["back"], st["starts"], st["back_total"])
    is_old = (pos < old[seq]).view(-1, 1, 1)
    row = (st["cu"].long()[seq] + pos - old[seq]).clamp(min=0)
    kept = read_cache(st["cache"], at, case["kv_heads"], case["dim"], page)
    return tuple(torch.where(is_old, t[seq, pos % page], dequantize(*quantize(x))[row]).bfloat16() for t, x in zip(kept, (st["k"], st["v"])))


def _gather(case, st):
    k, v = read_cache(st["cache"], st["table"], case["kv_heads"], case["dim"], case["page"])
    seq, pos = _spans(st["cu"], None, st["total"])
    return k[seq, pos].bfloat16(), v[seq, pos].bfloat16()


def _attention(case, st):
    b, hq, hk, dim, most = case["batch"], case["q_heads"], case["kv_heads"], case["dim"], case["q_hi"]
    k, v = read_cache(st["cache"], st["table"], hk, dim, case["page"])
    new = (st["cu"][1:] - st["cu"][:-1]).long()
    lens = st["lens"].long()
    seq, i = _spans(st["cu"], None, st["total"])
    q = torch.zeros(b, most, hq, dim, device=DEV)
    q[seq, i] = st["q"].float()
    q = q.view(b, most, hk, hq // hk, dim).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, dim)
    pos = (lens - new).view(b, 1) + torch.arange(most, device=DEV)  # position of each query
    slot = torch.arange(k.shape[1], device=DEV)
    seen = (slot <= pos.unsqueeze(-1)) & (slot < lens.view(b, 1, 1))  # [b, most, slots]
    seen = seen.view(b, 1, 1, most, -1).expand(b, 1, hq // hk, most, -1).reshape(b, 1, -1, k.shape[1])
    v = torch.where((slot < lens.view(b, 1)).view(b, -1, 1, 1), v, 0.0)  # stale slots may stand for anything
    s = torch.matmul(q * st["scale"], k.permute(0, 2, 3, 1))
    s = torch.where(seen, s, float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.transpose(1, 2)) / torch.where(total > 0, total, 1.0)
    o = o.view(b, hk, hq // hk, most, dim).permute(0, 3, 1, 2, 4).reshape(b, most, hq, dim)
    return o[seq, i].bfloat16()


def _pages(case, st):
    st["cache"][:, st["dst"]] = st["cache"][:, st["src"]]
    return st["cache"]


# ------------------------------------------------------------------ the definitions, in 64 bits

def _stored(rec, dim):
    """fp64 keys and values [16, dim] of records [n, 17 * dim], element by element from the layout's definition:
    the byte and nibble in which each code stands, and the byte of its exponent."""
    tok, d = torch.arange(16, device=DEV).view(16, 1), torch.arange(dim, device=DEV).view(1, dim)
    half, pair, odd = tok // 8, tok % 8 // 2, tok % 2
    kbyte = tok * (dim // 2) + d % 32 // 8 * (dim // 8) + d // 32 * 4 + d % 8 // 2
    vbyte = 8 * dim + d // 64 * 512 + (d % 8 * 4 + pair) * 16 + d % 64 // 16 * 4 + half * 2 + d % 16 // 8
    kexp = 16 * dim + tok * (dim // 32) + d // 32
    vexp = kexp + dim // 2
    values = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=DEV, dtype=torch.float64)
    out = []
    for byte, shift, ex in ((kbyte, d % 2 * 4 + 0 * tok, kexp), (vbyte, odd * 4 + 0 * d, vexp)):
        code = (rec[:, byte].int() >> shift.int()) & 15
        mag = values[code.long() & 7] * (1 - 2 * (code >> 3)).double()
        out.append(mag * torch.exp2(rec[:, ex].double() - 127))
    return out


def _tokens(cache, pages, first, last, case):
    """fp64 keys and values [last - first, kv_heads, dim] of one sequence's tokens."""
    dim, page, kv = case["dim"], case["page"], case["kv_heads"]
    if last <= first:
        return [torch.zeros(0, kv, dim, dtype=torch.float64, device=DEV)] * 2
    a, b = first // page, (last - 1) // page + 1
    rec = cache[pages[a:b].long()].view(b - a, kv, page // 16, 17 * dim)
    got = _stored(rec.transpose(1, 2).reshape(-1, 17 * dim), dim)  # page, group, head
    return [t.view(-1, kv, 16, dim).transpose(1, 2).reshape(-1, kv, dim)[first - a * page:last - a * page] for t in got]


def _nearest(x):
    """The values that the format holds for bf16 rows [..., dim], in fp64: of the eight magnitudes the nearest, of two as near the even one."""
    y = x.double().unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True)
    grid = torch.exp2(torch.arange(-127, 128, device=DEV, dtype=torch.float64))
    step = grid[torch.searchsorted(6 * grid, top).clamp(max=254)]  # the first power of two with 6 * 2^e >= top
    mags = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=DEV, dtype=torch.float64)
    a = y.abs() / step
    lo = (torch.searchsorted(mags, a, right=True) - 1).clamp(0, 6)
    down, up = a - mags[lo], mags[lo + 1] - a
    at = lo + ((up < down) | ((up == down) & (lo % 2 == 1))).long()
    return (mags[at] * step * torch.sign(y)).flatten(-2)


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None
    if op == "attn" and sum(n * ln for n, ln in _sequences(case)) * case["q_heads"] > 5e9:
        return None
    st = prepare(case, seed)
    if op == "norm":
        rot = case["rot"]
        table = st["cos_sin"].double()[st["pos"].long()]
        z = torch.complex(table[:, :rot // 2], table[:, rot // 2:]).unsqueeze(1)
        outs = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            y = x.double()
            y = y / (y.square().sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * w.double()
            pairs = y[..., :rot].unflatten(-1, (-1, 2)) if case["interleaved"] else y[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
            turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
            y[..., :rot] = (turned if case["interleaved"] else turned.transpose(-1, -2)).flatten(-2)
            outs.append(y)
        return tuple(outs)
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    ks, vs = [], []
    if op == "append":
        for s, ln in enumerate(lens):
            old = ln - (cu[s + 1] - cu[s])
            k, v = _tokens(st["cache"], st["table"][s], old // 16 * 16, old, case)
            ks += [k, _nearest(st["k"][cu[s]:cu[s + 1]])]
            vs += [v, _nearest(st["v"][cu[s]:cu[s + 1]])]
        return torch.cat(ks), torch.cat(vs)
    if op == "gather":
        for s, ln in enumerate(lens):
            k, v = _tokens(st["cache"], st["table"][s], 0, ln, case)
            ks.append(k)
            vs.append(v)
        return torch.cat(ks), torch.cat(vs)
    outs = []
    group = case["q_heads"] // case["kv_heads"]
    for s, ln in enumerate(lens):
        k, v = _tokens(st["cache"], st["table"][s], 0, ln, case)
        q = st["q"][cu[s]:cu[s + 1]].double()
        n = q.shape[0]
        later = torch.arange(ln, device=DEV).view(1, ln) > torch.arange(ln - n, ln, device=DEV).view(n, 1)
        o = torch.empty_like(q)
        for h in range(case["q_heads"]):
            w = (q[:, h] @ k[:, h // group].T) * st["scale"]
            w.masked_fill_(later, float("-inf"))
            o[:, h] = torch.softmax(w, -1) @ v[:, h // group]
        outs.append(o)
    return torch.cat(outs)
