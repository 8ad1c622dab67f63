"""Plain 64-bit references of the MXFP4 cache operators, on the CPU, from the
format's definition and the layout that csrc/kv4.cuh documents."""
import math

import numpy as np
import torch

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantize(x: torch.Tensor):
    """bf16 [..., dim] -> (codes uint8 [..., dim], exponents uint8 [..., dim / 32])."""
    y = x.double().numpy().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = np.abs(y).max(-1)
    mant, ex = np.frexp(amax)                      # amax = mant * 2^ex, 0.5 <= mant < 1; 6 = 0.75 * 2^3
    e = np.where(amax == 0, -127, np.clip(ex - 3 + (mant > 0.75), -127, 127)).astype(int)
    a = np.abs(y) / np.ldexp(1.0, e)[..., None]
    lo = np.clip(np.searchsorted(MAGNITUDES, a, side="right") - 1, 0, 6)
    down, up = a - MAGNITUDES[lo], MAGNITUDES[lo + 1] - a
    code = lo + ((up < down) | ((up == down) & (lo % 2 == 1)))
    code = code + 8 * np.signbit(y)
    return torch.from_numpy(code.reshape(x.shape).astype(np.uint8)), torch.from_numpy((e + 127).astype(np.uint8))


def value(codes: torch.Tensor, e: torch.Tensor) -> torch.Tensor:
    """fp64 values of codes [..., dim] with exponents [..., dim / 32]."""
    c = codes.numpy()
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    return torch.from_numpy(v * np.repeat(np.ldexp(1.0, e.numpy().astype(int) - 127), 32, axis=-1))


def places(dim: int):
    """Byte and shift of each code and byte of each exponent in a record: {k, v: (byte [16, dim], shift)}, {ke, ve: [16, dim / 32]}."""
    t, d = np.arange(16)[:, None], np.arange(dim)[None, :]
    b = np.arange(dim // 32)[None, :]
    k = 4 * ((t * 4 + d % 32 // 8) * (dim // 32) + d // 32) + d % 8 // 2
    pair, half, odd = t % 8 // 2, t // 8, t % 2
    v = 8 * dim + 4 * (((d // 64 * 8 + d % 8) * 4 + pair) * 4 + d % 64 // 16) + 2 * half + d % 16 // 8
    ke = 16 * dim + t * (dim // 32) + b
    return {"k": (k, 4 * (d % 2) + 0 * t), "v": (v, 4 * odd + 0 * d), "ke": ke, "ve": ke + dim // 2}


class Cache:
    """A cache on the CPU, token by token: what the pages hold, in bytes."""

    def __init__(self, pages, page_size, heads, dim, seed=0, fill=None):
        self.page_size, self.heads, self.dim = page_size, heads, dim
        g = torch.Generator().manual_seed(seed)
        n = page_size // 16 * heads * 17 * dim
        self.data = torch.randint(0, 256, (pages, n), generator=g, dtype=torch.int32).to(torch.uint8)
        if fill is not None:
            self.data.fill_(fill)
        self.places = places(dim)

    def record(self, page, head, group):
        n = self.page_size // 16
        return self.data[page].view(self.heads, n, 17 * self.dim)[head, group]

    def write(self, page, slot, kc, ke, vc, ve):
        """One token's codes [heads, dim] and exponents [heads, dim / 32]."""
        for h in range(self.heads):
            rec = self.record(page, h, slot // 16).numpy()
            t = slot % 16
            for name, codes in (("k", kc), ("v", vc)):
                byte, shift = self.places[name][0][t], self.places[name][1][t]
                for i, c in enumerate(codes[h].tolist()):
                    rec[byte[i]] = rec[byte[i]] & ~np.uint8(15 << shift[i]) | np.uint8(c << shift[i])
            rec[self.places["ke"][t]] = ke[h].numpy()
            rec[self.places["ve"][t]] = ve[h].numpy()

    def read(self, pages, length):
        """fp64 keys and values [length, heads, dim] of the tokens in these pages."""
        out = []
        n = self.page_size // 16
        rec = self.data[list(pages)].numpy().reshape(-1, self.heads, n, 17 * self.dim)
        for name, ex in (("k", "ke"), ("v", "ve")):
            byte, shift = self.places[name]
            codes = (rec[..., byte] >> shift) & 15                          # page, head, group, token, dim
            e = rec[..., self.places[ex]]
            with np.errstate(over="ignore", invalid="ignore"):
                val = value(torch.from_numpy(codes.astype(np.uint8)), torch.from_numpy(e.astype(np.uint8)))
            out.append(val.permute(0, 2, 3, 1, 4).reshape(-1, self.heads, self.dim)[:length])
        return out


def attention(q, k, v, scale):
    """fp64 attention of q [n, q_heads, dim] at the last n positions of k, v [len, heads, dim]: (out, sum of
    weight * |v|, lse)."""
    n, hq, dim = q.shape
    length, hk, _ = k.shape
    out = torch.zeros(n, hq, dim, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64)
    for i in range(n):
        seen = length - n + i + 1
        if seen <= 0:
            continue
        for h in range(hq):
            kk, vv = k[:seen, h // (hq // hk)], v[:seen, h // (hq // hk)]
            s = kk @ q[i, h].double() * scale
            p = torch.softmax(s, 0)
            out[i, h], mag[i, h], lse[i, h] = p @ vv, p @ vv.abs(), torch.logsumexp(s, 0)
    return out, mag, lse


def norm_rope(x, w, cos_sin, pos, eps, interleaved):
    """fp64 norm and rotation of x [T, H, dim]: (y, the size of what each element was summed from)."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    rot = cos_sin.shape[1]
    half = rot // 2
    cos, sin = cos_sin.double()[pos.long()][:, None].split(half, -1)
    i = torch.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = y[..., ia].clone(), y[..., ib].clone()
    out, size = y.clone(), y.abs().clone()
    out[..., ia], out[..., ib] = a * cos - b * sin, b * cos + a * sin
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size
