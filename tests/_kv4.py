"""The 4-bit paged cache restated in numpy for the tests: packing, unpacking,
the position rotation in fp32 step by step, and attention in 64 bits.  Shares
no code with the library."""
from __future__ import annotations

import numpy as np

import workloads as wl


def f32(bits) -> np.ndarray:
    return wl.bf16_to_f32(np.ascontiguousarray(bits, np.uint16))


def bf16(x) -> np.ndarray:
    """fp32 to BF16 bits, nearest even; NaN to the quiet NaN."""
    x = np.ascontiguousarray(x, np.float32)
    bits = wl.bf16_bits(np.where(np.isnan(x), np.float32(0), x))
    return np.where(np.isnan(x), np.uint16(0x7FC0), bits).astype(np.uint16)


def rotate(bits, cos, sin, interleaved) -> np.ndarray:
    """bits [tokens, heads, D]; cos, sin fp32 [tokens, pairs].  BF16 bits."""
    out = np.array(bits)
    n = cos.shape[1]
    if n == 0:
        return out
    a_at, b_at = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x = f32(bits).reshape(bits.shape)
    a, b, c, s = x[..., a_at], x[..., b_at], cos[:, None], sin[:, None]
    out[..., a_at] = bf16(a * c - b * s)
    out[..., b_at] = bf16(b * c + a * s)
    return out


def quantise(bits):
    """Vectors [.., D] of BF16 bits -> codes uint8 [.., D], (scale, lo) BF16 bits [.., 2]."""
    x = f32(bits).reshape(bits.shape)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], np.float32(0), x)
    half = np.float32(0.5)
    hi, lo = x.max(-1), x.min(-1)
    scale = bf16((hi * half - lo * half) / np.float32(7.5))
    s = f32(scale).reshape(scale.shape)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.rint((x * half - lo[..., None] * half) / (s * half))
    code = np.where(s > 0, np.clip(np.nan_to_num(code), 0, 15), 0).astype(np.uint8)
    par = np.stack([scale, bf16(lo)], -1)
    par[bad] = 0x7FC0
    code[bad] = 0
    return code, par


def value(code, par) -> np.ndarray:
    """What codes [.., D] and params [.., 2] stand for, in fp32."""
    p = f32(par).reshape(par.shape)
    return (p[..., 1:].astype(np.float64) + code.astype(np.float64) * p[..., :1].astype(np.float64)).astype(np.float32)


class Pages:
    """A pool of pages as bytes, and the regions of its blocks as views."""

    def __init__(self, n_pages, heads, dim, page, fill=0):
        self.dim, self.page, self.heads = dim, page, heads
        self.bytes = np.full((n_pages, heads, page * (dim + 8)), fill, np.uint8)
        cut = page * dim // 2
        b = self.bytes
        self.codes = [b[..., :cut].reshape(n_pages, heads, page, dim // 2),
                      b[..., cut:2 * cut].reshape(n_pages, heads, page, dim // 2)]
        self.pars = [b[..., 2 * cut:2 * cut + 4 * page].view(np.uint16).reshape(n_pages, heads, page, 2),
                     b[..., 2 * cut + 4 * page:].view(np.uint16).reshape(n_pages, heads, page, 2)]
        assert all(np.shares_memory(v, b) for v in self.codes + self.pars)

    def put(self, which, page, slot, head, code, par):
        self.codes[which][page, head, slot] = code[0::2] | code[1::2] << 4
        self.pars[which][page, head, slot] = par

    def get(self, which, table_row, length, head):
        """Codes [length, D] and params [length, 2] of one sequence's head."""
        at = np.arange(length)
        page, slot = table_row[at // self.page], at % self.page
        packed = self.codes[which][page, head, slot]
        code = np.empty((length, self.dim), np.uint8)
        code[:, 0::2], code[:, 1::2] = packed & 15, packed >> 4
        return code, self.pars[which][page, head, slot]


def random_table(rng, lens, page, spare=2):
    """Page numbers of every sequence in a mixed order; unused entries are -1."""
    counts = [-(-n // page) for n in lens]
    pool = sum(counts) + spare
    mixed = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(max(counts), 1)), -1, np.int32)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = mixed[at:at + c]
        at += c
    return table, pool


def starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def attention(q, pages, table, new, lens, kv_heads, causal, window, scale):
    """q [tokens, q heads, D] fp32.  Returns o, lse and, for the error bound,
    sum_j p_j (|v_j - z_j| + |z_j|) with z_j the middle of v_j's range, all in 64 bits."""
    t, hq, d = q.shape
    g = hq // kv_heads
    o, bound = np.zeros((t, hq, d)), np.zeros((t, hq, d))
    lse = np.full((t, hq), -np.inf)
    at = 0
    for s, (n, m) in enumerate(zip(new, lens)):
        pos = m - n + np.arange(n)[:, None]
        key = np.arange(m)
        seen = np.ones((n, m), bool)
        if causal:
            seen &= key <= pos
        if window:
            seen &= key > pos - window
        for h in range(kv_heads):
            (kc, kp), (vc, vp) = pages.get(0, table[s], m, h), pages.get(1, table[s], m, h)
            k, v = value(kc, kp).astype(np.float64), value(vc, vp).astype(np.float64)
            p32 = f32(vp).reshape(-1, 2).astype(np.float64)
            mid = p32[:, 1:] + 8 * p32[:, :1]
            for j in range(h * g, (h + 1) * g):
                # a masked key takes no part, whatever it holds
                sc = np.where(seen, q[at:at + n, j].astype(np.float64) @ k.T * scale, -np.inf)
                top = np.max(sc, 1, initial=-np.inf, keepdims=True)
                p = np.where(seen, np.exp(sc - np.where(np.isneginf(top), 0, top)), 0)
                tot = p.sum(1, keepdims=True)
                none = tot == 0
                pn = p / np.where(none, 1, tot)
                hurt = (seen & np.isnan(v).any(1)).any(1)[:, None]
                o[at:at + n, j] = np.where(hurt, np.nan, pn @ np.nan_to_num(v))
                bound[at:at + n, j] = pn @ np.nan_to_num(np.abs(v - mid) + np.abs(mid))
                lse[at:at + n, j] = np.where(none, -np.inf, np.log(np.where(none, 1, tot)) + top)[:, 0]
        at += n
    return o, lse, bound
