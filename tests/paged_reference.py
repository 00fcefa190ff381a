"""Plain CPU forms of the paged-cache operators for the tests: the rotary turn in fp32, the encoder of
the oracle written into page blocks, and decode attention in 64 bits from the blocks' fields."""
import numpy as np
import torch

import oracle

BLOCK, BYTES, D = 32, 3200, 128
F16_MAX = 65504.0


def fields(pages: np.ndarray):
    """pages u8 [..., 3200] -> views: bits u32 [..., 32, 4], nc f32 [..., 32], scale / min u16 [..., 4, 32],
    codes u32 [..., 128, 4]."""
    lead = pages.shape[:-1]
    return (pages[..., :512].view(np.uint32).reshape(lead + (BLOCK, 4)), pages[..., 512:640].view(np.float32),
            pages[..., 640:896].view(np.uint16).reshape(lead + (4, BLOCK)),
            pages[..., 896:1152].view(np.uint16).reshape(lead + (4, BLOCK)),
            pages[..., 1152:].view(np.uint32).reshape(lead + (D, 4)))


def bit_row(tok):
    t, r = tok // 8, tok % 8
    return 8 * (r // 2) + 2 * t + r % 2


def nibble(tok):
    j = tok % 8
    return j // 2 + 4 * (j % 2)


def turn(x: np.ndarray, cos_sin: np.ndarray, pos, sections, interleaved) -> np.ndarray:
    """Rotary turn of fp32 rows x [heads, 128] of one token; pos: one position per axis."""
    half = cos_sin.shape[1] // 2
    out = x.astype(np.float32).copy()
    axis = np.repeat(np.arange(len(sections)), sections)
    for i in range(half):
        c, s = cos_sin[pos[axis[i]], i], cos_sin[pos[axis[i]], half + i]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        xa, xb = x[:, a].astype(np.float32), x[:, b].astype(np.float32)
        out[:, a] = np.float32(xa * c) - np.float32(xb * s)
        out[:, b] = np.float32(xb * c) + np.float32(xa * s)
    return out


def put(pages: np.ndarray, page: int, h: int, off: int, k: np.ndarray, v: np.ndarray, signs: np.ndarray):
    """Write one token of one kv-head at offset `off` of a page: k, v fp32 [128]."""
    v = np.clip(np.where(np.isnan(v), 0.0, v), -F16_MAX, F16_MAX).astype(np.float32)
    e = oracle.encode(k[None], v[None], signs)
    bits, nc, scale, least, codes = fields(pages)
    blk, tok = off // BLOCK, off % BLOCK
    bits[page, h, blk, bit_row(tok)] = e["bits"][0]
    nc[page, h, blk, tok] = np.float32(e["norm"][0]) * np.float32(e["cinv"][0])
    sm = e["sm"][0]
    s16, m16 = (sm & 0xFFFF).astype(np.uint16), (sm >> 16).astype(np.uint16)
    c = ((e["codes"][0][:, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(D).astype(np.uint32)
    for g in range(4):  # the scale one step lower where the top code would leave the binary16 range
        sf, mf = oracle.half_to_double(s16[g]), oracle.half_to_double(m16[g])
        if mf + 15.0 * sf > F16_MAX:
            s16[g] -= 1
            sf32, mf32 = np.float32(oracle.half_to_double(s16[g])), np.float32(mf)
            y = np.floor((v[32 * g:32 * g + 32] - mf32) / sf32 + np.float32(0.5))
            c[32 * g:32 * g + 32] = np.clip(y, 0, 15).astype(np.uint32)
    scale[page, h, blk, :, tok] = s16
    least[page, h, blk, :, tok] = m16
    w, sh = tok // 8, np.uint32(4 * nibble(tok))
    codes[page, h, blk, :, w] = (codes[page, h, blk, :, w] & ~(np.uint32(15) << sh)) | (c << sh)


def append(pages, k, v, table, start, cu, signs, rope=None, positions=None):
    """The whole append on a copy of `pages` (u8 [pages, heads, blocks, 3200]); k, v fp32 [T, H, 128].
    rope: (cos_sin, sections, interleaved); positions [axes, T].  Tokens without a page are left out."""
    pages = pages.copy()
    page_tokens = pages.shape[2] * BLOCK
    for b in range(len(start)):
        for t in range(cu[b], cu[b + 1]):
            pos = start[b] + t - cu[b]
            lp = pos // page_tokens
            page = table[b][lp] if lp < len(table[b]) else -1
            if not 0 <= page < pages.shape[0]:
                continue
            kt = k[t]
            if rope is not None:
                ps = [positions[min(a, len(positions) - 1)][t] for a in range(len(rope[1]))]
                if min(ps) < 0 or max(ps) >= rope[0].shape[0]:
                    continue
                kt = turn(kt, rope[0], ps, rope[1], rope[2])
            for h in range(pages.shape[1]):
                put(pages, page, h, pos % page_tokens, kt[h], v[t, h], signs)
    return pages


def gather(pages, table, h, tokens):
    """(signs +-1 [n, 128], values f64 [n, 128], nc f64 [n], scale code f64 [n, 128], scale f64 [n, 128]) of
    tokens of one list of pages."""
    page_tokens = pages.shape[2] * BLOCK
    bits, nc, scale, least, codes = fields(pages)
    pg = np.asarray(table)[tokens // page_tokens]
    blk, tok = tokens % page_tokens // BLOCK, tokens % BLOCK
    w = bits[pg, h, blk, bit_row(tok)]
    sign = ((w[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(-1, D) * 2.0 - 1.0
    word = codes[pg, h, blk][np.arange(len(tokens)), :, tok // 8]
    c = ((word >> (4 * nibble(tok)).astype(np.uint32)[:, None]) & 15).astype(np.float64)
    s = scale[pg, h, blk].view(np.float16)[np.arange(len(tokens)), :, tok].astype(np.float64).repeat(32, 1)
    m = least[pg, h, blk].view(np.float16)[np.arange(len(tokens)), :, tok].astype(np.float64).repeat(32, 1)
    return sign, m + s * c, nc[pg, h, blk, tok].astype(np.float64), s * c, s


class Row:
    """Softmax attention of one query head in 64 bits over `parts` (gather results), and how far a kernel's
    output may be from it."""

    def __init__(self, q: np.ndarray, signs, scale, parts):
        r = oracle.query_prep(q, signs)
        sign, val, nc, reach, step = (np.concatenate([p[i] for p in parts]) for i in range(5))
        self.tokens = len(nc)
        self.out = np.zeros(D)
        if self.tokens == 0:
            return
        code = r["codes"].astype(np.float64)
        dl, vl = float(r["delta"]), float(r["vl"])
        s = (sign @ code * dl + sign.sum(1) * vl) * nc * (scale / 128.0)
        # the magnitude of a logit's terms
        self.mag = (3 * code.sum() * abs(dl) + 384 * abs(vl)) * float(np.abs(nc).max()) * abs(scale) / 128.0
        p = np.exp(s - s.max())
        p /= p.sum()
        self.out, self.spread, self.reach = p @ val, p @ np.abs(val), p @ np.abs(reach)
        self.largest, self.step = float(np.abs(val).max()), float(step.max())

    def tolerance(self, eps):
        """Channel by channel.  Relative to the weighted mean of |value|: a weight's rounding to binary16 in
        the numerator and in the normaliser, a value's (2^-11 each), the fp32 logit (16 roundings of its
        terms' magnitude) and its exponential (2^-21), twice, and 2^-18 for the fp32 sums.  Relative to the
        weighted mean of scale code: the rounding of weight scale to binary16, 2^-11; or, for fp16 results,
        which carry it in two parts, what the codes lose as subnormal operands: the tensor cores line a
        product up by its operands' exponents, and a code c 2^-24 counts as 2^-14, so its sum keeps 2^10
        fewer of 24 bits; seventeen terms a product of a code that is 8 on the mean, at most 2^-13.  Small
        weights: one is 2^(7 - k) at its reference, which some token attains,
        where every scale is below 2^(1 + k); as a subnormal it may lose 2^-25, 2^-21 where it enters 2^-4
        lower, and weight scale may lose 2^-25 times a code of 15: a token adds at most 2^(k - 28) of the
        largest |value|, twice for the normaliser, and 2^(k - 28) itself.  At the end one rounding of the
        result to its type, eps / 2 of it, or 2^-25 where it is subnormal."""
        if self.tokens == 0:
            return np.full(D, 1e-30)
        k = max(1.0, 2 * self.step)
        rel = 3 * 2.0 ** -11 + 2 * (16 * 2.0 ** -24 * self.mag + 2.0 ** -21) + 2.0 ** -18
        tail = self.tokens * k * 2.0 ** -28 * (2 * self.largest + 1)
        part = 2.0 ** -11 if eps > 2.0 ** -9 else 2.0 ** -13
        return (1 + eps) * (rel * self.spread + part * self.reach + tail) + eps / 2 * np.abs(self.out) + 2.0 ** -25


def to_np(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy()
