"""Oracle of the paged 8-bit cache and of prompt attention, in numpy: plans by
walking the requests token by token, codes from IEEE fp32 quotients, attention
in fp64 on the dequantized cache. Test infrastructure only."""
from __future__ import annotations

import numpy as np


def e4m3_values():
    """The 256 values of 1 sign, 4 exponent (bias 7), 3 fraction bits, by their
    bits; NaN where all exponent and fraction bits are set, no infinities."""
    out = np.empty(256, np.float64)
    for b in range(256):
        sign, e, f = (-1.0 if b & 128 else 1.0), (b >> 3) & 15, b & 7
        v = f / 8.0 * 2.0 ** -6 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)
        out[b] = np.nan if (e == 15 and f == 7) else sign * v
    return out


_E4M3 = e4m3_values()
_MAG = _E4M3[:127]  # magnitudes of bits 0 .. 126 in ascending order


def to_e4m3(y):
    """Bits of the value nearest to y (ties to the even fraction), |y| <= 448 after a clamp."""
    y = np.asarray(y, np.float64)
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(_MAG, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _MAG[lo], _MAG[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantize_page(x, code):
    """(codes, fp32 scale) of one page tile x [token][channel], code "int8" or
    "e4m3": s = absmax / Q and x / s in IEEE fp32, the code nearest to the quotient."""
    x = np.asarray(x, np.float32)
    q = np.float32(127.0 if code == "int8" else 448.0)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        s = np.float32(np.abs(x).max()) / q
        y = np.zeros_like(x) if s == 0 else (x / s).astype(np.float32)
    if code == "int8":
        return np.clip(np.rint(np.nan_to_num(y)), -127, 127).astype(np.int8), s
    return np.where(np.isnan(y), 127, to_e4m3(np.nan_to_num(y))).astype(np.uint8), s


def page_values(codes, scale, code):
    v = codes.astype(np.float64) if code == "int8" else _E4M3[codes]
    with np.errstate(invalid="ignore"):
        return v * np.float64(scale)


def reserve(lens, new, table, free_pages, free_count, max_tokens, page):
    """(table, cu, slots, positions, lens, free_count) after the step, or None
    where it does not fit."""
    table = table.copy()
    cu, slots, positions, count = [0], [], [], int(free_count)
    for b, (n, m) in enumerate(zip(lens.tolist(), new.tolist())):
        if n < 0 or m < 0 or -(-(n + m) // page) > table.shape[1]:
            return None
        for p in range(n, n + m):
            if p % page == 0:
                count -= 1
                if count < 0:
                    return None
                table[b, p // page] = free_pages[count]
            slots.append(int(table[b, p // page]) * page + p % page)
            positions.append(p)
        cu.append(cu[-1] + m)
    if cu[-1] > max_tokens:
        return None
    pad = [-1] * (max_tokens - len(slots))
    as32 = lambda x: np.array(x, np.int32)
    return table, as32(cu), as32(slots + pad), as32(positions + pad), (lens + new).astype(np.int32), count


def release(done, lens, table, free_pages, free_count, page):
    free_pages, lens, count = free_pages.copy(), lens.copy(), int(free_count)
    for b in np.flatnonzero(done):
        for j in range(-(-int(lens[b]) // page)):
            free_pages[count] = table[b, j]
            count += 1
        lens[b] = 0
    return lens, free_pages, count


class PagedOracle:
    """Tokens of every request as given; codes and scales by page id."""

    def __init__(self, requests, heads, dim, page, code):
        self.rows = [np.zeros((0, heads, 2, dim)) for _ in range(requests)]
        self.codes, self.scales = {}, {}
        self.heads, self.dim, self.page, self.code = heads, dim, page, code

    def write(self, b, k, v, table_row):
        """k, v [token][head][channel] of request b."""
        n = len(self.rows[b])
        self.rows[b] = np.concatenate([self.rows[b], np.stack([k, v], 2)])
        for j in range(n // self.page, len(self.rows[b]) // self.page):
            x = self.rows[b][j * self.page:(j + 1) * self.page]  # [token][head][2][channel]
            for h in range(self.heads):
                for i in range(2):
                    self.codes[int(table_row[j]), h, i], self.scales[int(table_row[j]), h, i] = quantize_page(
                        x[:, h, i], self.code)

    def end(self, b):
        self.rows[b] = self.rows[b][:0]

    def values(self, b, table_row):
        """K and V of request b as attention reads them: [2][head][token][channel] fp64."""
        n = len(self.rows[b])
        x = self.rows[b].transpose(2, 1, 0, 3).copy()
        for j in range(n // self.page):
            for h in range(self.heads):
                for i in range(2):
                    p = int(table_row[j])
                    x[i, h, j * self.page:(j + 1) * self.page] = page_values(self.codes[p, h, i],
                                                                             self.scales[p, h, i], self.code)
        return x

    def tail(self, b):
        """Rows of the open page [token][head][2][channel]."""
        return self.rows[b][len(self.rows[b]) // self.page * self.page:]


def attend(q, k, v, scale):
    """(o, sum_t p_t |v_t|, max_t scale * sum |q||k_t|) for one query row over k, v [token][channel]."""
    s = (k @ q) * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v), float(np.abs(scale) * (np.abs(k) @ np.abs(q)).max())


def prompt_attention(q, k, v, cu, scale):
    """(o, weighted |v|, score size) of packed causal attention; q [token][H_q][D]."""
    g = q.shape[1] // k.shape[1]
    o, w = np.zeros(q.shape), np.zeros(q.shape)
    size = np.zeros(q.shape[:2])
    for lo, hi in zip(cu[:-1], cu[1:]):
        for h in range(q.shape[1]):
            for i in range(lo, hi):
                o[i, h], w[i, h], size[i, h] = attend(q[i, h], k[lo:i + 1, h // g], v[lo:i + 1, h // g], scale)
    return o, w, size
