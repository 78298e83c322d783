"""Plain statements, on the CPU and in 64 bits, of the paged 8-bit cache and the decode step over it, written from the
definitions in ``include/swa_attn.h``: loops over requests, pages and heads, no code shared with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

E_MIN, E_MAX, TOP = -60, 120, 448.0


# ------------------------------------------------------------------------------------------- e4m3

def e4m3_table():
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 significand bits; 0x7f is NaN."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if c & 127 == 127 else -x if s else x
    return out


TABLE = e4m3_table()


def e4m3(x):
    """The nearest e4m3 value (ties to the even code), clamped at 448: a search among the 127 magnitudes."""
    x = np.asarray(x, dtype=np.float64)
    mags = TABLE[:127]
    a = np.minimum(np.abs(x), TOP)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.clip(np.searchsorted(mags, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - mags[lo], mags[hi] - a
    pick = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), np.nan, np.copysign(mags[pick], x))


def exponent(x):
    """The smallest e in [E_MIN, E_MAX] with max |x| <= 448 * 2^e; NaNs do not count."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = x[~np.isnan(x)]
    e = E_MIN
    top = x.max() if x.size else 0.0
    while e < E_MAX and top > TOP * 2.0 ** e:
        e += 1
    return e


class Cache:
    """Codes (as the values they have) and exponents of one tensor's pages."""

    def __init__(self, n_pages, Hkv, P, D):
        self.P, self.Hkv = P, Hkv
        self.codes = np.zeros((n_pages, Hkv, P, D))
        self.e = np.zeros((n_pages, Hkv), dtype=np.int64)

    def write(self, rows, slots):
        """rows (N, Hkv, D) into slots (N,): runs of consecutive slots of one page, head by head."""
        slots = [int(s) for s in slots]
        i = 0
        while i < len(slots):
            if slots[i] < 0:
                i += 1
                continue
            n = 1
            while i + n < len(slots) and slots[i + n] == slots[i] + n and slots[i + n] % self.P:
                n += 1
            page, off = divmod(slots[i], self.P)
            for h in range(self.Hkv):
                x = rows[i:i + n, h]
                e = exponent(x)
                if off > 0 and self.e[page, h] >= e:
                    e = int(self.e[page, h])
                elif off > 0:
                    self.codes[page, h, :off] = e4m3(self.codes[page, h, :off] * 2.0 ** (int(self.e[page, h]) - e))
                self.codes[page, h, off:off + n] = e4m3(x * 2.0 ** -e)
                self.e[page, h] = e
            i += n

    def values(self, slots):
        """(N, Hkv, D) of the given slots, zero rows for negative ones."""
        out = np.zeros((len(slots), self.Hkv, self.codes.shape[-1]))
        for i, s in enumerate(slots):
            if s >= 0:
                page, off = divmod(int(s), self.P)
                out[i] = self.codes[page, :, off] * 2.0 ** self.e[page].astype(float)[:, None]
        return out


# -------------------------------------------------------------------------------------- allocator

class Pages:
    """The allocator, request by request."""

    def __init__(self, B, max_pages, n_pages, P, W):
        self.P, self.W, self.M, self.N = P, W, max_pages, n_pages
        self.table = [[-1] * max_pages for _ in range(B)]
        self.kv_len, self.first = [0] * B, [0] * B
        self.ring, self.head, self.free = list(range(n_pages)), 0, n_pages

    def step(self, n_new, T):
        P, free0, wanted, taken, back = self.P, self.free, 0, 0, []
        slots, step_len = [[-1] * T for _ in n_new], [0] * len(n_new)
        for b, n in enumerate(n_new):
            L, row = self.kv_len[b], self.table[b]
            have = -(-L // P)
            upto = have if n < 0 else max(self.first[b], max(0, L - self.W + 1) // P if self.W > 0 else 0)
            for j in range(self.first[b], upto):
                back.append(row[j])
                row[j] = -1
            self.first[b] = 0 if n < 0 else upto
            if n < 0:
                self.kv_len[b] = 0
                continue
            if n > T or -(-(L + n) // P) > self.M:
                continue
            need = -(-(L + n) // P) - have
            wanted += need
            if n == 0 or (need > 0 and wanted > free0):
                continue
            for j in range(have, have + need):
                row[j] = self.ring[(self.head + taken) % self.N]
                taken += 1
            self.kv_len[b] = step_len[b] = L + n
            for t in range(n):
                slots[b][t] = row[(L + t) // P] * P + (L + t) % P
        for i, page in enumerate(back):
            self.ring[(self.head + free0 + i) % self.N] = page
        self.head = (self.head + taken) % self.N
        self.free = free0 - taken + len(back)
        return slots, step_len


# -------------------------------------------------------------------------------------- attention

def visible(n, window, start):
    lo = max(0, n - window) if window > 0 else 0
    return max(lo, min(start, n - 1))


def attend(q, k, v):
    """One request: q (H, D), k, v (n, Hkv, D) -> out (H, D), lse (H), and sum_j p_j |v_j| (H, D), the scale of the
    error that rounding the weights makes."""
    H, D = q.shape
    G = H // k.shape[1]
    out, lse, mag = np.zeros((H, D)), np.full(H, -np.inf), np.zeros((H, D))
    for h in range(H):
        x = k[:, h // G] @ q[h] / math.sqrt(D)
        top = x.max()
        w = np.exp(x - top)
        lse[h] = top + math.log(w.sum())
        p = w / w.sum()
        out[h], mag[h] = p @ v[:, h // G], p @ np.abs(v[:, h // G])
    return out, lse, mag


def prologue(x, pos, base=10000.0, eps=1e-6):
    """RMS(RoPE(x)) of rows (heads, D) at position pos, exact up to 64 bits (not rounded to bf16)."""
    D = x.shape[-1]
    ang = pos * base ** (-2.0 * np.arange(D // 2) / D)
    a, b = x[:, :D // 2], x[:, D // 2:]
    y = np.concatenate([a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)], 1)
    return y / np.sqrt((y ** 2).mean(1, keepdims=True) + eps)


def out_tolerance(ref, mag):
    """bf16 rounding of the output (half a step: 2^-8 of it); the weights, rounded to 11 bits before the products with v,
    each off by 2^-11 (half of that in the kernel, whose sum is taken before the rounding); fp32 scores and sums, below 2^-13."""
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * mag + 1e-30


def lse_tolerance(lse, D):
    """A score is a sum of D products in fp32, |q| |k| <= D (1 + 2^-4) for unit root mean square rows with k cached, scaled by
    1/sqrt(D): off by (D + 8) 2^-24 sqrt(D) (1 + 2^-4); exp2 and log2 within 2^-20; one rounding of the result."""
    return (D + 8) * 2.0 ** -24 * math.sqrt(D) * (1 + 2.0 ** -4) + 2.0 ** -20 + 2.0 ** -23 * np.abs(lse)
