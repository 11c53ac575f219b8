"""Plain reference of the paged cache in 64 bits, on the CPU: attention, the
cache writer and the pages' bookkeeping, straight from their definitions
(include/fd_paged_attn.h) and sharing no code with the library."""

from __future__ import annotations

import math

import numpy as np

BF16, E4M3 = 0, 1
NAN_CODE = 0x7F


def e4m3_table() -> np.ndarray:
    """Values of the 256 codes: 1 sign, 4 exponent (bias 7), 3 fraction bits; x1111111 is NaN, no infinity."""
    out = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if c & 127 == 127:
            v = math.nan
        out[c] = -v if c & 128 else v
    return out


TABLE = e4m3_table()
_MAG = TABLE[:127]


def e4m3_code(x: np.ndarray) -> np.ndarray:
    """Nearest code of each value, ties to the even code, saturating at 448; NaN gives NAN_CODE."""
    x = np.asarray(x, dtype=np.float64)
    m = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.minimum(np.searchsorted(_MAG, m), 126)
    lo = np.maximum(hi - 1, 0)
    below, above = m - _MAG[lo], _MAG[hi] - m
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), NAN_CODE, code).astype(np.uint8)


def block_scale(amax: float) -> float:
    if amax == 0:
        return 0.0
    k = -126
    e = math.frexp(amax)[1]
    for t in range(max(-126, e - 12), e + 3):  # the least power of two, by trying
        if amax <= 448 * 2.0 ** t:
            k = t
            break
    return 2.0 ** k


def attend(q, k, v, ks, vs, table, lens, window, scale, num_pages):
    """q [B,NH,HS] float64; k, v [num_pages,NKV,P,HS] float64 values (bf16) or uint8 codes with ks, vs [num_pages,NKV].
    Returns out float64 and, for each (b, h), the largest |V| that takes part and the largest scale * sum |q_d k_d|."""
    B, NH, HS = q.shape
    NKV, P = k.shape[1], k.shape[2]
    G = NH // NKV
    out, big, mass = np.zeros((B, NH, HS)), np.zeros((B, NH)), np.zeros((B, NH))
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * P)
        pos = np.arange(max(0, n - window) if window > 0 else 0, n)
        pages = table[b][pos // P]
        ok = (pages >= 0) & (pages < num_pages)
        pages, slot = pages[ok], pos[ok] % P
        if not len(pages):
            continue
        for h in range(NKV):
            kk, vv = k[pages, h, slot], v[pages, h, slot]
            if ks is not None:
                kk = TABLE[kk] * ks[pages, h].astype(np.float64)[:, None]
                vv = TABLE[vv] * vs[pages, h].astype(np.float64)[:, None]
            qq = q[b, h * G:(h + 1) * G]
            s = qq @ kk.T * scale
            p = np.exp(s - s.max(1, keepdims=True))
            out[b, h * G:(h + 1) * G] = (p / p.sum(1, keepdims=True)) @ vv
            big[b, h * G:(h + 1) * G] = np.abs(vv).max()
            mass[b, h * G:(h + 1) * G] = (np.abs(qq) @ np.abs(kk).T * scale).max(1)
    return out, big, mass


def append(new, pool, scale, table, lens, start, count, num_pages):
    """Writes new float64 [T,NKV,HS] into pool (float64 values, or uint8 codes with scale [num_pages,NKV]), in place."""
    T = new.shape[0]
    P = pool.shape[2]
    for b in range(len(lens)):
        r0 = int(start[b]) if start is not None else b
        n = int(start[b + 1]) - r0 if start is not None else 1
        if count is not None:
            n = min(n, max(int(count[b]), 0))
        todo = {}
        for i in range(max(n, 0)):
            row, pos = r0 + i, int(lens[b]) - n + i
            if 0 <= row < T and pos >= 0 and pos // P < table.shape[1]:
                todo.setdefault(pos // P, []).append((row, pos % P))
        for j, tokens in todo.items():
            page = int(table[b][j])
            if not 0 <= page < num_pages:
                continue
            rows, slots = [t[0] for t in tokens], [t[1] for t in tokens]
            for h in range(new.shape[1]):
                x = new[rows, h]
                if scale is None:
                    pool[page, h, slots] = x
                    continue
                finite = np.isfinite(x)
                s = block_scale(float(np.abs(np.where(finite, x, 0.0)).max()))
                old = float(scale[page, h]) if slots[0] > 0 else 0.0
                s = max(s, old)
                if slots[0] > 0 and s > old:
                    pool[page, h, :slots[0]] = e4m3_code(TABLE[pool[page, h, :slots[0]]] * (old / s))
                pool[page, h, slots] = e4m3_code(np.where(finite, x / s if s > 0 else 0.0, math.nan))
                scale[page, h] = s


class Book:
    """table, lens, refs as lists, and the operations on them."""

    def __init__(self, table, lens, refs, P):
        self.table, self.lens, self.refs, self.P = table.copy(), lens.copy(), refs.copy(), P

    def reserve(self, grow):
        P, (B, wide) = self.P, self.table.shape
        free = [p for p in range(len(self.refs)) if self.refs[p] <= 0]
        refs0, upto, granted, moves, lost, taken = self.refs.copy(), 0, [0] * B, [], [], 0
        for b in range(B):
            n, old = max(int(grow[b]), 0), max(int(self.lens[b]), 0)
            if n == 0:
                continue
            have, want = -(-old // P), -(-(old + n) // P)
            if want > wide:
                continue
            shared, last = 0, -1
            if old % P:
                last = int(self.table[b][old // P])
                if not 0 <= last < len(self.refs):
                    continue
                shared = int(refs0[last] > 1)
            need = want - have + shared
            begin, upto = upto, upto + need
            if need and upto > len(free):
                continue
            pages = free[begin:begin + need]
            taken += need
            if shared:
                moves.append((last, pages[0]))
                lost.append(last)
                self.table[b][old // P] = pages.pop(0)
                self.refs[moves[-1][1]] = 1
            for i, p in enumerate(pages):
                self.table[b][have + i] = p
                self.refs[p] = 1
            granted[b] = n
            self.lens[b] = old + n
        for p in lost:
            self.refs[p] -= 1
        return granted, moves, len(free) - taken

    def fork(self, parent):
        wide = self.table.shape[1]
        table = np.full((len(parent), wide), -1, dtype=np.int32)
        lens = np.zeros(len(parent), dtype=np.int32)
        for row in self.table:
            for p in row[row >= 0]:
                self.refs[p] -= 1
        for i, f in enumerate(parent):
            if 0 <= f < len(self.lens):
                table[i], lens[i] = self.table[f], self.lens[f]
        for row in table:
            for p in row[row >= 0]:
                self.refs[p] += 1
        self.table, self.lens = table, lens

    def free(self, keep, window):
        for b in range(len(self.lens)):
            n = max(int(self.lens[b]), 0)
            n = n if keep is None else min(n, max(int(keep[b]), 0))
            self.lens[b] = n
            first = max(0, n - window) // self.P if window > 0 else 0
            for j in range(self.table.shape[1]):
                if not first <= j < -(-n // self.P) and self.table[b][j] >= 0:
                    self.refs[self.table[b][j]] -= 1
                    self.table[b][j] = -1

    def compact(self):
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        n = len(used)
        src = [p for p in used if p >= n]
        dst = [p for p in range(n) if self.refs[p] <= 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = np.array([[to.get(int(p), int(p)) for p in row] for row in self.table], dtype=np.int32)
        return list(to.items()), len(self.refs) - n
