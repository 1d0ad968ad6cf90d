"""fp64 / integer restatement of the paged 8-bit cache (plan, append, attention) in numpy.

Test infrastructure: plain loops over requests, pages and heads, no code shared with the
library.  e4m3 codes are encoded by searching the table of the 256 code values, so the
encoder shares nothing with rounding arithmetic either.
"""
from __future__ import annotations

import math

import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (NaN for 0x7f and 0xff)."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = math.nan if (c & 0x7f) == 0x7f else (-x if s else x)
    return v


_VAL = e4m3_values()
_POS = _VAL[:0x7f]                       # 0 .. 448 ascending, code = index


def decode(codes: np.ndarray, kv: str) -> np.ndarray:
    return _VAL[codes.astype(np.uint8)] if kv == "e4m3" else codes.astype(np.int8).astype(np.float64)


def encode(y: np.ndarray, kv: str) -> np.ndarray:
    """Nearest code (uint8), ties to the even one, saturating; NaN gives 0."""
    y = np.where(np.isnan(y), 0.0, y)
    if kv == "int8":
        return np.rint(np.clip(y, -127, 127)).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(y), 448.0)
    hi = np.minimum(np.searchsorted(_POS, a, side="left"), 0x7e)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POS[hi] - a, a - _POS[lo]
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(hi % 2 == 0, hi, lo)))
    sign = np.where(np.signbit(y), 0x80, 0).astype(np.int64)
    return (code + sign).astype(np.uint8)


def scale_for(amax: float, kv: str) -> float:
    q = 448.0 if kv == "e4m3" else 127.0
    e = -40
    while e < 40 and amax > q * 2.0 ** e:
        e += 1
    return 2.0 ** e


def plan(kv_len, q_len, table, ring, state, page, max_tokens, held=None):
    """Returns (kv_out, cu, slots, positions, granted, state_out, table, ring), and the pages each
    row has afterwards if `held` says how many it had."""
    table, ring = np.array(table), np.array(ring)
    S, W = table.shape
    N = len(ring)
    head, count = int(state[0]), int(state[1])
    kv_out, cu, granted, held_out = [], [0], [], []
    slots, pos = np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int64)
    tok = taken = back = want = 0
    for s in range(S):
        kv, n = int(kv_len[s]), int(q_len[s])
        old = min(-(-kv // page), W)
        if held is not None:
            old = min(max(old, int(held[s])), W)
        if n < 0:
            for i in range(old):
                if 0 <= table[s, i] < N:             # else a page that is gone
                    ring[(head + count + back) % N] = table[s, i]
                    back += 1
            kv_out.append(0)
            granted.append(1)
            held_out.append(0)
        else:
            new = max(old, -(-(kv + n) // page))
            fits = kv + n <= W * page and tok + n <= max_tokens
            if fits:
                want += new - old
            ok = fits and (new == old or want <= count)
            if ok:
                for i in range(old, new):
                    table[s, i] = ring[(head + taken) % N]
                    taken += 1
                for i in range(n):
                    p = int(table[s, (kv + i) // page])
                    if 0 <= p < N:
                        slots[tok + i] = p * page + (kv + i) % page
                        pos[tok + i] = kv + i
            tok += n
            kv_out.append(kv + n if ok else kv)
            granted.append(int(ok))
            held_out.append(new if ok else old)
        cu.append(min(tok, max_tokens))
    out = kv_out, cu, slots, pos, granted, [(head + taken) % N, count - taken + back], table, ring
    return out if held is None else (*out, held_out)


def append(x, slots, codes, scale, page, kv):
    """One tensor: x [T,H,D] float64, codes uint8 [N,H,P,D] and scale [N,H], updated in place."""
    N = codes.shape[0]
    T, H, _ = x.shape
    t = 0
    while t < T:
        s = int(slots[t])
        if s < 0 or s >= N * page:
            t += 1
            continue
        n = 1
        while t + n < T and slots[t + n] == s + n and (s + n) % page:
            n += 1
        p, off = s // page, s % page
        for h in range(H):
            run = x[t:t + n, h]
            fin = np.abs(run[np.isfinite(run)])
            new = scale_for(float(fin.max()) if fin.size else 0.0, kv)
            old = float(scale[p, h])
            if off:
                if new > old:
                    codes[p, h, :off] = encode(decode(codes[p, h, :off], kv) * old / new, kv)
                else:
                    new = old
            scale[p, h] = new
            codes[p, h, off:off + n] = encode(run / new, kv)
        t += n


def attention(q, kc, vc, ks, vs, table, kv_len, cu, scale, kv):
    """q [T,Hq,D] float64, codes uint8 [N,H,P,D], scales [N,H].  Returns (out, lse) in fp64;
    rows outside every request are NaN."""
    N, H, P, D = kc.shape
    T, Hq, _ = q.shape
    G = Hq // H
    out = np.full((T, Hq, D), math.nan)
    lse = np.full((T, Hq), math.nan)
    for s in range(len(kv_len)):
        a, b, n = int(cu[s]), int(cu[s + 1]), int(kv_len[s])
        if b <= a:
            continue
        pages = np.array(table[s][:-(-n // P)], dtype=np.int64) if n else np.zeros(0, np.int64)
        there = (pages >= 0) & (pages < N)
        pg = np.where(there, pages, 0)
        seen = np.repeat(there, P)[:n]
        for h in range(H):
            k = (decode(kc[pg, h], kv) * ks[pg, h][:, None, None]).reshape(-1, D)[:n]
            v = (decode(vc[pg, h], kv) * vs[pg, h][:, None, None]).reshape(-1, D)[:n]
            for i in range(a, b):
                end = max(0, min(n, n - (b - a) + (i - a) + 1))
                m = seen[:end]
                g = slice(h * G, (h + 1) * G)
                if not m.any():
                    out[i, g], lse[i, g] = 0.0, -math.inf
                    continue
                x = scale * (k[:end][m] @ q[i, g].T)                 # [keys, G]
                top = x.max(0)
                w = np.exp(x - top)
                out[i, g] = (w.T @ v[:end][m]) / w.sum(0)[:, None]
                lse[i, g] = top + np.log(w.sum(0))
    return out, lse
