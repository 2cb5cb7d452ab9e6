"""Plain 64-bit definition of the 8-bit paged cache and the attention that reads it (numpy, CPU).

Test infrastructure only: it shares no code with the CUDA path.  A cache is a dict of numpy arrays
k, v [pages, HKV, page_size, D] uint8 e4m3 codes and k_exp, v_exp [pages, HKV] int8.
"""
from __future__ import annotations

import math

import numpy as np

EXP_MIN, EXP_MAX = -32, 60


def _code_values() -> np.ndarray:
    """The value of each e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if s else x
    return v


CODE = _code_values()
_POS = CODE[:127]  # 0 .. 448, increasing with the code


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code of each value, ties to the even code, saturating at 448; a zero keeps its sign."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (pick + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def block_exponent(amax: float) -> int:
    e = EXP_MIN
    while e < EXP_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(cache: dict, k_new, v_new, lens, starts, table, page_size: int) -> None:
    """Quantises rows (packed [T, HKV, D]) into the cache in place; starts[n] < 0 is padding."""
    for name, new in (("k", k_new), ("v", v_new)):
        codes, exps = cache[name], cache[name + "_exp"]
        row0 = 0
        for n, L in enumerate(lens):
            t, end = starts[n], starts[n] + L
            while starts[n] >= 0 and t < end:
                page, r0 = table[n][t // page_size], t % page_size
                m = min(page_size - r0, end - t)
                x = np.asarray(new[row0 + t - starts[n]:row0 + t - starts[n] + m], dtype=np.float64)
                for h in range(x.shape[1]):
                    y = x[:, h]
                    fin = np.abs(y[np.isfinite(y)])
                    e = block_exponent(float(fin.max()) if fin.size else 0.0)
                    if r0:
                        old = int(exps[page, h])
                        e = max(e, old)
                        if e > old:
                            codes[page, h, :r0] = encode(CODE[codes[page, h, :r0]] * 2.0 ** (old - e))
                    exps[page, h] = e
                    codes[page, h, r0:r0 + m] = encode(np.where(np.isnan(y), 0.0, y) * 2.0 ** -e)
                t += m
            row0 += L


def values(cache: dict, name: str, pages, h: int, count: int) -> np.ndarray:
    """[count, D]: the first `count` cached tokens of a request's pages, key/value head h."""
    x = CODE[cache[name][pages, h]] * 2.0 ** cache[name + "_exp"][pages, h].astype(np.float64)[:, None, None]
    return x.reshape(-1, x.shape[-1])[:count]


def attend(cache: dict, q, lens, kv_lens, table, page_size: int, scale: float = 0.0, cap: float = 0.0,
           window: int = 0, slopes=None, prefix=None, parents=None, faint: bool = False):
    """(out, lse, spread, reach) for packed rows q [T, HQ, D]; spread [T, HQ, D] = sum_j p_j |v_j| and reach
    [T, HQ] = the largest scale * sum_d |q_d k_jd| over visible tokens, for error bounds.  With `faint` a fifth array
    [T, HQ, D]: the sum of |code_jd| over visible tokens times the largest p_j 2^(value exponent of j) among them,
    the scale of errors of weights that are small beside that."""
    q = np.asarray(q, dtype=np.float64)
    T, HQ, D = q.shape
    HKV = cache["k"].shape[1]
    G = HQ // HKV
    scale = scale if scale > 0 else 1.0 / math.sqrt(D)
    out, spread = np.zeros((T, HQ, D)), np.zeros((T, HQ, D))
    lse, reach = np.full((T, HQ), -np.inf), np.zeros((T, HQ))
    far = np.zeros((T, HQ, D))
    row0 = 0
    for n, L in enumerate(lens):
        kv = int(kv_lens[n])
        if kv <= 0 or kv < L:
            row0 += L
            continue
        base = kv - L
        pos_k = np.arange(kv)
        pos_q = np.arange(base, kv)
        sees = pos_k[None, :] <= pos_q[:, None]
        if parents is not None:
            sees[:, base:] = False
            for t in range(L):
                u, depth = t, -1
                while u >= 0:
                    sees[t, base + u] = True
                    u, depth = int(parents[n][u]), depth + 1
                pos_q[t] = base + depth
            pos_k = np.concatenate([pos_k[:base], pos_q])
        dist = pos_q[:, None] - pos_k[None, :]
        if window > 0:
            sees &= dist < window
        if prefix is not None:
            sees |= np.arange(kv)[None, :] < int(prefix[n])
        pages = np.asarray(table[n][: -(-kv // page_size)])
        used = np.zeros(len(pages), dtype=bool)  # pages that no row sees may be absent (any entry) or hold anything
        used[np.unique(np.nonzero(sees.any(0))[0] // page_size)] = True
        pages = np.where(used, pages, 0)
        live = sees.any(0)
        for h in range(HKV):
            K = np.where(live[:, None], values(cache, "k", pages, h, kv), 0.0)
            V = np.where(live[:, None], values(cache, "v", pages, h, kv), 0.0)
            step = np.repeat(2.0 ** cache["v_exp"][pages, h].astype(np.float64), page_size)[:kv]
            for g in range(h * G, h * G + G):
                x = q[row0:row0 + L, g]
                s = scale * x @ K.T
                if cap > 0:
                    s = cap * np.tanh(s / cap)
                if slopes is not None:
                    s = s - float(slopes[g]) * np.abs(dist)
                s = np.where(sees, s, -np.inf)
                m = s.max(-1, keepdims=True)
                w = np.exp(s - np.where(np.isfinite(m), m, 0.0))
                l = w.sum(-1, keepdims=True)
                some = l[:, 0] > 0
                p = w / np.where(l > 0, l, 1.0)
                out[row0:row0 + L, g] = p @ V
                spread[row0:row0 + L, g] = p @ np.abs(V)
                if faint:
                    far[row0:row0 + L, g] = (p * step).max(-1, keepdims=True) * (sees @ np.abs(V / step[:, None]))
                lse[row0:row0 + L, g][some] = (m + np.log(np.where(l > 0, l, 1.0)))[some, 0]
                reach[row0:row0 + L, g] = np.where(sees, scale * np.abs(x) @ np.abs(K).T, 0.0).max(-1)
        row0 += L
    return (out, lse, spread, reach, far) if faint else (out, lse, spread, reach)
