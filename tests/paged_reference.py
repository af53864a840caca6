"""Plain 64-bit implementation of the paged 8-bit cache (numpy, loops over sequences and
pages): what include/lowram.h defines, written apart from the kernels."""
import math

import numpy as np


def e4m3_table() -> np.ndarray:
    """Value of every e4m3 byte (fp64): 4 exponent bits of bias 7, 3 fraction bits."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        mag = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if c & 127 == 127:
            mag = math.nan
        out[c] = -mag if c & 128 else mag
    return out


TABLE = e4m3_table()
_POS = TABLE[:127]                       # ascending: 0 .. 448


def decode(codes) -> np.ndarray:
    return TABLE[np.asarray(codes, np.uint8)]


def encode(x) -> np.ndarray:
    """Nearest e4m3 code of |x| <= 448 (ties to the even code), 0x7f for non-finite x."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    a = np.abs(np.where(fin, x, 0.0))
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(fin, code, 0x7f).astype(np.uint8)


def scale_for(amax: float) -> float:
    e = -64
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x, pos, theta):
    """Rotate-half rotation of x [..., d] by positions pos (broadcast over x.shape[:-1])."""
    d = x.shape[-1]
    th = np.power(float(theta), -2.0 * np.arange(d // 2) / d)
    ang = np.asarray(pos, np.float64)[..., None] * th
    c, s = np.cos(ang), np.sin(ang)
    a, b = x[..., : d // 2], x[..., d // 2:]
    return np.concatenate([a * c - b * s, a * s + b * c], axis=-1)


class Pages:
    """k_code, v_code uint8 [n_pages][H][P][d]; k_scale, v_scale fp64 [n_pages][H]."""

    def __init__(self, k_code, v_code, k_scale, v_scale):
        self.code = {"k": np.array(k_code), "v": np.array(v_code)}
        self.scale = {"k": np.array(k_scale, np.float64), "v": np.array(v_scale, np.float64)}

    @property
    def page_tokens(self):
        return self.code["k"].shape[2]

    def values(self, name, pages, n):
        """Tokens 0 .. n-1 of a page list: [n][H][d]."""
        P = self.page_tokens
        pages = list(pages)[: -(-n // P)]
        if not pages:
            _, H, _, d = self.code[name].shape
            return np.zeros((0, H, d))
        x = decode(self.code[name][pages]) * self.scale[name][pages][:, :, None, None]
        x = x.transpose(0, 2, 1, 3)
        return x.reshape(-1, *x.shape[2:])[:n]

    def append(self, table, lens, k_new, v_new, counts, base, theta, rotate_keys=True):
        """k_new, v_new fp64 [n][H][d]. Returns {name: fp64 array of the values written,
        before rounding, NaN elsewhere} beside the updated pages."""
        P = self.page_tokens
        wrote = {n: np.full(self.code[n].shape, np.nan) for n in ("k", "v")}
        at = 0
        for b, n in enumerate(counts):
            first = lens[b] - n
            pos = base[b] + first + np.arange(n)
            rows = {"k": k_new[at:at + n], "v": v_new[at:at + n]}
            if rotate_keys and n:
                rows["k"] = rotate(rows["k"], pos[:, None], theta)
            at += n
            for p in range(first // P, -(-lens[b] // P) if n else 0):
                lo, hi = max(first, p * P), min(lens[b], (p + 1) * P)
                g = table[b][p]
                for name in ("k", "v"):
                    for h in range(k_new.shape[1]):
                        x = rows[name][lo - first:hi - first, h].astype(np.float32).astype(np.float64)
                        fin = np.abs(x[np.isfinite(x)])
                        s = scale_for(fin.max() if fin.size else 0.0)
                        if lo > p * P:
                            old = self.scale[name][g, h]
                            s = max(s, old)
                            head = self.code[name][g, h, : lo - p * P]
                            if s > old:
                                head[...] = encode(decode(head) * (old / s))
                        self.scale[name][g, h] = s
                        self.code[name][g, h, lo - p * P:hi - p * P] = encode(x / s)
                        wrote[name][g, h, lo - p * P:hi - p * P] = rows[name][lo - first:hi - first, h]
        return wrote

    def attend(self, table, lens, q, group):
        """q fp64 [B][n_q][H_q][d]. Returns out, lse, sum p |v|, the largest sum |q_i k_i| /
        sqrt(d) of a row (the last two scale the error bounds)."""
        B, nq, hq, d = q.shape
        out = np.zeros(q.shape)
        lse = np.full((B, nq, hq), -np.inf)
        absv = np.zeros(q.shape)
        zabs = np.zeros((B, nq, hq))
        for b in range(B):
            k, v = (self.values(x, table[b], lens[b]) for x in ("k", "v"))
            for j in range(nq):
                n = lens[b] - nq + j + 1
                if n <= 0:
                    continue
                for i in range(hq):
                    kk, vv = k[:n, i // group], v[:n, i // group]
                    z = kk @ q[b, j, i] / math.sqrt(d)
                    m = z.max()
                    e = np.exp(z - m)
                    l = e.sum()
                    out[b, j, i] = e @ vv / l
                    lse[b, j, i] = m + math.log(l)
                    absv[b, j, i] = e @ np.abs(vv) / l
                    zabs[b, j, i] = (np.abs(kk) @ np.abs(q[b, j, i])).max() / math.sqrt(d)
        return out, lse, absv, zabs
