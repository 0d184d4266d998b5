"""Plain implementations, in 64 bits on the CPU, of the decode-step operators,
and the inputs their tests share."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def bf16(a) -> torch.Tensor:
    return torch.as_tensor(np.asarray(a)).to(torch.bfloat16)


# ---- 4-bit linear -----------------------------------------------------------

def w4_dequant(fmt, q, scale, zero, group):
    """[N][K] float64 weights and the magnitudes |scale| (|code| + |zero|) that
    the sums are formed from."""
    N, K2 = q.shape
    codes = np.empty((N, 2 * K2), np.int64)
    codes[:, 0::2], codes[:, 1::2] = q & 15, q >> 4
    g = np.arange(2 * K2) // group
    if fmt == "fp4":
        s = np.ldexp(1.0, scale.astype(int) - 127)
        s[scale == 255] = np.nan
        w = E2M1[codes] * s[:, g]
        return w, np.abs(w)
    s = scale.double().numpy()[:, g]
    z = (zero[:, g] if zero is not None else np.full_like(codes, 8)).astype(np.float64)
    return s * (codes - z), np.abs(s) * (codes + z)


# ---- rotation and cache ---------------------------------------------------------

def rope_table(rows, rot):
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)[None]
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rotate_f32(x, table_rows, rot, pairs):
    """x [T][H][D] float32, rotated with every operation rounded to float32."""
    x = x.copy()
    if rot == 0:
        return x
    c, s = table_rows[:, None, :rot // 2], table_rows[:, None, rot // 2:]
    ia = np.arange(0, rot, 2) if pairs else np.arange(rot // 2)
    ib = ia + 1 if pairs else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def fp8_rows(x):
    """E4M3 codes (uint8) and float32 scales of float32 rows [..., D]."""
    amax = np.abs(x).max(-1)
    s = (amax / np.float32(448)).astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(amax[..., None] == 0, np.float32(0), x / s[..., None])
    codes = torch.from_numpy(q.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes, s


class Cache:
    """A paged cache on the CPU: float64 values of K and V and the tensors as
    the library takes them."""

    def __init__(self, rng, n_pages, page, Hkv, D, fp8, fill=None):
        self.page, self.fp8 = page, fp8
        shape = (n_pages, Hkv, page, D)
        self.t = {}
        for n in "kv":
            x = rng.standard_normal(shape).astype(np.float32)
            if fp8:
                codes, s = fp8_rows(x)
                self.t[n], self.t[n + "s"] = torch.from_numpy(codes), torch.from_numpy(s)
            else:
                self.t[n], self.t[n + "s"] = bf16(x), None

    def values(self, n):
        if not self.fp8:
            return self.t[n].double().numpy()
        return self.t[n].view(torch.float8_e4m3fn).double().numpy() * \
            self.t[n + "s"].double().numpy()[..., None]


def attention(q, kv, pos, prefix_pages, P, table, scale, Q, max_keys):
    """q [T][Hq][D] float64.  Returns o, lse, sum p|v| and the largest sum |q k|
    of each row (float64); rows that see nothing: 0, -inf, 0, 0."""
    T, Hq, D = q.shape
    K, V = kv.values("k"), kv.values("v")
    n_pages, Hkv, page = K.shape[:3]
    G = Hq // Hkv
    o, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, qk = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for t in range(T):
        j = np.arange(min(pos[t] + 1, max_keys))
        pg = np.array([prefix_pages[i // page] if i < P else table[t // Q][i // page] for i in j], int)
        ok = (pg >= 0) & (pg < n_pages)
        j, pg = j[ok], pg[ok]
        if not len(j):
            continue
        for h in range(Hq):
            k, v = K[pg, h // G, j % page], V[pg, h // G, j % page]
            s = k @ q[t, h] * scale
            m = s.max()
            if m == -np.inf:
                continue
            e = np.exp(s - m)
            p = e / e.sum()
            o[t, h], mag[t, h] = p @ v, p @ np.abs(v)
            lse[t, h] = m + np.log(e.sum())
            qk[t, h] = (np.abs(k) @ np.abs(q[t, h])).max() * scale
    return o, lse, mag, qk
