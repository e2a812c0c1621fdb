"""Plain references for the rotary positions and the 4-bit cache (not
collected by pytest): the definitions of ikbo.h in numpy / torch on the CPU,
in 64 bits except where the definition itself rounds.
"""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 2560


def bf16(x: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16 (nearest even), as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


# ------------------------------------------------------------------- rope
def rope_ref(x: np.ndarray, pos: np.ndarray, freqs, interleaved=False, magnitude=1.0, backward=False) -> np.ndarray:
    """x [n, H, L, d] float64, pos [n, L]; a rotation of the first 2 * len(freqs) elements."""
    half = len(freqs)
    y = np.array(x, dtype=np.float64)
    for j, f in enumerate(freqs):
        # whole turns leave before the product loses bits (positions are whole numbers)
        turns = np.longdouble(f) / (2 * np.longdouble(math.pi) + np.longdouble(2.4492935982947064e-16))
        part = pos.astype(np.longdouble) * turns
        a = ((part - np.floor(part)) * 2 * np.pi).astype(np.float64)[:, None, :]
        c, s = np.cos(a) * magnitude, np.sin(a) * magnitude * (-1 if backward else 1)
        i, k = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        y[..., i] = x[..., i] * c - x[..., k] * s
        y[..., k] = x[..., k] * c + x[..., i] * s
    return y


# ------------------------------------------------------------- quantising
def quantise(x: np.ndarray):
    """bf16 values (as fp32) [..., 128] -> codes [..., 4, 32], s and z [..., 4] (fp32 holding bf16)."""
    v = x.astype(np.float32).reshape(x.shape[:-1] + (4, 32))
    with np.errstate(all="ignore"):
        lo, hi = v.min(-1), v.max(-1)  # NaN where the group holds one
        s = bf16((hi * np.float32(0.5) - lo * np.float32(0.5)) / np.float32(7.5))
        z = bf16(lo - np.float32(16) * s)
        bad = ~(np.isfinite(s) & np.isfinite(z))
        s, z = np.where(bad, np.float32(np.nan), s), np.where(bad, np.float32(np.nan), z)
        q = (v - z[..., None]) / s[..., None]
        c = np.clip(np.rint(q) - 16, 0, 15)
        c = np.where((s > 0)[..., None], c, 0)
    return c.astype(np.uint8), s, z


def values(c, s, z) -> np.ndarray:
    with np.errstate(all="ignore"):
        v = z[..., None].astype(np.float64) + (16.0 + c.astype(np.float64)) * s[..., None].astype(np.float64)
        return bf16(v.astype(np.float32)).reshape(c.shape[:-2] + (128,))


def pairs_bytes(s, z) -> np.ndarray:
    """[..., 4] -> the 16 bytes of a token's pairs."""
    t = torch.from_numpy(np.stack([s, z], axis=-1).astype(np.float32)).to(torch.bfloat16)
    return t.view(torch.uint8).numpy().reshape(s.shape[:-1] + (16,))


def codes_bytes(c) -> np.ndarray:
    n = c.reshape(c.shape[:-2] + (64, 2))
    return (n[..., 0] | (n[..., 1] << 4)).astype(np.uint8)


def store(data: np.ndarray, page: int, slots, K: np.ndarray, V: np.ndarray) -> None:
    """Write rows K, V [n, H, 128] (bf16 as fp32) into data [n_pages, H, page / 16, 2560] in place."""
    for r, slot in enumerate(slots):
        if slot < 0:
            continue
        pg, place = divmod(int(slot), page)
        blk, row = divmod(place, 16)
        for which, x in enumerate((K, V)):
            c, s, z = quantise(x[r])
            at = which * 1280
            data[pg, :, blk, at + row * 64:at + row * 64 + 64] = codes_bytes(c)
            data[pg, :, blk, at + 1024 + row * 16:at + 1024 + row * 16 + 16] = pairs_bytes(s, z)


def nan_safe_equal(a: np.ndarray, b: np.ndarray) -> bool:
    """Byte equality of two caches, any two bf16 NaNs in a pair counting as equal."""
    if np.array_equal(a, b):
        return True
    for at in (0, 1280):
        if not np.array_equal(a[..., at:at + 1024], b[..., at:at + 1024]):
            return False
        pa = np.ascontiguousarray(a[..., at + 1024:at + 1280]).view(np.uint16)
        pb = np.ascontiguousarray(b[..., at + 1024:at + 1280]).view(np.uint16)
        nan = ((pa & 0x7fff) > 0x7f80) & ((pb & 0x7fff) > 0x7f80)
        if not np.array_equal(pa[~nan], pb[~nan]):
            return False
    return True


def read(data: np.ndarray, page: int, row_of_table, length: int):
    """K, V [length, H, 128] (fp32 holding bf16) of one user."""
    H = data.shape[1]
    out = np.zeros((2, length, H, 128), dtype=np.float32)
    t = np.arange(length)
    pg = np.asarray(row_of_table)[t // page].astype(np.int64)
    blk, row = (t % page) // 16, t % 16
    for which in range(2):
        at = which * 1280
        raw = data[pg, :, blk]  # [length, H, 2560]
        idx = at + row[:, None] * 64 + np.arange(64)[None, :]
        codes = np.take_along_axis(raw, np.broadcast_to(idx[:, None, :], (length, H, 64)), axis=2)
        c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(length, H, 4, 32)
        idx = at + 1024 + row[:, None] * 16 + np.arange(16)[None, :]
        p = np.take_along_axis(raw, np.broadcast_to(idx[:, None, :], (length, H, 16)), axis=2)
        p = np.ascontiguousarray(p).reshape(-1).view(np.uint16).astype(np.uint32) << 16
        p = p.view(np.float32).reshape(length, H, 4, 2)
        out[which] = values(c, p[..., 0], p[..., 1])
    return out[0], out[1]


# ----------------------------------------------------------------- tables
def resize(lens, new_lens, table, page, free, n_free, max_new):
    """The definition of ikbo_qcache_resize, one page and token at a time; all
    or nothing.  Returns (ok, lens, table, free, n_free, slots, offsets, positions)."""
    lens, new = [int(x) for x in lens], [int(x) for x in new_lens]
    old = (list(lens), table.copy(), free.copy(), n_free)
    U, B = table.shape
    n_pages = len(free)
    refused = (False, np.array(old[0], np.int32), old[1], old[2], n_free, np.full(max_new, -1, np.int32),
               np.zeros(U + 1, np.int32), np.zeros(max_new, np.int32))
    if any(not 0 <= x <= B * page for x in lens + new) or not 0 <= n_free <= n_pages:
        return refused
    have, need = [-(-x // page) for x in lens], [-(-x // page) for x in new]
    takes = sum(max(0, b - a) for a, b in zip(have, need))
    tokens = sum(max(0, b - a) for a, b in zip(lens, new))
    gives = sum(max(0, a - b) for a, b in zip(have, need))
    if takes > n_free or tokens > max_new or n_free - takes + gives > n_pages:
        return refused
    table, free = table.copy(), free.copy()
    k = 0
    for u in range(U):
        for b in range(have[u], need[u]):
            table[u, b] = free[n_free - 1 - k]
            k += 1
    slots, positions, offsets = np.full(max_new, -1, np.int32), np.zeros(max_new, np.int32), [0]
    i = 0
    for u in range(U):
        for pos in range(lens[u], new[u]):
            slots[i] = table[u, pos // page] * page + pos % page
            positions[i] = pos
            i += 1
        offsets.append(i)
    r = 0
    for u in range(U):
        for b in range(need[u], have[u]):
            free[n_free - takes + r] = table[u, b]
            table[u, b] = -1
            r += 1
    return True, np.array(new, np.int32), table, free, n_free - takes + gives, slots, np.array(offsets, np.int32), positions


# -------------------------------------------------------------- attention
def attend(Q: np.ndarray, kv, map_, H_kv: int, scale: float):
    """O, lse and the error bound of O for every row, in float64.

    Q [n, H, Lq, 128]; kv[u] = (K, V) [L_u, H_kv, 128].  The bound counts what
    the kernels round: each p to bf16 (2^-8 of sum p |v|), the output to bf16
    (2^-8), and the scores: 128 products accumulated in fp32, each addition off
    by at most 2^-23 of the partial sum (<= sum |q k|), and 2^-20 for exp2 and
    its argument; a relative error e of every p moves O by at most 2 e sum p |v|.
    """
    n, H, Lq, d = Q.shape
    O = np.zeros(Q.shape)
    lse = np.full((n, H, Lq), -np.inf)
    bound = np.zeros(Q.shape)
    for i in range(n):
        u = int(map_[i])
        if not 0 <= u < len(kv):
            continue
        K, V = kv[u]
        if len(K) == 0:
            continue
        for h in range(H):
            k, v = K[:, h // (H // H_kv)].astype(np.float64), V[:, h // (H // H_kv)].astype(np.float64)
            q = Q[i, h].astype(np.float64)
            s = scale * q @ k.T
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(-1, keepdims=True)
            O[i, h] = p @ v / l
            lse[i, h] = (m + np.log(l))[:, 0]
            mass = p @ np.abs(v) / l
            e = 2.0 ** -16 * scale * (np.abs(q) @ np.abs(k).T).max(-1, keepdims=True) + 2.0 ** -20
            bound[i, h] = 2.0 ** -8 * mass + 2.0 ** -8 * np.abs(O[i, h]) + 2 * e * mass + 1e-30
    return O, lse, bound


class Store:
    """A small cache on the host: pages in a shuffled order, NaN pairs wherever
    nothing was written (so that a kernel that uses them shows)."""

    def __init__(self, seed: int, lens, H: int, page: int, spare: int = 3, outlier: float = 4.0):
        rng = np.random.default_rng(seed)
        self.page, self.H, self.lens = page, H, np.asarray(lens, dtype=np.int32)
        blocks = [-(-int(x) // page) for x in lens]
        self.n_pages = sum(blocks) + spare
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(lens), max(1, max(blocks))), -1, np.int32)
        at = 0
        for u, b in enumerate(blocks):
            self.table[u, :b] = order[at:at + b]
            at += b
        self.data = np.full((self.n_pages, H, page // 16, BLOCK), 0xFF, np.uint8)
        self.kv = []
        for u, L in enumerate(self.lens):
            K = rng.standard_normal((L, H, 128)).astype(np.float32)
            K[..., 7::41] *= outlier
            K, V = bf16(K), bf16(rng.standard_normal((L, H, 128)))
            slots = [int(self.table[u, t // page]) * page + t % page for t in range(L)]
            store(self.data, page, slots, K, V)
            self.kv.append(read(self.data, page, self.table[u], int(L)))

    def cuda(self):
        return (torch.from_numpy(self.data).cuda(), torch.from_numpy(self.table).cuda(),
                torch.from_numpy(self.lens).cuda())
