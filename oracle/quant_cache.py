"""Float64 oracle of the quantised paged cache: its format, write and read, and the decode operators
that read it (softmax rows, mapped product, attention).

The textbook definitions of softmax attention are those of the other oracles [GLIDE II-B], the mapped
decode step that of [IAM-4]; the format is the one include/iamap.h states. Everything is numpy, the
rounding to fp16 is numpy's (to nearest even).
"""

from __future__ import annotations

import math

import numpy as np

LEVELS = {4: 7, 8: 127}
GROUP = 32


def quantise(x: np.ndarray, bits: int):
    """(codes int [..., d], scales float16 [..., d / 32]) of float64 rows x [..., d]."""
    q = LEVELS[bits]
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    with np.errstate(all="ignore"):
        m = np.abs(g).max(axis=-1)
        bad = ~np.isfinite(m)
        s = np.where(bad, 1.0, np.minimum(m / q, 65504.0)).astype(np.float16)
        c = np.rint(g / s.astype(np.float64)[..., None])
        c = np.where((s > 0)[..., None] & ~bad[..., None], np.clip(c, -q, q), 0.0)
    s[bad] = np.float16(np.nan)
    return c.reshape(x.shape).astype(np.int64), s


def place(d: int) -> np.ndarray:
    """Code number at which element e of a row is stored."""
    e = np.arange(d)
    return ((e % GROUP) // 4) * (d // 8) + (e // GROUP) * 4 + e % 4


def pack(codes: np.ndarray, bits: int) -> np.ndarray:
    """Stored bytes uint8 [..., d * bits / 8] of codes [..., d] in element order."""
    d = codes.shape[-1]
    u = np.empty(codes.shape, dtype=np.uint8)
    u[..., place(d)] = (codes + (8 if bits == 4 else 128)).astype(np.uint8)
    return u if bits == 8 else (u[..., 0::2] | (u[..., 1::2] << 4))


def unpack(stored: np.ndarray, bits: int) -> np.ndarray:
    """Codes [..., d] in element order of stored bytes."""
    if bits == 8:
        u = stored.astype(np.int64) - 128
    else:
        u = np.empty(stored.shape[:-1] + (stored.shape[-1] * 2,), dtype=np.int64)
        u[..., 0::2] = (stored & 15).astype(np.int64) - 8
        u[..., 1::2] = (stored >> 4).astype(np.int64) - 8
    return u[..., place(u.shape[-1])]


def values(stored: np.ndarray, scales: np.ndarray, bits: int) -> np.ndarray:
    """float64 rows that stored rows stand for."""
    c = unpack(stored, bits)
    return c * np.repeat(scales.astype(np.float64), GROUP, axis=-1)


def slots(cu, starts, page_table, page_size: int, num_pages: int, n: int):
    """(rows, pages, slots) of the packed rows that have a place, and the number that have none
    although they belong to a sequence."""
    rows, pages, slot, bad = [], [], [], 0
    for s in range(len(starts)):
        for i in range(int(cu[s]), min(int(cu[s + 1]), n)):
            pos = int(starts[s]) + i - int(cu[s])
            if 0 <= pos < page_table.shape[1] * page_size:
                pg = int(page_table[s, pos // page_size])
                if 0 <= pg < num_pages:
                    rows.append(i)
                    pages.append(pg)
                    slot.append(pos % page_size)
                    continue
            bad += 1
    as_int = lambda v: np.asarray(v, dtype=np.int64)  # noqa: E731
    return as_int(rows), as_int(pages), as_int(slot), bad


def sequence(pool, scales, bits, page_table, b, n, page_size):
    """float64 [n, H, d] rows of sequence b's first n tokens, and which of them have a page."""
    pos = np.arange(n)
    pg = page_table[b, pos // page_size].astype(np.int64)
    ok = (pg >= 0) & (pg < pool.shape[0])
    pg = np.where(ok, pg, 0)
    v = values(pool[pg, :, pos % page_size], scales[pg, :, pos % page_size], bits)
    return np.where(ok[:, None, None], v, 0.0), ok


def softmax_rows(q, pool, scales, bits, page_table, ctx_lens, page_size, stride):
    """p [batch, Hq, stride] and log-sum-exp [batch, Hq] of one query row q[b, h] a head (float64)
    over the first ctx_lens[b] cached keys, key head h // (Hq / H)."""
    batch, hq, d = q.shape
    rep = hq // pool.shape[1]
    p = np.zeros((batch, hq, stride))
    lse = np.full((batch, hq), -np.inf)
    for b in range(batch):
        n = int(ctx_lens[b])
        k, ok = sequence(pool, scales, bits, page_table, b, n, page_size)
        if not ok.any():
            continue
        x = np.einsum("hd,nhd->hn", q[b], np.repeat(k, rep, axis=1)) / math.sqrt(d)
        x = np.where(ok, x, -np.inf)
        m = x.max(axis=1, keepdims=True)
        e = np.exp(x - m)
        z = e.sum(axis=1, keepdims=True)
        p[b, :, :n] = e / z
        lse[b] = (m + np.log(z))[:, 0]
    return p, lse


def weighted_values(w, pool, scales, bits, page_table, ctx_lens, page_size):
    """(sum_j w[b, h, j] v[b, j, h // (Hq / H)], the same of magnitudes): [batch, Hq, d] each, over
    the first ctx_lens[b] cached values."""
    batch, hq = w.shape[:2]
    rep = hq // pool.shape[1]
    d = scales.shape[-1] * GROUP
    o, mag = np.zeros((batch, hq, d)), np.zeros((batch, hq, d))
    for b in range(batch):
        n = int(ctx_lens[b])
        v, _ = sequence(pool, scales, bits, page_table, b, n, page_size)
        v = np.repeat(v, rep, axis=1)
        o[b] = np.einsum("hn,nhd->hd", w[b, :, :n], v)
        mag[b] = np.einsum("hn,nhd->hd", np.abs(w[b, :, :n]), np.abs(v))
    return o, mag
