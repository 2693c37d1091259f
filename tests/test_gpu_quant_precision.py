"""Precision of the quantised paged cache and of the decode operators over it where magnitudes differ widely:
scales of every bf16 magnitude, groups of very different size in one head, a token that takes almost all
of the weight. Against the float64 oracle (oracle/quant_cache.py).
"""

import math

import numpy as np
import pytest
import torch

from oracle import quant_cache as Q
from synth.workloads import bf16_bits, bf16_bits_to_f64

from _gpu_common import bf16
from test_gpu_quant_cache import cache, check_mapped, i32, mapped_inputs, score_tol, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C():
    from cross_model_attention_map_b200 import iamap
    return iamap


def pool_with(rng, rows, table, total, page, bits):
    """Codes and scales of the float64 rows [n, H, d] of each sequence, garbage elsewhere."""
    H, d = rows[0].shape[1:]
    pool = rng.integers(0, 256, size=(total, H, page, d * bits // 8), dtype=np.uint8)
    scales = rng.choice(np.array([np.nan, np.inf, 6e4], dtype=np.float16), size=(total, H, page, d // 32))
    for b, x in enumerate(rows):
        pos = np.arange(len(x))
        c, s = Q.quantise(x, bits)
        pool[table[b, pos // page], :, pos % page] = Q.pack(c, bits)
        scales[table[b, pos // page], :, pos % page] = s
    return pool, scales


# ------------------------------------------------------------------------------------------------
# Scales
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [4, 8])
def test_scales_of_every_magnitude(C, bits):
    """A group for each of the 32640 finite bf16 magnitudes: scale and codes exact, the quotients that lie
    halfway between two subnormal fp16 numbers among them (91, 175 and 203 times 2^-25 in 4 bits)."""
    rng = np.random.default_rng(3)
    m = bf16_bits_to_f64(np.arange(0x7f80, dtype=np.uint16))
    x = m[:, None] * rng.uniform(-1, 1, size=(len(m), 32))
    x = bf16_bits_to_f64(bf16_bits(x.astype(np.float32)))
    x[np.arange(len(m)), rng.integers(0, 32, size=len(m))] = m
    x = x.reshape(-1, 1, 64)
    n, page = len(x), 16
    table = np.arange(-(-n // page), dtype=np.int32)[None]
    ck = cache(np.zeros((table.size, 1, page, 64 * bits // 8), dtype=np.uint8),
               np.zeros((table.size, 1, page, 2), dtype=np.float16), bits)
    ck.write(bf16(bf16_bits(x.astype(np.float32))), i32([0, n]), i32([0]), i32(table))
    assert C.iamap_device_status() == 0
    c, s = Q.quantise(x, bits)
    got = ck.scales.cpu().numpy().reshape(-1, 2)[:n]
    bad = np.flatnonzero((got != s[:, 0]).ravel())
    assert bad.size == 0, [(float(m[i] * 2.0 ** 25), float(got.ravel()[i]), float(s.ravel()[i])) for i in bad[:8]]
    np.testing.assert_array_equal(Q.unpack(ck.codes.cpu().numpy().reshape(-1, 64 * bits // 8)[:n], bits), c[:, 0])


# ------------------------------------------------------------------------------------------------
# Mapped product: the bound of fp32 sums, element by element
# ------------------------------------------------------------------------------------------------

def run_mapped(p, W, pool, scales, bits, table, lens, H_kv, d):
    from cross_model_attention_map_b200.runner import QuantDecodeStep
    st = QuantDecodeStep(len(lens), p.shape[1], W.shape[0], d, p.shape[2], H_kv=H_kv)
    return st.run(torch.from_numpy(p).cuda(), torch.from_numpy(W).cuda(), cache(pool, scales, bits),
                  i32(table), i32(lens)).cpu().numpy()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H,H_kv,d", [(3, 3, 128), (6, 2, 64), (16, 2, 128)])
@pytest.mark.parametrize("outlier,small", [(64.0, 1e-3), (3000.0, 1e-2), (6e4, 1e-2), (4e5, 1e-3)])
@pytest.mark.parametrize("where", ["all", "one"])
def test_mapped_groups_of_different_size(C, bits, H, H_kv, d, outlier, small, where):
    """One group of 32 elements is large, in every token or in one of them; the others, which share
    nothing with it, keep the precision that they have alone."""
    rng = np.random.default_rng(81)
    lens, page = [600, 70], 16
    table, total = table_of(rng, lens, page)
    rows = []
    for n in lens:
        x = rng.standard_normal((n, H_kv, d))
        x[..., 32:64] *= small
        x[..., 96:] *= 10 * small
        at = slice(None) if where == "all" else slice(n // 2, n // 2 + 1)
        x[at, :, :32] *= outlier
        rows.append(x)
    pool, scales = pool_with(rng, rows, table, total, page, bits)
    p, W = mapped_inputs(rng, lens, 5, H, max(lens))
    got = run_mapped(p, W, pool, scales, bits, table, lens, H_kv, d)
    assert C.iamap_device_status() == 0
    check_mapped(got, p, W, pool, scales, bits, table, lens, page)


def heavy(rng, lens, S, rest):
    """Rows of probabilities whose token 0 has all but `rest` of the mass."""
    p, _ = mapped_inputs(rng, lens, S, 1, max(lens))
    p = p.astype(np.float64)
    p[:, :, 0] = 0
    p *= rest / np.maximum(p.sum(-1, keepdims=True), 1e-30)
    p[:, :, 0] = 1 - rest
    return p.astype(np.float32)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H,H_kv,d", [(3, 3, 128), (6, 2, 64), (16, 2, 128)])
@pytest.mark.parametrize("rest", [1e-3, 1e-5, 1e-7])
def test_mapped_beside_a_heavy_token(C, bits, H, H_kv, d, rest):
    """A first token that takes almost all of the weight and whose values are zero: what the others add up to
    keeps its precision."""
    rng = np.random.default_rng(82)
    lens, page = [2000, 40], 16
    table, total = table_of(rng, lens, page)
    rows = [rng.standard_normal((n, H_kv, d)) for n in lens]
    for x in rows:
        x[0] = 0
    pool, scales = pool_with(rng, rows, table, total, page, bits)
    p, W = heavy(rng, lens, 5, rest), rng.standard_normal((H, 5)).astype(np.float32)
    got = run_mapped(p, W, pool, scales, bits, table, lens, H_kv, d)
    assert C.iamap_device_status() == 0
    check_mapped(got, p, W, pool, scales, bits, table, lens, page)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H,H_kv,d", [(3, 3, 128), (6, 2, 64), (16, 2, 128)])
@pytest.mark.parametrize("outlier,small", [(1.0, 1e-4), (6e4, 1e-3)])
def test_mapped_small_groups_beside_a_heavy_token(C, bits, H, H_kv, d, outlier, small):
    """Both at once: a token with almost all of the weight and no values, and small groups beside a large one."""
    rng = np.random.default_rng(83)
    lens, page = [1100, 40], 16
    table, total = table_of(rng, lens, page)
    rows = [rng.standard_normal((n, H_kv, d)) for n in lens]
    for x in rows:
        x[..., 32:] *= small
        x[..., :32] *= outlier
        x[0] = 0
    pool, scales = pool_with(rng, rows, table, total, page, bits)
    p, W = heavy(rng, lens, 5, 1e-5), rng.standard_normal((H, 5)).astype(np.float32)
    got = run_mapped(p, W, pool, scales, bits, table, lens, H_kv, d)
    assert C.iamap_device_status() == 0
    check_mapped(got, p, W, pool, scales, bits, table, lens, page)


# ------------------------------------------------------------------------------------------------
# Attention
# ------------------------------------------------------------------------------------------------

def check_weights(got, q, k, v, kb, vb, table, lens, page, off=0.0):
    """The error of attention's output, group by group. The probability p' = 2^(x - ref) and the product
    p' s / 2^E are rounded to fp16: by at most 2^-11 of themselves each (3 counted, for the exponential and the
    sums), or by 2^-25 where they are subnormal. The largest p' of 32 tokens lies between 2^2 and 2^14, and at
    2^10 or above in those that hold a sequence's largest score, so that 2^ref is at most 2^-2 of the 32 tokens'
    largest probability, or 2^-10. 2^E is 1 where a group's largest scale S is in [2^-8, 2), and otherwise at
    most 2 S, or 2^-15 (fp16 has no larger power of two than 2^15 to bring a scale up with). For S of 2 and
    more s / 2^E <= 2 may become subnormal and is rounded by 2^-25, which is 2^-24 S in each value at most."""
    p, _ = Q.softmax_rows(q, *k, kb, table, lens, page, max(lens))
    ref, mag = Q.weighted_values(p, *v, vb, table, lens, page)
    st = (score_tol(q, *k, kb, table, lens, page) + off)[:, None, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2 * st + 3 * 2.0 ** -11) * mag
    rep, qv = q.shape[1] // k[0].shape[1], Q.LEVELS[vb]
    for b, n in enumerate(lens):
        pos = np.arange(n)
        s = v[1][table[b, pos // page], :, pos % page].astype(np.float64)
        top = np.repeat(np.repeat(s.max(0), rep, axis=0), 32, axis=-1)
        unit = np.where((top >= 2.0 ** -8) & (top < 2), 1.0, np.maximum(2 * top, 2.0 ** -15))
        tol[b] += np.where(top >= 2, 2.0 ** -24 * top * qv, 0.0)
        for j in range(0, n, 32):
            largest = p[b, :, j:j + 32].max(-1)
            ulp = np.where(largest == p[b, :, :n].max(-1), 2.0 ** -10, 2.0 ** -2) * largest
            tol[b] += min(32, n - j) * 2.0 ** -25 * qv * ulp[:, None] * (top + unit)
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


def run_attention(qb, k, v, kb, vb, table, lens):
    from cross_model_attention_map_b200.runner import QuantAttention
    a = QuantAttention(len(lens), qb.shape[1], qb.shape[2], max(lens), H_kv=k[0].shape[1])
    return a.run(bf16(qb), cache(*k, kb), cache(*v, vb), i32(table), i32(lens)).float().cpu().numpy()


@pytest.mark.parametrize("vb", [4, 8])
@pytest.mark.parametrize("H,H_kv,d", [(4, 4, 128), (8, 1, 128), (6, 2, 64)])
@pytest.mark.parametrize("outlier,small", [(1.0, 1e-6), (300.0, 1e-5), (6e4, 1e-4), (4e5, 1e-5)])
@pytest.mark.parametrize("where", ["all", "one"])
def test_attention_groups_of_different_size(C, vb, H, H_kv, d, outlier, small, where):
    """One group large, in every token or in one, and the others small and the same in every token, so that
    roundings do not cancel."""
    rng = np.random.default_rng(91)
    lens, page = [700, 45], 16
    table, total = table_of(rng, lens, page)
    one = np.abs(rng.standard_normal((1, H_kv, d)))
    ks, vs = [], []
    for n in lens:
        ks.append(np.repeat(rng.standard_normal((1, H_kv, d)), n, axis=0))
        x = np.repeat(one, n, axis=0)
        x[..., 32:] *= small
        x[slice(None) if where == "all" else slice(n - 1, n), :, :32] *= outlier
        vs.append(x)
    k = pool_with(rng, ks, table, total, page, 8)
    v = pool_with(rng, vs, table, total, page, vb)
    qb = bf16_bits(rng.standard_normal((2, H, d)).astype(np.float32))
    got = run_attention(qb, k, v, 8, vb, table, lens)
    assert C.iamap_device_status() == 0
    check_weights(got, bf16_bits_to_f64(qb), k, v, 8, vb, table, lens, page)


@pytest.mark.parametrize("vb,size", [(4, 1.0), (8, 1.0), (8, 0.1)])
@pytest.mark.parametrize("H,H_kv,d", [(4, 4, 128), (8, 1, 128), (6, 2, 64)])
@pytest.mark.parametrize("rest", [1e-3, 1e-4, 1e-6, 1e-12])
@pytest.mark.parametrize("at", [0, 130])
def test_attention_beside_a_heavy_token(C, vb, size, H, H_kv, d, rest, at):
    """A token that takes all but `rest` of the mass and whose values are zero. The others have the same
    probability and nearly the same values, so that roundings do not cancel."""
    rng = np.random.default_rng(92)
    lens, page, kb = [2048, 300], 16, 8
    table, total = table_of(rng, lens, page)
    dirs = rng.choice([-1.0, 1.0], size=(H_kv, d))             # |dir|^2 = d: a key t dir scores t sqrt(d) x
    qb = bf16_bits(np.repeat(dirs, H // H_kv, axis=0)[None].repeat(2, 0).astype(np.float32))
    ks, vs = [], []
    for n in lens:
        key = np.zeros((n, H_kv, d))
        key[at] = dirs * math.log((n - 1) / rest) / math.sqrt(d)
        ks.append(key)
        x = np.abs(rng.standard_normal((1, H_kv, d))) * size * rng.uniform(0.9, 1.1, size=(n, 1, 1))
        x[at] = 0
        vs.append(x)
    k = pool_with(rng, ks, table, total, page, kb)
    v = pool_with(rng, vs, table, total, page, vb)
    got = run_attention(qb, k, v, kb, vb, table, lens)
    assert C.iamap_device_status() == 0
    check_weights(got, bf16_bits_to_f64(qb), k, v, kb, vb, table, lens, page)


# ------------------------------------------------------------------------------------------------
# Queries
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_different_size(C, bits, d):
    """A query's first 32 elements are 2^30 times the others and meet keys of zeros; the others make up the
    scores. The query is held in fp16 with its largest element q_max in [2^14, 2^15): fp16's smallest step there
    is 2^-24, so an element is off by at most 2^-25 / 2^14 = 2^-39 of q_max (an element above 2^-31 q_max, that is
    2^-17, ends its 8 bits at 2^-24 and is exact), and a score by 2^-39 q_max sum |k| / sqrt(d). To first order a row is
    off by twice that, relative, and attention's output by twice that times sum p |v|."""
    from cross_model_attention_map_b200.runner import QuantSenderRows
    rng = np.random.default_rng(95)
    lens, H, H_k, page = [300, 33], 6, 2, 16
    table, total = table_of(rng, lens, page)
    ks = [rng.standard_normal((n, H_k, d)) for n in lens]
    for x in ks:
        x[..., :32] = 0
    k = pool_with(rng, ks, table, total, page, bits)
    q = rng.standard_normal((2, H, d))
    q[..., :32] = 2.0 ** 30 * rng.uniform(1, 2, size=(2, H, 32))
    qb = bf16_bits(q.astype(np.float32))
    got = QuantSenderRows(2, H, d, max(lens), H_k=H_k).run(bf16(qb), cache(*k, bits), i32(table), i32(lens))
    assert C.iamap_device_status() == 0
    q = bf16_bits_to_f64(qb)
    off = np.array([2.0 ** -39 * np.abs(q[b]).max() * np.abs(Q.sequence(*k, bits, table, b, n, page)[0]).sum(-1).max()
                    / math.sqrt(d) for b, n in enumerate(lens)])
    assert off.max() < 0.05                                   # first order will do
    p, _ = Q.softmax_rows(q, *k, bits, table, lens, page, max(lens))
    tol = 2 * (score_tol(q, *k, bits, table, lens, page) + off) + 2.0 ** -20
    assert (np.abs(got.cpu().numpy() - p) <= tol[:, None, None] * p).all()
    v = pool_with(rng, ks, table, total, page, bits)
    out = run_attention(qb, k, v, bits, bits, table, lens)
    check_weights(out, q, k, v, bits, bits, table, lens, page, off)


@pytest.mark.parametrize("n,page", [(300, 16), (5000, 16), (600, 8)])
def test_rows_of_equal_large_scores(C, n, page):
    """n equal keys whose score is large: every probability is 1 / n to fp32's rounding (one exponential of 0, a sum
    of n ones, a quotient and a product: 2^-22), however large the score."""
    from cross_model_attention_map_b200.runner import QuantSenderRows
    rng = np.random.default_rng(96)
    table, total = table_of(rng, [n], page)
    key = rng.choice([-1.0, 1.0], size=(1, 1, 64))
    k = pool_with(rng, [np.repeat(7 * key, n, axis=0)], table, total, page, 4)
    qb = bf16_bits((key * np.array([[[60.0], [61.0], [-59.0]]])).reshape(1, 3, 64).astype(np.float32))
    got = QuantSenderRows(1, 3, 64, n, H_k=1).run(bf16(qb), cache(*k, 4), i32(table), i32([n])).cpu().numpy()
    assert C.iamap_device_status() == 0
    assert (np.abs(got * np.float64(n) - 1) <= 2.0 ** -22).all(), np.abs(got * n - 1).max()
