"""GPU parity of the quantised paged cache and of the decode operators over it, against the float64
oracle (oracle/quant_cache.py), through the C ABI.

Tolerances, from the arithmetic (u = 2^-24, an fp32 rounding; u11 = 2^-11, an fp16 one; u8 = 2^-8, a
bf16 one):
  codes, scales, read-back   exact: codes are decided by exact comparisons, c * s has 8 + 11 bits and
                             is rounded once
  scores                     products of q and the codes are exact in fp32, their sums err by at most
                             (d + 8) 2u sum |q k| / sqrt(d) (2u an addition: a matrix instruction may
                             truncate), the change of base and the exponent's rounding by 4u |x|
  rows                       relative: the scores' error twice (the row and its log-sum-exp), + 2^-20
                             for two approximate exponentials and the logarithm
  mapped                     (ctx / 8 + H_s + 32) 2u sum |w| |v|: the weights' own sum, their two fp16
                             parts (2^-22), and the accumulation in steps of 16 tokens over any split
  attention                  half a bf16 step of the result, + sum p |v| times twice the scores' error
                             and 3 u11 (the probability, the scale product and its use), + the absolute
                             step of fp16. A probability is held as p' = 2^(x - ref) and used as p' s, each
                             rounded to at worst 2^-25 where it is subnormal, so a token's term p' s c is
                             off by at most 2^-25 (s + 1) Q, in units of 2^(ref - lse). ref is 8 or more
                             below the largest score, and higher only where a p' s would pass 2^15: it is
                             then raised until the largest lies between 2^13 and 2^14, so that
                             2^(ref - lse) <= max(2^-8, 2^-13 s) and n tokens give
                             n 2^-25 (s + 1) Q max(2^-8, 2^-13 s), s the largest scale
"""

import math

import numpy as np
import pytest
import torch

from oracle import quant_cache as Q
from synth.workloads import bf16_bits, bf16_bits_to_f64

from _gpu_common import bf16

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def C():
    from cross_model_attention_map_b200 import iamap
    return iamap


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def table_of(rng, lens, page, spare=2):
    """A shuffled page table and the number of pages; entries past a sequence's pages are bad indices,
    which a kernel must not look at."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    perm = rng.permutation(total)
    table = np.full((len(lens), max(1, max(need))), 1 << 30, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, total


def pool_of(rng, lens, table, total, page, H, d, bits, std=1.0):
    """Codes and scales with rows for every token and garbage elsewhere: any code bytes, scales of
    infinity and NaN, as memory that nothing was written to may hold."""
    pool = rng.integers(0, 256, size=(total, H, page, d * bits // 8), dtype=np.uint8)
    scales = rng.choice(np.array([np.nan, np.inf, -np.inf, 6e4], dtype=np.float16),
                        size=(total, H, page, d // 32))
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pos = np.arange(n)
        x = rng.standard_normal((n, H, d)) * std * np.exp(0.5 * rng.standard_normal((1, H, d)))
        c, s = Q.quantise(x, bits)
        pool[table[b, pos // page], :, pos % page] = Q.pack(c, bits)
        scales[table[b, pos // page], :, pos % page] = s
    return pool, scales


def cache(pool, scales, bits):
    from cross_model_attention_map_b200.runner import QuantCache
    return QuantCache.over(torch.from_numpy(pool).cuda(), torch.from_numpy(scales).cuda(), bits)


def score_tol(q, pool, scales, bits, table, lens, page):
    """Largest error of a score, natural units, per sequence."""
    rep = q.shape[1] // pool.shape[1]
    d = q.shape[2]
    out = []
    for b, n in enumerate(lens):
        if n == 0:
            out.append(0.0)
            continue
        k, _ = Q.sequence(pool, scales, bits, table, b, int(n), page)
        k = np.abs(np.repeat(k, rep, axis=1))
        mag = np.einsum("hd,nhd->hn", np.abs(q[b]), k).max() / math.sqrt(d)
        out.append(float(mag) * ((d + 8) * 2 * U + 4 * U))
    return np.array(out)


# ------------------------------------------------------------------------------------------------
# Write and read
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,H", [(1, 1), (7, 3), (16, 14), (24, 5), (64, 2)])
def test_write_then_read(C, bits, d, page, H):
    """Ragged appends (an empty one among them) after cached prefixes, from a strided projection slice
    with padded rows: codes and scales of the written slots exact, all other slots as they were, and
    the read-back exact with the rows behind the last sequence as they were."""
    rng = np.random.default_rng(100 + bits + d + page)
    ends, new = [37, 20, 5, 1, 130], [37, 1, 0, 1, 64]
    starts = [e - k for e, k in zip(ends, new)]
    table, total = table_of(rng, ends, page)
    pool, scales = pool_of(rng, ends, table, total, page, H, d, bits)
    n, pad = sum(new), 9
    x = (rng.standard_normal((n + pad, 3, H, d)) * np.exp(rng.uniform(-3, 3, (n + pad, 3, H, 1))))
    x = x.astype(np.float32)
    x[0, 1, 0, :32] = 0.0                                    # an empty group
    x[1, 1, 0, 3] = np.inf
    x[2, 1, 0, 40] = np.nan
    x[3, 1, 0, :32] = 1e-38 * np.arange(32)                  # under the scale's range
    x[4, 1, 0, :32] = 3e5 * np.arange(-16, 16)               # above it
    x[5, 1, 0, :32] = np.arange(32) * (0.5 if bits == 4 else 0.25) - 3.5   # ties between two levels
    x[6, 1, 0, :32] = 1e-5 * np.arange(-16, 16)              # subnormal fp16 scales
    xb = bf16_bits(x)
    dev = bf16(xb)
    ck = cache(pool, scales, bits)
    cu = np.concatenate([[0], np.cumsum(new)])
    ck.write(dev.view(n + pad, -1)[:, H * d:2 * H * d], i32(cu), i32(starts), i32(table))
    assert C.iamap_device_status() == 0
    c, s = Q.quantise(bf16_bits_to_f64(xb)[:, 1], bits)
    rows, pg, slot, bad = Q.slots(cu, starts, table, page, total, n + pad)
    assert bad == 0 and len(rows) == n
    pool[pg, :, slot] = Q.pack(c, bits)[rows]
    scales[pg, :, slot] = s[rows]
    np.testing.assert_array_equal(ck.codes.cpu().numpy(), pool)
    got = ck.scales.cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(scales))
    np.testing.assert_array_equal(np.where(np.isnan(got), 0, got), np.where(np.isnan(scales), 0, scales))
    # ranges: everything, a tail and nothing
    lo = [0, 3, 0, 0, 129]
    take = [37, 17, 5, 0, 1]
    cu_r = np.concatenate([[0], np.cumsum(take)])
    out = torch.full((sum(take) + 4, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ck.read(i32(cu_r), i32(lo), i32(table), out)
    assert C.iamap_device_status() == 0
    rows, pg, slot, _ = Q.slots(cu_r, lo, table, page, total, len(out))
    with np.errstate(all="ignore"):
        ref = Q.values(pool[pg, :, slot], scales[pg, :, slot], bits).astype(np.float32)
    ref = torch.from_numpy(ref).to(torch.bfloat16)
    assert torch.equal(out[:len(ref)].cpu().nan_to_num(nan=12345.0), ref.nan_to_num(nan=12345.0))
    assert bool((out[len(ref):] == 7.0).all())


def test_one_head_and_no_rows(C):
    """A single head's rows may carry any stride in the head's place; an empty batch does nothing."""
    from cross_model_attention_map_b200.runner import QuantCache
    ck = QuantCache(2, 16, 1, 64, 8)
    x = torch.randn(1, 20, 64, device="cuda").bfloat16().transpose(0, 1)
    assert x.stride()[1] == 20 * 64
    table = i32([[1, 0]])
    ck.write(x, i32([0, 20]), i32([0]), table)
    a = ck.read(i32([0, 20]), i32([0]), table, torch.empty(20, 1, 64, dtype=torch.bfloat16, device="cuda"))
    # half a step of the scale (at most max |x| / 127 and an fp16 rounding), then a bf16 rounding
    assert float((a.float() - x.float()).abs().max()) <= float(x.float().abs().max()) * (0.501 / 127 + 2.0 ** -8)
    before = ck.codes.clone()
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    ck.write(none, i32([0, 0]), i32([0]), table)
    assert ck.read(i32([0, 0]), i32([0]), table, none) is none
    torch.cuda.synchronize()
    assert torch.equal(ck.codes, before) and C.iamap_device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
def test_every_bf16_quotient_near_a_border(C, bits):
    """Codes are decided by exact comparisons: rows whose elements lie at, and one bf16 step beside,
    the borders (k + 1/2) s of every level, for many scales."""
    rng = np.random.default_rng(7)
    q = Q.LEVELS[bits]
    rows = []
    for _ in range(512):
        m = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-8, 8))
        m = bf16_bits_to_f64(bf16_bits(np.array([m])))[0]
        s = float(np.float16(m / q))
        k = rng.integers(0, q, size=31)
        b = bf16_bits(((k + 0.5) * s).astype(np.float32)).astype(np.int64) + rng.integers(-1, 2, size=31)
        x = bf16_bits_to_f64(b.astype(np.uint16)) * rng.choice([-1, 1], size=31)
        rows.append(np.concatenate([[m], np.clip(x, -m, m)]))
    x = np.stack(rows).reshape(-1, 1, 64)
    ck_pool = np.zeros((1, 1, len(x), 64 * bits // 8), dtype=np.uint8)
    ck = cache(ck_pool, np.zeros((1, 1, len(x), 2), dtype=np.float16), bits)
    ck.write(bf16(bf16_bits(x.astype(np.float32))), i32([0, len(x)]), i32([0]), i32([[0]]))
    c, s = Q.quantise(x, bits)
    np.testing.assert_array_equal(ck.scales.cpu().numpy()[0, 0], s[:, 0])
    np.testing.assert_array_equal(Q.unpack(ck.codes.cpu().numpy()[0, 0], bits), c[:, 0])


def test_bad_places_are_reported_and_skipped(C):
    """Tokens outside the page table, bad page indices and negative starts: not stored, flagged, and
    nothing else changes; such tokens read as 0."""
    rng = np.random.default_rng(8)
    page, H, d, bits = 4, 2, 64, 4
    table = np.array([[0, 7, 2], [3, -1, 1]], dtype=np.int32)     # 7 and -1: outside 5 pages
    pool, scales = pool_of(rng, [], table, 5, page, H, d, bits)
    x = bf16_bits(rng.standard_normal((26, H, d)).astype(np.float32))
    for starts in ([0, 0], [-3, 5]):
        ck = cache(pool, scales, bits)
        cu = [0, 14, 26]                                            # 14 tokens, 12 places
        ck.write(bf16(x), i32(cu), i32(starts), i32(table))
        assert C.iamap_device_status() & C.IAMAP_DEV_BAD_INDEX
        rows, pg, slot, bad = Q.slots(cu, starts, table, page, 5, 26)
        assert bad > 0
        c, s = Q.quantise(bf16_bits_to_f64(x), bits)
        want_c, want_s = pool.copy(), scales.copy()
        want_c[pg, :, slot] = Q.pack(c, bits)[rows]
        want_s[pg, :, slot] = s[rows]
        np.testing.assert_array_equal(ck.codes.cpu().numpy(), want_c)
        np.testing.assert_array_equal(ck.scales.cpu().numpy().view(np.uint16), want_s.view(np.uint16))
        out = torch.full((26, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
        ck.read(i32(cu), i32(starts), i32(table), out)
        assert C.iamap_device_status() & C.IAMAP_DEV_BAD_INDEX
        ref = np.zeros((26, H, d), dtype=np.float32)
        ref[rows] = Q.values(want_c[pg, :, slot], want_s[pg, :, slot], bits)
        assert torch.equal(out.cpu(), torch.from_numpy(ref).to(torch.bfloat16))


def test_pool_beyond_32_bit_offsets(C):
    """A pool of more than 4 GiB of codes, its last pages in use."""
    page, H, d, bits = 16, 64, 128, 8
    total = (4 << 30) // (page * H * d) + 2048
    codes = torch.empty(total, H, page, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(total, H, page, d // 32, dtype=torch.float16, device="cuda")
    from cross_model_attention_map_b200.runner import (QuantAttention, QuantCache, QuantDecodeStep,
                                                       QuantSenderRows)
    ck = QuantCache.over(codes, scales, bits)
    table = np.array([[total - 1, 5, total - 2]], dtype=np.int32)
    rng = np.random.default_rng(9)
    n = 40
    x = bf16_bits(rng.standard_normal((n, H, d)).astype(np.float32))
    ck.write(bf16(x), i32([0, n]), i32([0]), i32(table))
    out = torch.empty(n, H, d, dtype=torch.bfloat16, device="cuda")
    ck.read(i32([0, n]), i32([0]), i32(table), out)
    c, s = Q.quantise(bf16_bits_to_f64(x), bits)
    v = c * np.repeat(s.astype(np.float64), 32, axis=-1)
    assert torch.equal(out.cpu(), torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16))
    q = bf16_bits(rng.standard_normal((1, H, d)).astype(np.float32))
    rows = QuantSenderRows(1, H, d, n).run(bf16(q), ck, i32(table), i32([n]))
    xs = np.einsum("hd,nhd->hn", bf16_bits_to_f64(q)[0], v) / math.sqrt(d)
    p = np.exp(xs - xs.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    np.testing.assert_allclose(rows.cpu().numpy()[0], p, rtol=1e-4)
    o = QuantDecodeStep(1, H, H, d, n).run(rows, torch.eye(H, device="cuda"), ck, i32(table), i32([n]))
    ref = np.einsum("hn,nhd->hd", p, v)
    np.testing.assert_allclose(o.cpu().numpy()[0], ref, atol=1e-4)
    at = QuantAttention(1, H, d, n).run(bf16(q), ck, ck, i32(table), i32([n]))
    np.testing.assert_allclose(at.float().cpu().numpy()[0], ref, atol=2e-2)
    assert C.iamap_device_status() == 0


# ------------------------------------------------------------------------------------------------
# Rows
# ------------------------------------------------------------------------------------------------

def check_rows(got, q, pool, scales, bits, table, lens, page):
    p, _ = Q.softmax_rows(q, pool, scales, bits, table, lens, page, got.shape[2])
    tol = 2 * score_tol(q, pool, scales, bits, table, lens, page) + 2.0 ** -20
    err = np.abs(got - p)
    assert (err <= tol[:, None, None] * p + 1e-37).all(), (err / np.maximum(p, 1e-30)).max()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens,H_s,H_k,d,page,extra", [
    ([1], 1, 1, 64, 16, 0),
    ([0, 1, 15, 16, 17], 3, 3, 64, 16, 5),
    ([600, 0, 17, 513], 6, 2, 128, 16, 3),
    ([64, 65, 63], 14, 2, 64, 8, 0),
    ([100, 250], 16, 1, 128, 7, 1),
    ([1000, 31], 12, 1, 64, 1, 0),
    ([4100, 2049], 14, 14, 64, 32, 0),
    ([9001], 9, 1, 128, 24, 0),
    ([33000, 5], 7, 1, 64, 64, 11),
    ([500, 0, 37], 3, 3, 64, 16, 1700),
    ([500, 0, 37], 3, 3, 64, 16, 3700),
    ([4096, 4097, 0], 2, 1, 64, 16, 0),
])
def test_rows(C, bits, lens, H_s, H_k, d, page, extra):
    from cross_model_attention_map_b200.runner import QuantSenderRows
    rng = np.random.default_rng(sum(lens) + H_s + bits)
    table, total = table_of(rng, lens, page)
    pool, scales = pool_of(rng, lens, table, total, page, H_k, d, bits)
    qb = bf16_bits(rng.standard_normal((len(lens), H_s, d)).astype(np.float32))
    r = QuantSenderRows(len(lens), H_s, d, max(lens), H_k=H_k, ctx_stride=max(lens) + extra)
    r.rows.fill_(float("nan"))
    got = r.run(bf16(qb), cache(pool, scales, bits), i32(table), i32(lens)).cpu().numpy()
    assert C.iamap_device_status() == 0
    check_rows(got, bf16_bits_to_f64(qb), pool, scales, bits, table, lens, page)
    for b, n in enumerate(lens):
        assert not got[b, :, n:].any()


@pytest.mark.parametrize("size", [1e-30, 1e-3, 300.0, 1e30])
def test_rows_of_large_and_small_queries(C, size):
    """Queries of any magnitude: near-uniform rows, and rows whose maximum takes everything."""
    from cross_model_attention_map_b200.runner import QuantSenderRows
    rng = np.random.default_rng(21)
    lens, page, d, bits = [777, 40], 16, 64, 4
    table, total = table_of(rng, lens, page)
    pool, scales = pool_of(rng, lens, table, total, page, 2, d, bits)
    qb = bf16_bits((rng.standard_normal((2, 4, d)) * size).astype(np.float32))
    got = QuantSenderRows(2, 4, d, 777, H_k=2).run(bf16(qb), cache(pool, scales, bits), i32(table),
                                                   i32(lens)).cpu().numpy()
    q = bf16_bits_to_f64(qb)
    if size <= 300:
        check_rows(got, q, pool, scales, bits, table, lens, page)
    else:
        p, _ = Q.softmax_rows(q, pool, scales, bits, table, lens, page, 777)
        np.testing.assert_array_equal(got.argmax(-1), p.argmax(-1))
        np.testing.assert_array_equal(got.max(-1), 1.0)


def test_lengths_are_read_on_the_device_and_clamped(C):
    from cross_model_attention_map_b200.runner import QuantAttention, QuantDecodeStep, QuantSenderRows
    rng = np.random.default_rng(22)
    lens, page, d, bits = [50, 50, 50], 16, 64, 8
    table, total = table_of(rng, lens, page)
    pool, scales = pool_of(rng, lens, table, total, page, 2, d, bits)
    ck = cache(pool, scales, bits)
    qb = bf16_bits(rng.standard_normal((3, 4, d)).astype(np.float32))
    r = QuantSenderRows(3, 4, d, 50, H_k=2)
    got = r.run(bf16(qb), ck, i32(table), i32([60, -7, 50])).cpu().numpy()
    assert C.iamap_device_status() & C.IAMAP_DEV_BAD_INDEX
    check_rows(got, bf16_bits_to_f64(qb), pool, scales, bits, table, [50, 0, 50], page)
    W = torch.eye(4, device="cuda")
    o = QuantDecodeStep(3, 4, 4, d, 50, H_kv=2).run(r.rows, W, ck, i32(table), i32([60, -7, 50]))
    assert C.iamap_device_status() & C.IAMAP_DEV_BAD_INDEX and not o[1].any()
    a, lse = QuantAttention(3, 4, d, 50, H_kv=2, want_lse=True).run(bf16(qb), ck, ck, i32(table),
                                                                    i32([60, -7, 50]))
    assert C.iamap_device_status() & C.IAMAP_DEV_BAD_INDEX
    assert not a[1].any() and bool((lse[1] == -math.inf).all()) and bool(torch.isfinite(lse[0]).all())


# ------------------------------------------------------------------------------------------------
# Mapped product
# ------------------------------------------------------------------------------------------------

def mapped_inputs(rng, lens, S, H, stride):
    p = rng.gamma(1.0, 1.0, size=(len(lens), S, stride))
    for b, n in enumerate(lens):
        p[b, :, n:] = 0
    p = (p / np.maximum(p.sum(-1, keepdims=True), 1e-30)).astype(np.float32)
    return p, rng.standard_normal((H, S)).astype(np.float32)


def check_mapped(got, p, W, pool, scales, bits, table, lens, page):
    w = np.einsum("rs,bsj->brj", W.astype(np.float64), np.nan_to_num(p.astype(np.float64)))
    a = np.einsum("rs,bsj->brj", np.abs(W).astype(np.float64), np.abs(np.nan_to_num(p.astype(np.float64))))
    ref, _ = Q.weighted_values(w, pool, scales, bits, table, lens, page)
    _, mag = Q.weighted_values(a, pool, scales, bits, table, lens, page)
    n = np.array(lens)[:, None, None]
    tol = (n / 8 + W.shape[1] + 32) * 2 * U * mag
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens,S,H,H_kv,d,page,extra", [
    ([1], 1, 1, 1, 64, 16, 0),
    ([0, 1, 15, 16, 17], 3, 4, 4, 64, 16, 2),
    ([300, 1, 17, 0, 256], 6, 12, 12, 64, 16, 0),
    ([600, 130], 14, 8, 1, 128, 7, 1),
    ([129, 64], 5, 6, 3, 128, 1, 0),
    ([513, 1000], 32, 64, 8, 128, 24, 0),
    ([2100, 999, 3], 14, 64, 64, 128, 16, 0),
    ([5000, 77], 2, 34, 2, 64, 32, 0),
    ([700], 128, 128, 128, 64, 16, 0),
    ([90, 33], 1, 128, 2, 64, 64, 3),
    # more sequences than a warp has lanes, groups of 32 of them empty, more ranges than CTAs
    ([0] * 40 + [n * 97 % 1300 for n in range(50)] + [0] * 70 + [700, 0], 14, 64, 64, 64, 16, 0),
    ([3, 0, 513] * 14 + [1025], 17, 6, 2, 128, 16, 0),
])
def test_mapped(C, bits, lens, S, H, H_kv, d, page, extra):
    """Rows past a sequence's length hold NaN: they are not used."""
    from cross_model_attention_map_b200.runner import QuantDecodeStep
    rng = np.random.default_rng(sum(lens) + S + H + bits)
    table, total = table_of(rng, lens, page)
    pool, scales = pool_of(rng, lens, table, total, page, H_kv, d, bits)
    stride = max(lens) + extra
    p, W = mapped_inputs(rng, lens, S, H, stride)
    for b, n in enumerate(lens):
        p[b, :, n:] = np.nan
    st = QuantDecodeStep(len(lens), S, H, d, max(lens), H_kv=H_kv, ctx_stride=stride)
    st.out.fill_(float("nan"))
    got = st.run(torch.from_numpy(p).cuda(), torch.from_numpy(W).cuda(), cache(pool, scales, bits),
                 i32(table), i32(lens)).cpu().numpy()
    assert C.iamap_device_status() == 0
    check_mapped(got, p, W, pool, scales, bits, table, lens, page)


@pytest.mark.parametrize("wsize,vsize", [(1e-25, 1.0), (1e25, 1e3), (1.0, 1e-3), (3.0, 3e4), (0.0, 1.0)])
@pytest.mark.parametrize("H_kv", [4, 2])
def test_mapped_weights_of_any_size(C, wsize, vsize, H_kv):
    """Weights far from 1, growing by many orders of magnitude along the context, and all zero."""
    from cross_model_attention_map_b200.runner import QuantDecodeStep
    rng = np.random.default_rng(31)
    lens, S, H, d, page, bits = [400, 37], 2, 4, 64, 16, 4
    table, total = table_of(rng, lens, page)
    pool, scales = pool_of(rng, lens, table, total, page, H_kv, d, bits, std=vsize)
    p, W = mapped_inputs(rng, lens, S, H, 400)
    p *= (wsize * 10.0 ** rng.uniform(-12, 0, size=(1, 1, 400))).astype(np.float32)
    p[:, :, :64] *= np.float32(1e-6)
    got = QuantDecodeStep(2, S, H, d, 400, H_kv=H_kv).run(
        torch.from_numpy(p).cuda(), torch.from_numpy(W).cuda(), cache(pool, scales, bits), i32(table),
        i32(lens)).cpu().numpy()
    check_mapped(got, p, W, pool, scales, bits, table, lens, page)


def test_mapped_infinities_stay_in_their_head(C):
    """A weight of infinity or NaN inside the context reaches its own receiver head only; a NaN group of
    the cache reaches its own elements only."""
    from cross_model_attention_map_b200.runner import QuantDecodeStep
    rng = np.random.default_rng(32)
    lens, S, H, d, page, bits = [100], 4, 4, 64, 16, 4
    table, total = table_of(rng, lens, page)
    pool, scales = pool_of(rng, lens, table, total, page, H, d, bits)
    p, _ = mapped_inputs(rng, lens, S, H, 100)
    ck = cache(pool, scales, bits)
    eye = torch.eye(4, device="cuda")
    st = QuantDecodeStep(1, S, H, d, 100)
    clean = st.run(torch.from_numpy(p).cuda(), eye, ck, i32(table), i32(lens)).clone()
    ck.scales[int(table[0, 2]), 1, 3, 0] = float("nan")       # head 1, elements 0..31
    got = st.run(torch.from_numpy(p).cuda(), eye, ck, i32(table), i32(lens))
    assert bool(torch.isnan(got[0, 1, :32]).all()) and torch.equal(got[0, 1, 32:], clean[0, 1, 32:])
    assert torch.equal(got[0, [0, 2, 3]], clean[0, [0, 2, 3]])


def test_mapped_with_room_for_a_very_long_context(C):
    """max_ctx beyond 65535 ranges of 512 tokens, as a captured step that is to serve any length has it."""
    from cross_model_attention_map_b200.runner import QuantDecodeStep
    rng = np.random.default_rng(33)
    lens, page, d, bits, most = [700, 30], 64, 64, 4, 33_600_000
    table, total = table_of(rng, lens, page)
    pool, scales = pool_of(rng, lens, table, total, page, 1, d, bits)
    wide = torch.full((2, most // page), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = i32(table)
    p, W = mapped_inputs(rng, lens, 1, 1, 700)
    rows = torch.zeros(2, 1, most, device="cuda")
    rows[:, :, :700] = torch.from_numpy(p).cuda()
    got = QuantDecodeStep(2, 1, 1, d, most).run(rows, torch.from_numpy(W).cuda(), cache(pool, scales, bits), wide,
                                                i32(lens))
    assert C.iamap_device_status() == 0
    check_mapped(got.cpu().numpy(), p, W, pool, scales, bits, table, lens, page)


# ------------------------------------------------------------------------------------------------
# Attention
# ------------------------------------------------------------------------------------------------

def check_attention(got, lse, q, k, v, kb, vb, table, lens, page):
    p, ref_lse = Q.softmax_rows(q, *k, kb, table, lens, page, max(max(lens), 1))
    ref, mag = Q.weighted_values(p, *v, vb, table, lens, page)
    st = score_tol(q, *k, kb, table, lens, page)[:, None, None]
    tol = 2.0 ** -8 * np.abs(ref) + (2 * st + 3 * 2.0 ** -11) * mag
    for b, n in enumerate(lens):
        pos = np.arange(n)
        pg = table[b, pos // page]
        ok = (pg >= 0) & (pg < v[1].shape[0])
        s = v[1][pg[ok], :, pos[ok] % page].astype(np.float64).max(initial=0.0)
        tol[b] += n * 2.0 ** -25 * (s + 1) * Q.LEVELS[vb] * max(2.0 ** -8, 2.0 ** -13 * s)
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
    if lse is not None:
        fine = np.isfinite(ref_lse)
        np.testing.assert_array_equal(np.isfinite(lse), fine)
        assert (lse[~fine] == -np.inf).all()
        bound = st[:, :, 0] + 2.0 ** -20 + 4 * U * np.abs(np.where(fine, ref_lse, 0))
        assert (np.abs(np.where(fine, lse, 0) - np.where(fine, ref_lse, 0)) <= bound).all()


@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8), (8, 4), (4, 8)])
@pytest.mark.parametrize("lens,H,H_kv,d,page", [
    ([1], 1, 1, 64, 16),
    ([0, 1, 15, 16, 17], 3, 3, 64, 16),
    ([512, 1, 0, 201], 14, 2, 64, 16),
    ([600, 130], 8, 1, 128, 7),
    ([129, 64], 6, 3, 128, 1),
    ([513, 1000], 64, 8, 128, 24),
    ([2100, 999, 3], 16, 16, 128, 16),
    ([5000, 77], 34, 2, 64, 32),
    ([20000], 8, 1, 128, 64),
    ([9000, 12], 2, 1, 64, 32),
])
def test_attention(C, kb, vb, lens, H, H_kv, d, page):
    from cross_model_attention_map_b200.runner import QuantAttention
    rng = np.random.default_rng(sum(lens) + H + kb + 2 * vb)
    table, total = table_of(rng, lens, page)
    k = pool_of(rng, lens, table, total, page, H_kv, d, kb)
    v = pool_of(rng, lens, table, total, page, H_kv, d, vb)
    qb = bf16_bits(rng.standard_normal((len(lens), H, d)).astype(np.float32))
    a = QuantAttention(len(lens), H, d, max(lens), H_kv=H_kv, want_lse=True)
    a.out.fill_(float("nan"))
    a.lse.fill_(float("nan"))
    out, lse = a.run(bf16(qb), cache(*k, kb), cache(*v, vb), i32(table), i32(lens))
    assert C.iamap_device_status() == 0
    check_attention(out.float().cpu().numpy(), lse.cpu().numpy(), bf16_bits_to_f64(qb), k, v, kb, vb,
                    table, lens, page)
    plain = QuantAttention(len(lens), H, d, max(lens), H_kv=H_kv)
    assert torch.equal(plain.run(bf16(qb), cache(*k, kb), cache(*v, vb), i32(table), i32(lens)), out)


@pytest.mark.parametrize("size,vsize", [(20.0, 1.0), (1e-20, 1.0), (1.0, 1e-2), (1.0, 3e4), (4.0, 100.0)])
def test_attention_of_any_size(C, size, vsize):
    """Peaked and flat rows, large and small values; the running maximum moves throughout."""
    from cross_model_attention_map_b200.runner import QuantAttention
    rng = np.random.default_rng(41)
    lens, H, H_kv, d, page = [1500, 300], 4, 2, 64, 16
    table, total = table_of(rng, lens, page)
    k = pool_of(rng, lens, table, total, page, H_kv, d, 8)
    v = pool_of(rng, lens, table, total, page, H_kv, d, 4, std=vsize)
    qb = bf16_bits((size * rng.standard_normal((2, H, d))).astype(np.float32))
    out, lse = QuantAttention(2, H, d, 1500, H_kv=H_kv, want_lse=True).run(
        bf16(qb), cache(*k, 8), cache(*v, 4), i32(table), i32(lens))
    check_attention(out.float().cpu().numpy(), lse.cpu().numpy(), bf16_bits_to_f64(qb), k, v, 8, 4,
                    table, lens, page)


@pytest.mark.parametrize("page", [16, 8])
def test_bad_pages_are_absent_tokens(C, page):
    """A page index outside the pool: its tokens have probability and contribution 0, a sequence with no
    good page is an empty one, and the status says so."""
    from cross_model_attention_map_b200.runner import QuantAttention, QuantDecodeStep, QuantSenderRows
    rng = np.random.default_rng(51)
    lens, H, H_kv, d, bits = [300, 40, 20], 6, 2, 64, 8
    table, total = table_of(rng, lens, page)
    k = pool_of(rng, lens, table, total, page, H_kv, d, bits)
    v = pool_of(rng, lens, table, total, page, H_kv, d, bits)
    table[0, 3], table[0, 5], table[2, :] = total, -5, total + 100
    qb = bf16_bits(rng.standard_normal((3, H, d)).astype(np.float32))
    q = bf16_bits_to_f64(qb)
    got = QuantSenderRows(3, H, d, 300, H_k=H_kv).run(bf16(qb), cache(*k, bits), i32(table), i32(lens))
    assert C.iamap_device_status() & C.IAMAP_DEV_BAD_INDEX
    check_rows(got.cpu().numpy(), q, *k, bits, table, lens, page)
    assert not got[0, :, 3 * page:4 * page].any() and not got[2].any()
    p, W = mapped_inputs(rng, lens, 3, H, 300)
    o = QuantDecodeStep(3, 3, H, d, 300, H_kv=H_kv).run(
        torch.from_numpy(p).cuda(), torch.from_numpy(W).cuda(), cache(*v, bits), i32(table), i32(lens))
    assert C.iamap_device_status() & C.IAMAP_DEV_BAD_INDEX
    check_mapped(o.cpu().numpy(), p, W, *v, bits, table, lens, page)
    out, lse = QuantAttention(3, H, d, 300, H_kv=H_kv, want_lse=True).run(
        bf16(qb), cache(*k, bits), cache(*v, bits), i32(table), i32(lens))
    assert C.iamap_device_status() & C.IAMAP_DEV_BAD_INDEX
    check_attention(out.float().cpu().numpy(), lse.cpu().numpy(), q, k, v, bits, bits, table, lens, page)


def test_a_batch_of_empty_sequences(C):
    """No sequence has a token, and the page table no column."""
    from cross_model_attention_map_b200.runner import QuantAttention, QuantCache, QuantDecodeStep, QuantSenderRows
    ck = QuantCache(2, 16, 2, 64, 4)
    table, lens = torch.empty(3, 0, dtype=torch.int32, device="cuda"), i32([0, 0, 0])
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    r = QuantSenderRows(3, 4, 64, 0, H_k=2, ctx_stride=5)
    r.rows.fill_(float("nan"))
    assert not r.run(q, ck, table, lens).any()
    st = QuantDecodeStep(3, 4, 4, 64, 0, H_kv=2, ctx_stride=5)
    st.out.fill_(float("nan"))
    assert not st.run(r.rows, torch.randn(4, 4, device="cuda"), ck, table, lens).any()
    a = QuantAttention(3, 4, 64, 0, H_kv=2, want_lse=True)
    a.out.fill_(float("nan"))
    out, lse = a.run(q, ck, ck, table, lens)
    assert not out.any() and bool((lse == -math.inf).all())
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    ck.write(none, i32([0, 0, 0, 0]), lens, table)
    assert ck.read(i32([0, 0, 0, 0]), lens, table, none) is none
    assert C.iamap_device_status() == 0


# ------------------------------------------------------------------------------------------------
# Together
# ------------------------------------------------------------------------------------------------

class Decode:
    """The decode step of a sender layer and a mapped receiver layer over quantised caches: the sender
    appends its key and value and attends, its rows feed the receiver, which appends its value."""

    def __init__(self, lens, page, seed, max_ctx=None):
        from cross_model_attention_map_b200 import runner as R
        rng = np.random.default_rng(seed)
        self.lens, self.page = list(lens), page
        b, most = len(lens), max(lens) if max_ctx is None else max_ctx
        self.table, self.total = table_of(rng, [most] * b, page)
        self.k = pool_of(rng, lens, self.table, self.total, page, 2, 64, 4)
        self.v = pool_of(rng, lens, self.table, self.total, page, 2, 64, 8)
        self.r = pool_of(rng, lens, self.table, self.total, page, 8, 128, 4)
        self.caches = [cache(*self.k, 4), cache(*self.v, 8), cache(*self.r, 4)]
        draw = lambda *s: bf16_bits(rng.standard_normal(s).astype(np.float32))  # noqa: E731
        self.q, self.nk, self.nv, self.nr = draw(b, 6, 64), draw(b, 2, 64), draw(b, 2, 64), draw(b, 8, 128)
        self.W = rng.standard_normal((8, 6)).astype(np.float32)
        self.rows = R.QuantSenderRows(b, 6, 64, most, H_k=2)
        self.step = R.QuantDecodeStep(b, 6, 8, 128, most)
        self.attend = R.QuantAttention(b, 6, 64, most, H_kv=2, want_lse=True)
        self.dev = [bf16(x) for x in (self.q, self.nk, self.nv, self.nr)]
        self.devW, self.devt = torch.from_numpy(self.W).cuda(), i32(self.table)
        self.cu, self.starts, self.ctx = i32(range(b + 1)), i32([n - 1 for n in lens]), i32(lens)

    def run(self, stream=None):
        q, nk, nv, nr = self.dev
        for c, x in zip(self.caches, (nk, nv, nr)):
            c.write(x, self.cu, self.starts, self.devt, stream)
        rows = self.rows.run(q, self.caches[0], self.devt, self.ctx, stream)
        o, lse = self.attend.run(q, self.caches[0], self.caches[1], self.devt, self.ctx, stream)
        return rows, o, lse, self.step.run(rows, self.devW, self.caches[2], self.devt, self.ctx, stream)

    def check(self, lens, got):
        for (pool, scales), x, bits in ((self.k, self.nk, 4), (self.v, self.nv, 8), (self.r, self.nr, 4)):
            c, s = Q.quantise(bf16_bits_to_f64(x), bits)
            for b, n in enumerate(lens):
                pg, at = self.table[b, (n - 1) // self.page], (n - 1) % self.page
                pool[pg, :, at], scales[pg, :, at] = Q.pack(c[b], bits), s[b]
        rows, o, lse, out = (t.float().cpu().numpy() for t in got)
        q = bf16_bits_to_f64(self.q)
        check_rows(rows, q, *self.k, 4, self.table, lens, self.page)
        check_attention(o, lse, q, self.k, self.v, 4, 8, self.table, lens, self.page)
        check_mapped(out, rows, self.W, *self.r, 4, self.table, lens, self.page)


@pytest.mark.parametrize("page", [16, 24])
def test_a_decode_step(C, page):
    d = Decode([700, 1, 33, 1025], page, 61)
    d.check(d.lens, d.run())
    again = [t.clone() for t in d.run()]
    for a, b in zip(again, d.run()):
        assert torch.equal(a, b)                              # same inputs, same bits
    assert C.iamap_device_status() == 0


def test_captured_steps_replayed_with_other_lengths(C):
    """A captured step is replayed as the sequences grow; two captured steps with workspaces of their own
    run on two streams at once."""
    C.iamap_device_status()
    a, b = Decode([200, 17], 16, 62, max_ctx=2000), Decode([900, 400], 16, 63, max_ctx=2000)
    graphs = []
    for d in (a, b):
        d.check(d.lens, d.run())                              # eager first: the oracle's pages follow
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = d.run()
        graphs.append((g, got))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens_a, lens_b in (([201, 18], [901, 401]), ([202, 19], [902, 402]), ([203, 20], [903, 403])):
        for d, lens in ((a, lens_a), (b, lens_b)):
            d.starts.copy_(i32([n - 1 for n in lens]))
            d.ctx.copy_(i32(lens))
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        a.check(lens_a, graphs[0][1])
        b.check(lens_b, graphs[1][1])
    assert C.iamap_device_status() == 0


def test_on_a_stream_of_its_own(C):
    s = torch.cuda.Stream()
    d = Decode([130, 64], 16, 64)
    torch.cuda.synchronize()
    got = d.run(stream=s)
    s.synchronize()
    d.check(d.lens, got)


def test_mapped_step_equals_the_bf16_operator(C):
    """Values that both caches hold exactly (integers of at most 7 with a scale of 1 / 8): the quantised
    step and the bf16 step of the same rows agree to fp32 sums."""
    from cross_model_attention_map_b200.runner import DecodeStep, QuantDecodeStep
    rng = np.random.default_rng(71)
    lens, S, H, d, page = [500, 37], 3, 8, 64, 16
    table, total = table_of(rng, lens, page, spare=0)
    c = rng.integers(-7, 8, size=(total, page, H, d))
    c[..., ::32] = 7
    st = np.full((total, H, page, 2), 0.125, dtype=np.float16)
    ck = cache(np.ascontiguousarray(Q.pack(c, 4).transpose(0, 2, 1, 3)), st, 4)
    pages = bf16(bf16_bits((c / 8).astype(np.float32)))
    p, W = mapped_inputs(rng, lens, S, H, 500)
    args = torch.from_numpy(p).cuda(), torch.from_numpy(W).cuda()
    safe = np.where(table >= total, 0, table)
    a = QuantDecodeStep(2, S, H, d, 500).run(*args, ck, i32(safe), i32(lens))
    b = DecodeStep(2, S, H, d, lens, 500, table.shape[1], page, total).run(*args, pages, i32(safe))
    np.testing.assert_allclose(a.cpu().numpy(), b.cpu().numpy(), rtol=0, atol=500 * 2 * U)


def test_chunked_prefill_over_a_quantised_cache(C):
    """A prefill chunk whose keys and values live in quantised pages: written chunk by chunk, read back
    packed, then compress and mapped_av of the chunk equal the same calls on the values that the cache
    stands for."""
    from cross_model_attention_map_b200.runner import ChunkPrefillLayer, QuantCache
    rng = np.random.default_rng(72)
    H, d, page = 4, 64, 16
    starts, ends = [128, 0], [300, 90]
    table, total = table_of(rng, ends, page)
    xs = [bf16_bits(rng.standard_normal((sum(ends), H, d)).astype(np.float32)) for _ in range(2)]
    cu_k = np.concatenate([[0], np.cumsum(ends)])
    packed = []
    for x in xs:
        ck = QuantCache(total, page, H, d, 8)
        dev = bf16(x)
        for lo, hi in (([0, 0], starts), (starts, ends)):       # two chunks of every sequence
            new = [h - l for l, h in zip(lo, hi)]
            rows = torch.cat([dev[cu_k[s] + lo[s]:cu_k[s] + hi[s]] for s in range(2)])
            ck.write(rows, i32(np.concatenate([[0], np.cumsum(new)])), i32(lo), i32(table))
        out = torch.empty(sum(ends), H, d, dtype=torch.bfloat16, device="cuda")
        packed.append(ck.read(i32(cu_k), i32([0, 0]), i32(table), out))
        c, s = Q.quantise(bf16_bits_to_f64(x), 8)
        v = (c * np.repeat(s.astype(np.float64), 32, axis=-1)).astype(np.float32)
        assert torch.equal(out.cpu(), torch.from_numpy(v).to(torch.bfloat16))
    q = torch.cat([bf16(xs[0])[cu_k[s] + starts[s]:cu_k[s] + ends[s]] for s in range(2)])
    W = torch.randn(4, H, device="cuda")
    layer = ChunkPrefillLayer(starts, ends, H, d, 4, d, 0.95)
    got = layer.step(q, packed[0], W, packed[1])
    assert C.iamap_device_status() == 0 and bool(torch.isfinite(got).all()) and bool(got.any())


def test_chunked_prefill_over_a_quantised_cache_matches_its_values(C):
    """compress and mapped_av of a chunk whose keys and values were read back from quantised pages: the
    float64 oracle of the chunk on the values that the pages stand for, and the bits of the same calls on
    those values."""
    import dataclasses

    from cross_model_attention_map_b200.runner import ChunkPrefillLayer, QuantCache
    from oracle import chunked as CH
    from synth import chunk_of, make_prefill

    from _gpu_common import check_output, gpu_kept
    rng = np.random.default_rng(73)
    H, H_r, d, page, starts, ends = 4, 6, 64, 16, [128, 0], [300, 90]
    wl = make_prefill(ends, H_s=H, d=d, H_r=H_r, d_v=d, B=64, tau=0.9, seed=73)
    cw = chunk_of(wl, starts, ends)
    table, total = table_of(rng, ends, page)
    read, stand = [], []
    for x in (cw.k, cw.v):
        ck = QuantCache(total, page, x.shape[1], d, 8)
        ck.write(bf16(x), i32(cw.cu_k), i32([0, 0]), i32(table))
        read.append(ck.read(i32(cw.cu_k), i32([0, 0]), i32(table),
                            torch.empty(*x.shape, dtype=torch.bfloat16, device="cuda")))
        c, s = Q.quantise(bf16_bits_to_f64(x), 8)
        stand.append(bf16_bits((c * np.repeat(s.astype(np.float64), 32, axis=-1)).astype(np.float32)))
    W = torch.from_numpy(wl.W).cuda()
    outs, layers = [], []
    for k, v in (read, [bf16(x) for x in stand]):
        layers.append(ChunkPrefillLayer(starts, ends, H, d, H_r, d, wl.tau))
        outs.append(layers[-1].step(bf16(cw.q), k, W, v))
    torch.cuda.synchronize()
    assert C.iamap_device_status() == 0
    assert torch.equal(outs[0], outs[1])
    ref = dataclasses.replace(cw, k=stand[0], v=stand[1])
    check_output(outs[0].cpu().numpy(), CH.mapped_av_chunk(ref, gpu_kept(layers[0])))


@pytest.mark.parametrize("H,H_kv", [(4, 4), (6, 2), (16, 2)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_mapped_weights_that_are_not_finite(C, bits, H, H_kv, bad):
    """An infinity or NaN in a row of W reaches that receiver alone, one in a row of probabilities inside the context
    that sequence alone; the others are the same to the bit."""
    from cross_model_attention_map_b200.runner import QuantDecodeStep
    rng = np.random.default_rng(34)
    lens, S, d, page = [100, 1, 1100], 3, 64, 16
    table, total = table_of(rng, lens, page)
    ck = cache(*pool_of(rng, lens, table, total, page, H_kv, d, bits), bits)
    p, W = mapped_inputs(rng, lens, S, H, max(lens))
    run = lambda p, W: QuantDecodeStep(3, S, H, d, max(lens), H_kv=H_kv).run(  # noqa: E731
        torch.from_numpy(p).cuda(), torch.from_numpy(W).cuda(), ck, i32(table), i32(lens))
    clean = run(p, W)
    assert bool(torch.isfinite(clean).all())
    W2 = W.copy()
    W2[1, 2] = bad
    got = run(p, W2)
    rest = [r for r in range(H) if r != 1]
    assert not torch.isfinite(got[:, 1]).any() and torch.equal(got[:, rest], clean[:, rest])
    p2 = p.copy()
    p2[2, 0, 700] = bad
    got = run(p2, W)
    assert not torch.isfinite(got[2]).any() and torch.equal(got[:2], clean[:2])
    assert C.iamap_device_status() == 0
