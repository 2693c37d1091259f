"""CPU pins of the quantised-cache oracle (hand-worked groups, the error bound, the stored order) and
the refusals of its entry points, which validate their arguments on the host."""

import numpy as np
import pytest
import torch

from oracle import quant_cache as Q


def test_hand_worked_groups():
    x = np.zeros((5, 32))
    x[0, :4] = [7.0, -3.5, 0.5, 1.5]              # s = 1: ties go to the even level
    x[1, :3] = [1e6, -1e6, 3e5]                   # s saturates at 65504
    x[2, 0] = np.inf
    x[3, 0] = np.nan
    c, s = Q.quantise(x, 4)
    assert s[0, 0] == 1.0 and list(c[0, :4]) == [7, -4, 0, 2]
    assert s[1, 0] == 65504.0 and list(c[1, :3]) == [7, -7, 5]
    assert np.isnan(s[2, 0]) and np.isnan(s[3, 0]) and not c[2:].any()
    assert s[4, 0] == 0.0
    c, s = Q.quantise(np.full((1, 32), 127.0), 8)
    assert s[0, 0] == 1.0 and (c == 127).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_error_is_at_most_half_a_step(bits):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((400, 128)) * np.exp(rng.uniform(-6, 6, (400, 1)))
    c, s = Q.quantise(x, bits)
    step = np.repeat(s.astype(np.float64), 32, axis=-1)
    assert (np.abs(x - c * step) <= step * 0.5 * (1 + 1e-12)).all()
    assert np.abs(c).max() == Q.LEVELS[bits]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_stored_order(bits, d):
    """pack and unpack are inverse, and element 32 g + 4 r + i is code number r d / 8 + 4 g + i."""
    rng = np.random.default_rng(2)
    q = Q.LEVELS[bits]
    c = rng.integers(-q, q + 1, size=(3, 5, d))
    u = Q.pack(c, bits)
    assert u.shape == (3, 5, d * bits // 8) and (Q.unpack(u, bits) == c).all()
    for g in range(d // 32):
        for r in range(8):
            for i in range(4):
                at = r * (d // 8) + 4 * g + i
                byte = u[0, 0, at if bits == 8 else at // 2]
                code = int(byte) - 128 if bits == 8 else ((int(byte) >> (4 * (at % 2))) & 15) - 8
                assert code == c[0, 0, 32 * g + 4 * r + i]


def test_softmax_and_product_against_torch():
    rng = np.random.default_rng(3)
    pool = rng.integers(0, 256, size=(6, 2, 4, 64), dtype=np.uint8)
    scales = rng.uniform(0.01, 0.1, size=(6, 2, 4, 2)).astype(np.float16)
    table = np.array([[5, 0, 3], [1, 4, 2]], dtype=np.int32)
    q = rng.standard_normal((2, 4, 64))
    p, lse = Q.softmax_rows(q, pool, scales, 8, table, [11, 5], 4, 12)
    o, _ = Q.weighted_values(p, pool, scales, 8, table, [11, 5], 4)
    for b, n in enumerate([11, 5]):
        kv, _ = Q.sequence(pool, scales, 8, table, b, n, 4)
        k = torch.from_numpy(np.repeat(kv, 2, axis=1)).transpose(0, 1)
        x = (torch.from_numpy(q[b])[:, None] @ k.transpose(1, 2))[:, 0] / 8.0
        np.testing.assert_allclose(p[b, :, :n], torch.softmax(x, -1).numpy(), atol=1e-14)
        np.testing.assert_allclose(lse[b], torch.logsumexp(x, -1).numpy(), atol=1e-12)
        np.testing.assert_allclose(o[b], (torch.softmax(x, -1)[:, None] @ k)[:, 0].numpy(), atol=1e-12)
        assert not p[b, :, n:].any()


# ------------------------------------------------------------------------------------------------
# Refusals (no device work: every call below fails validation first, so no address is read)
# ------------------------------------------------------------------------------------------------

A = 4096   # an aligned address


@pytest.fixture(scope="module")
def lib():
    from cross_model_attention_map_b200 import build
    build.build()
    from cross_model_attention_map_b200 import iamap
    return iamap


def _write(lib, x=A, stride=256, n=4, cu=A, starts=A, seqs=1, table=A, max_pages=1, page=16, pages=1,
           H=2, d=64, bits=4, codes=A, scales=A):
    return lib._lib.iamap_cache_write(x, stride, n, cu, starts, seqs, table, max_pages, page, pages,
                                      H, d, bits, codes, scales, None)


def _read(lib, codes=A, scales=A, pages=1, table=A, max_pages=1, page=16, cu=A, starts=A, seqs=1, n=4,
          H=2, d=64, bits=4, out=A):
    return lib._lib.iamap_cache_read(codes, scales, pages, table, max_pages, page, cu, starts, seqs, n,
                                     H, d, bits, out, None)


def _rows(lib, q=A, codes=A, scales=A, pages=1, table=A, max_pages=2, page=16, lens=A, max_ctx=20,
          batch=1, H_s=4, H_k=2, d=64, bits=4, rows=A, stride=32, ws=A, ws_bytes=1 << 30):
    return lib._lib.iamap_sender_rows_quant(q, codes, scales, pages, table, max_pages, page, lens,
                                            max_ctx, batch, H_s, H_k, d, bits, rows, stride, ws,
                                            ws_bytes, None)


def _mapped(lib, rows=A, stride=32, W=A, codes=A, scales=A, pages=1, table=A, max_pages=2, page=16,
            lens=A, max_ctx=20, batch=1, H_s=4, H_r=4, H_kv=2, d=64, bits=4, out=A, ws=A,
            ws_bytes=1 << 30):
    return lib._lib.iamap_mapped_av_paged_quant(rows, stride, W, codes, scales, pages, table, max_pages,
                                                page, lens, max_ctx, batch, H_s, H_r, H_kv, d, bits, out,
                                                ws, ws_bytes, None)


def _attend(lib, q=A, kc=A, ks=A, kb=4, vc=A, vs=A, vb=8, pages=1, table=A, max_pages=2, page=16, lens=A,
            max_ctx=20, batch=1, H_q=4, H_kv=2, d=64, out=A, lse=None, ws=A, ws_bytes=1 << 30):
    return lib._lib.iamap_attention_paged_quant(q, kc, ks, kb, vc, vs, vb, pages, table, max_pages, page,
                                                lens, max_ctx, batch, H_q, H_kv, d, out, lse, ws,
                                                ws_bytes, None)


INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -6


@pytest.mark.parametrize("call", [_write, _read, _rows, _mapped])
def test_format_refusals(lib, call):
    for bits in (0, 2, 5, 16):
        assert call(lib, bits=bits) == UNSUPPORTED and "4 or 8 bits" in lib.iamap_last_error()
    for d in (0, 32, 96, 256):
        assert call(lib, d=d) == UNSUPPORTED
    for bad in (dict(codes=None), dict(scales=None), dict(table=None), dict(codes=A + 8),
                dict(scales=A + 2), dict(pages=-1), dict(max_pages=-1), dict(page=0)):
        assert call(lib, **bad) == INVALID, bad


@pytest.mark.parametrize("call,bad", [
    (_write, dict(x=None)), (_write, dict(x=A + 2)), (_write, dict(stride=120)), (_write, dict(stride=129)),
    (_write, dict(n=-1)), (_write, dict(n=2**31)), (_write, dict(seqs=0)), (_write, dict(cu=None)),
    (_write, dict(starts=None)), (_write, dict(H=0)),
    (_read, dict(out=None)), (_read, dict(out=A + 4)), (_read, dict(n=-1)), (_read, dict(seqs=0)),
    (_rows, dict(q=None)), (_rows, dict(rows=None)), (_rows, dict(lens=None)), (_rows, dict(H_k=3)),
    (_rows, dict(H_s=0)), (_rows, dict(batch=0)), (_rows, dict(max_ctx=33)), (_rows, dict(max_ctx=-1)),
    (_rows, dict(stride=19)), (_rows, dict(q=A + 2)),
    (_mapped, dict(rows=None)), (_mapped, dict(W=None)), (_mapped, dict(out=None)),
    (_mapped, dict(out=A + 4)), (_mapped, dict(H_kv=3)), (_mapped, dict(H_kv=0)), (_mapped, dict(stride=19)),
    (_mapped, dict(max_ctx=33)), (_mapped, dict(lens=None)),
    (_attend, dict(q=None)), (_attend, dict(out=None)), (_attend, dict(out=A + 2)),
    (_attend, dict(H_kv=3)), (_attend, dict(max_ctx=33)), (_attend, dict(kc=None)), (_attend, dict(vs=None)),
    (_attend, dict(vc=A + 4)), (_attend, dict(batch=0)),
])
def test_argument_refusals(lib, call, bad):
    assert call(lib, **bad) == INVALID and lib.iamap_last_error()


def test_other_refusals(lib):
    assert _mapped(lib, H_s=129) == UNSUPPORTED
    assert _mapped(lib, H_r=130) == UNSUPPORTED
    assert _mapped(lib, H_s=0) != 0
    assert _attend(lib, kb=3) == UNSUPPORTED and _attend(lib, vb=16) == UNSUPPORTED
    for call in (_rows, _mapped, _attend):
        assert call(lib, ws=None) == WORKSPACE
        assert call(lib, ws_bytes=0) == WORKSPACE
    # nothing to do: no row, no launch
    assert _write(lib, n=0) == 0 and _read(lib, n=0) == 0


def test_workspace_queries(lib):
    for f in (lib.iamap_mapped_av_paged_quant_workspace_bytes,
              lib.iamap_attention_paged_quant_workspace_bytes):
        assert f(4, 64, 128, 8704) > 0 and f(0, 64, 128, 8704) == 0
        assert f(64, 64, 128, 131072) >= f(1, 64, 128, 131072)
    assert lib.iamap_sender_rows_quant_workspace_bytes(4, 14, 8704) > 0


def test_runner_refusals(lib):
    from cross_model_attention_map_b200.runner import QuantCache
    codes = torch.zeros(3, 2, 16, 32, dtype=torch.uint8)
    scales = torch.zeros(3, 2, 16, 2, dtype=torch.float16)
    c = QuantCache.over(codes, scales, 4)
    assert (c.num_pages, c.H, c.page_size, c.d) == (3, 2, 16, 64)
    with pytest.raises(ValueError):
        QuantCache.over(codes, scales, 3)
    with pytest.raises(ValueError):
        QuantCache.over(codes, scales.float(), 4)
    with pytest.raises(ValueError):
        QuantCache.over(codes, scales, 8)                     # the row is not d bytes with d / 32 scales
    with pytest.raises(ValueError):
        QuantCache.over(codes.transpose(1, 2), scales, 4)
    with pytest.raises(ValueError):
        QuantCache(3, 16, 2, 96, 4, device="cpu")
    empty = QuantCache(3, 16, 2, 64, 4, device="cpu")
    from oracle import quant_cache as Q
    assert not Q.values(empty.codes.numpy(), empty.scales.numpy(), 4).any()


def test_runner_refuses_a_cache_on_another_device(lib):
    from cross_model_attention_map_b200.runner import (QuantAttention, QuantCache, QuantDecodeStep,
                                                       QuantSenderRows)
    ck = QuantCache(1, 16, 2, 64, 4, device="cpu")
    meta = lambda *shape, t=torch.float32: torch.empty(*shape, dtype=t, device="meta")  # noqa: E731
    q, lens = meta(1, 2, 64, t=torch.bfloat16), meta(1, t=torch.int32)
    table = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="on meta expected"):
        QuantSenderRows(1, 2, 64, 16, device="meta").run(q, ck, table, lens)
    with pytest.raises(ValueError, match="on meta expected"):
        QuantDecodeStep(1, 2, 2, 64, 16, device="meta").run(meta(1, 2, 16), meta(2, 2), ck, table, lens)
    with pytest.raises(ValueError, match="on meta expected"):
        QuantAttention(1, 2, 64, 16, device="meta").run(q, ck, ck, table, lens)


def test_no_rows(lib):
    """An empty tensor has no address."""
    assert _write(lib, n=0, x=None) == 0 and _read(lib, n=0, out=None) == 0


def test_batches_that_are_too_large(lib):
    """Refused by the calls, and the workspace queries name no size for them."""
    big = dict(batch=65536, ws_bytes=1 << 62)
    for call in (_rows, _mapped, _attend):
        assert call(lib, **big) == UNSUPPORTED, lib.iamap_last_error()
    assert _rows(lib, batch=65535, H_s=256, ws_bytes=1 << 62) == UNSUPPORTED
    assert _attend(lib, batch=65535, H_q=256, ws_bytes=1 << 62) == UNSUPPORTED
    assert lib.iamap_sender_rows_quant_workspace_bytes(65536, 4, 20) == 0
    assert lib.iamap_sender_rows_quant_workspace_bytes(65535, 1 << 30, 20) == 0
    assert lib.iamap_mapped_av_paged_quant_workspace_bytes(65536, 4, 64, 20) == 0
    assert lib.iamap_attention_paged_quant_workspace_bytes(65536, 4, 64, 20) == 0
    assert lib.iamap_attention_paged_quant_workspace_bytes(65535, 1 << 30, 64, 20) == 0
    for call in (_rows, _mapped, _attend):
        assert call(lib, ws=A + 8) == INVALID and "16-byte" in lib.iamap_last_error()


def test_contexts_that_are_too_long(lib):
    """max_ctx is bounded alike in the calls and in their workspace queries; what the grid cannot hold is refused
    whatever the workspace."""
    long = dict(max_ctx=(1 << 30) + 1, max_pages=1 << 27, stride=2**31 - 1)
    for call in (_rows, _mapped):
        assert call(lib, **long) == UNSUPPORTED and "2^30" in lib.iamap_last_error()
    del long["stride"]
    assert _attend(lib, **long) == UNSUPPORTED and "2^30" in lib.iamap_last_error()
    for n in ((1 << 30) + 1, 2**31 - 1):
        assert lib.iamap_sender_rows_quant_workspace_bytes(1, 4, n) == 0
        assert lib.iamap_mapped_av_paged_quant_workspace_bytes(1, 4, 64, n) == 0
        assert lib.iamap_attention_paged_quant_workspace_bytes(1, 4, 64, n) == 0
    assert lib.iamap_mapped_av_paged_quant_workspace_bytes(1, 4, 64, 1 << 30) > 0
    at_most = dict(max_ctx=1 << 30, max_pages=1 << 27, stride=1 << 30, ws_bytes=0)
    assert _mapped(lib, **at_most) == WORKSPACE
    assert _mapped(lib, **at_most, batch=1024) == UNSUPPORTED and "too large" in lib.iamap_last_error()
