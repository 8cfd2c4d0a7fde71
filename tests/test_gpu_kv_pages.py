"""GPU tests of the page caches: tq_append_kv_pages and tq_read_kv_pages (through the C ABI)
against a plain 64-bit restatement. Rotated vectors are held to the fp32 arithmetic's error
bound plus one rounding, MXFP4 codes and scales to equality; bytes that a call does not name
must keep their contents."""
import ctypes

import numpy as np
import pytest

import _pages as P

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import kv_cache_vector_05_b200 as T  # noqa: E402
from kv_cache_vector_05_b200 import _lib  # noqa: E402

DEV = "cuda:0"


def make_ctx(d):
    c, t = T.tq_lloyd_max_codebook(d, 2)
    return T.tq_codebook_load(d, 2, 4, c, t, None, hadamard_signs=np.ones(d, np.int8))


def table_for(rng, n_pos, rot):
    ang = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check_rotated(got, x, table, pos, interleaved, fmt):
    """|got - exact| <= two products and a sum in fp32 (2 x 2^-24 of |a c| + |b s|), then half a
    step of the type."""
    if table is None:
        np.testing.assert_array_equal(got, x)
        return
    want = P.rotate(x, table, pos, interleaved)
    err32 = 2 * 2.0 ** -24 * (1 + 2.0 ** -20) * P.rotate_abs(x, table, pos, interleaved) + 2.0 ** -148
    tol = err32 + P.EPS[fmt] * (np.abs(want) + err32) + P.TINY[fmt]
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()


CASES = [
    # fmt, d, hq, hkv, n, page, per_head, order, rot, interleaved, fused
    ("bf16", 128, 32, 8, 1, 16, False, "nhd", 128, False, True),
    ("bf16", 128, 4, 2, 333, 16, False, "hnd", 128, True, False),
    ("bf16", 64, 7, 1, 130, 1, False, "nhd", 16, False, False),
    ("bf16", 256, 3, 3, 65, 48, True, "nhd", 256, False, True),
    ("bf16", 128, 16, 2, 5000, 24, False, "gap", 64, False, True),
    ("f16", 64, 8, 4, 257, 7, False, "gap", 64, True, True),
    ("f16", 128, 5, 5, 100, 512, True, "nhd", 32, False, False),
    ("f16", 256, 1, 1, 3, 2, False, "nhd", 0, False, False),
    ("mxfp4", 64, 2, 2, 77, 16, False, "nhd", 32, False, True),
    ("mxfp4", 128, 32, 8, 700, 24, False, "hnd", 128, False, True),
    ("mxfp4", 128, 0, 3, 1, 512, True, "nhd", 16, True, False),
    ("mxfp4", 256, 4, 1, 200, 33, False, "gap", 96, False, False),
    ("mxfp4", 128, 4, 4, 3001, 64, True, "nhd", 0, False, True),
]


@pytest.mark.parametrize("fmt,d,hq,hkv,n,page,per_head,order,rot,interleaved,fused", CASES)
def test_append_and_read(fmt, d, hq, hkv, n, page, per_head, order, rot, interleaved, fused):
    rng = np.random.default_rng(n + d)
    ctx = make_ctx(d)
    n_pages = -(-n * (hkv if per_head else 1) // page) + 3
    cache = P.make_cache(fmt, n_pages, page, hkv, d, per_head, order)
    pages = T.KVPages(*cache)
    dt = P.TORCH[fmt]
    x = rng.standard_normal((n, hq + 2 * hkv, d)) * np.exp(rng.standard_normal(d) * 2)
    x[:, :, rng.integers(d)] = 0
    x = up(x.astype(np.float32)).to(dt)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q = q if hq else None
    slot = P.slots_for(rng, n, n_pages, page, hkv, per_head)
    if n > 50:
        slot[[7, 40]] = -1                            # padding rows
    live = (slot != -1).reshape(n, -1)[:, 0]
    table = table_for(rng, 4000, rot) if rot else None
    pos = rng.integers(0, 4000, n)
    if n > 50 and rot:
        pos[7] = -123456                              # a padding row's position is not read
    q_out = torch.full((n, hq, d), 77.0, dtype=dt, device=DEV) if hq else None
    T.tq_append_kv_pages(ctx, pages, k, v, up(slot), q=q, q_out=q_out, cos_sin=None if table is None else up(table),
                         positions=up(pos) if rot else None, interleaved=interleaved)
    T.tq_check_device(ctx)
    pos = np.where(live, pos, 0)
    if hq:
        got = P.f64(q_out)
        check_rotated(got[live], P.f64(q)[live], table, pos[live], interleaved, fmt)
        assert (got[~live] == 77.0).all()
    if fmt == "mxfp4":
        for xx, w in ((k, 0), (v, 1)):
            x32 = P.f64(xx).astype(np.float32)
            if w == 0 and rot:
                x32 = P.rotate(x32, table, pos, interleaved, np.float32)
            codes, scales = P.quantise(x32)
            np.testing.assert_array_equal(P.gather(cache, slot[live], hkv, w).numpy(), codes[live])
            np.testing.assert_array_equal(P.gather(cache, slot[live], hkv, w + 2).numpy(), scales[live])
    else:
        check_rotated(P.f64(P.gather(cache, slot[live], hkv, 0)), P.f64(k)[live], table, pos[live], interleaved, fmt)
        np.testing.assert_array_equal(P.f64(P.gather(cache, slot[live], hkv, 1)), P.f64(v)[live])
    # bytes of other rows keep their contents
    rows = np.setdiff1d(np.arange(n_pages * page), slot.reshape(-1))
    for t in cache:
        if t is not None:
            raw = t.cpu().contiguous().view(torch.uint8).reshape(n_pages * page, -1)
            assert (raw[torch.from_numpy(rows)] == P.SENTINEL).all()
    # read back, repeated rows included
    rd = np.concatenate([slot, slot[: n // 3]])
    ko, vo = T.tq_read_kv_pages(ctx, pages, up(rd), hkv, k_out=torch.full((len(rd), hkv, d), 3.0, dtype=dt, device=DEV))
    T.tq_check_device(ctx)
    lv = (rd != -1).reshape(len(rd), -1)[:, 0]
    for got, w in ((ko, 0), (vo, 1)):
        want = P.gather(cache, rd[lv], hkv, w)
        want = (P.dequantise(want.numpy(), P.gather(cache, rd[lv], hkv, w + 2).numpy()) if fmt == "mxfp4"
                else P.f64(want))
        np.testing.assert_array_equal(P.f64(got)[lv], want)
    assert (P.f64(ko)[~lv] == 3.0).all()
    only, none = T.tq_read_kv_pages(ctx, pages, up(rd[lv]), hkv, values=False)
    assert none is None and torch.equal(only.cpu(), ko.cpu()[torch.from_numpy(lv)])
    none, only = T.tq_read_kv_pages(ctx, pages, up(rd[lv]), hkv, keys=False)
    assert none is None and torch.equal(only.cpu(), vo.cpu()[torch.from_numpy(lv)])


def test_mxfp4_ties_extremes_and_nonfinite():
    """Every tie, saturation, subnormal and largest blocks, zero blocks, infinities and NaN."""
    d = 64
    ctx = make_ctx(d)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.5, 0.2500001])
    rows = np.zeros((12, 1, d), np.float32)
    rows[0, 0, :10], rows[0, 0, 32:42] = ties, -ties
    rows[1, 0, 0] = 4.0                                # the rest of the block rounds to zero
    rows[1, 0, 1:32] = 0.25
    rows[2, 0, :32] = 2.0 ** -130
    rows[2, 0, 32:] = 2.0 ** -133
    rows[3, 0, :32] = 3.3895314e38                     # the largest bf16
    rows[4] = -0.0
    rows[5, 0, 3], rows[5, 0, 40] = np.inf, -np.inf
    rows[6, 0, 3] = np.nan
    rows[7, 0, ::2] = 2.0 ** np.arange(32)
    rows[8] = np.float32(2.0 ** -126)
    rows[9:] = np.random.default_rng(0).standard_normal((3, 1, d)) * 2.0 ** 100
    x = up(rows).to(torch.bfloat16)
    cache = P.make_cache("mxfp4", 2, 8, 1, d, False)
    slot = up(np.arange(12, dtype=np.int64) + 2)
    T.tq_append_kv_pages(ctx, T.KVPages(*cache), x, x, slot)
    T.tq_check_device(ctx)
    codes, scales = P.quantise(P.f64(x))
    for w in (0, 1):
        got_c, got_s = (P.gather(cache, slot.cpu().numpy(), 1, i).numpy() for i in (w, w + 2))
        np.testing.assert_array_equal(got_s, scales)
        # the sign of a value that rounds to zero is free
        np.testing.assert_array_equal(P.dequantise(got_c, got_s), P.dequantise(codes, scales))
    k, v = T.tq_read_kv_pages(ctx, T.KVPages(*cache), slot, 1)
    np.testing.assert_array_equal(P.f64(k), P.dequantise(codes, scales))
    assert np.isnan(P.f64(k)[5]).all() and np.isnan(P.f64(k)[6, 0, :32]).all() and (P.f64(k)[6, 0, 32:] == 0).all()
    # every scale byte reads back as its value
    allc = P.make_cache("mxfp4", 256, 1, 1, d, False)
    allc[0].fill_(0x21)
    allc[1].fill_(0xF9)
    for t in allc[2:]:
        t.copy_(torch.arange(256, dtype=torch.uint8, device=DEV)[:, None, None, None].expand_as(t))
    k, v = T.tq_read_kv_pages(ctx, T.KVPages(*allc), up(np.arange(256)), 1)
    for got, w in ((k, 0), (v, 1)):
        want = P.dequantise(allc[w].cpu().numpy(), allc[w + 2].cpu().numpy()).reshape(256, 1, d)
        want = torch.from_numpy(want).to(torch.bfloat16).double().numpy()       # 6 x 2^127 is beyond bf16
        np.testing.assert_array_equal(P.f64(got), want)


def test_append_in_place_queries_and_bad_indexes():
    d, n, hq, hkv, page = 128, 300, 6, 2, 16
    rng = np.random.default_rng(5)
    ctx = make_ctx(d)
    x = up(rng.standard_normal((n, hq + 2 * hkv, d)).astype(np.float32)).to(torch.bfloat16)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    table, pos = up(table_for(rng, 500, 128)), rng.integers(0, 500, n)
    cache = P.make_cache("bf16", 25, page, hkv, d, False)
    pages = T.KVPages(*cache)
    slot = P.slots_for(rng, n, 25, page, hkv, False)
    want = T.tq_append_kv_pages(ctx, pages, k, v, up(slot), q=q, cos_sin=table, positions=up(pos))
    keep = [t.clone() for t in cache[:2]]
    xx = x.clone()
    got = T.tq_append_kv_pages(ctx, pages, xx[:, hq:hq + hkv], xx[:, hq + hkv:], up(slot), q=xx[:, :hq],
                               q_out=xx[:, :hq], cos_sin=table, positions=up(pos))
    T.tq_check_device(ctx)
    assert torch.equal(got, want) and torch.equal(xx[:, hq:], x[:, hq:])
    assert all(torch.equal(a, b) for a, b in zip(cache[:2], keep))
    # a bad slot and a bad position: reported, not written, the others are
    cache = P.make_cache("bf16", 25, page, hkv, d, False)
    pages = T.KVPages(*cache)
    bad_slot, bad_pos = slot.copy(), pos.copy()
    bad_slot[3], bad_slot[9], bad_pos[20], bad_pos[21] = 25 * page, -2, 500, -1
    T.tq_append_kv_pages(ctx, pages, k, v, up(bad_slot), q=q, cos_sin=table, positions=up(bad_pos))
    with pytest.raises(T.TQError):
        T.tq_check_device(ctx)
    T.tq_check_device(ctx)                             # the word is cleared
    ok = np.setdiff1d(np.arange(n), [3, 9, 20, 21])
    for w in (0, 1):
        assert torch.equal(P.gather(cache, slot[ok], hkv, w), P.gather(keep, slot[ok], hkv, w))
        raw = P.gather(cache, slot[[3, 9, 20, 21]], hkv, w).contiguous().view(torch.uint8)
        assert (raw == P.SENTINEL).all()
    out = torch.full((3, hkv, d), 9.0, dtype=torch.bfloat16, device=DEV)
    T.tq_read_kv_pages(ctx, pages, up(np.array([slot[0], 25 * page, slot[1]])), hkv, k_out=out)
    with pytest.raises(T.TQError):
        T.tq_check_device(ctx)
    assert (out[1] == 9.0).all() and torch.equal(out[0].cpu(), P.gather(cache, slot[:1], hkv, 0)[0])


def test_append_per_head_slots_may_be_padding_one_by_one():
    d, n, hkv, page = 64, 40, 3, 32
    rng = np.random.default_rng(6)
    ctx = make_ctx(d)
    k, v = (up(rng.standard_normal((n, hkv, d)).astype(np.float32)).to(torch.float16) for _ in range(2))
    q = k[:, :2].contiguous()
    cache = P.make_cache("f16", 6, page, hkv, d, True)
    slot = P.slots_for(rng, n, 6, page, hkv, True)
    slot[rng.random(slot.shape) < 0.3] = -1
    slot[5] = -1
    pos, table = rng.integers(0, 99, n), up(table_for(rng, 99, 64))
    pos[5] = 10 ** 9                                   # a row without slots has no position
    out = torch.full_like(q, 7.0)
    T.tq_append_kv_pages(ctx, T.KVPages(*cache), k, v, up(slot), q=q, q_out=out, cos_sin=table, positions=up(pos))
    T.tq_check_device(ctx)
    live = slot != -1
    flat = cache[1].cpu().reshape(-1, d)
    assert torch.equal(flat[torch.from_numpy(slot[live])], v.cpu()[torch.from_numpy(live)])
    assert (out.cpu()[torch.from_numpy(slot[:, 0] == -1)] == 7.0).all()
    assert not (out.cpu()[torch.from_numpy(slot[:, 0] != -1)] == 7.0).all(-1).any()
    rows = np.setdiff1d(np.arange(6 * page), slot[live])
    assert (cache[0].cpu().view(torch.uint8).reshape(6 * page, -1)[torch.from_numpy(rows)] == P.SENTINEL).all()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_append_and_read_past_32_bit_offsets(fmt):
    """Pages that lie more than 2^32 bytes apart."""
    d, hkv = 128, 2
    ctx = make_ctx(d)
    big = torch.zeros((1 << 32) + (1 << 20), dtype=torch.uint8, device=DEV)
    if fmt == "bf16":
        flat = big.view(torch.bfloat16)
        kc = flat.as_strided((2, 16, hkv, d), (1 << 31, hkv * d, d, 1))
        vc = flat.as_strided((2, 16, hkv, d), (1 << 31, hkv * d, d, 1), storage_offset=1 << 16)
        cache = (kc, vc, None, None)
    else:
        kc = big.as_strided((2, 16, hkv, 64), (1 << 32, hkv * 64, 64, 1))
        vc = big.as_strided((2, 16, hkv, 64), (1 << 32, hkv * 64, 64, 1), storage_offset=1 << 16)
        ks = big.as_strided((2, 16, hkv, 4), (1 << 32, hkv * 4, 4, 1), storage_offset=1 << 17)
        vs = big.as_strided((2, 16, hkv, 4), (1 << 32, hkv * 4, 4, 1), storage_offset=1 << 18)
        cache = (kc, vc, ks, vs)
    k, v = (torch.randn((5, hkv, d), device=DEV).to(torch.bfloat16) for _ in range(2))
    slot = up(np.array([31, 2, 17, 16, 15]))
    pages = T.KVPages(*cache)
    T.tq_append_kv_pages(ctx, pages, k, v, slot)
    ko, vo = T.tq_read_kv_pages(ctx, pages, slot, hkv)
    T.tq_check_device(ctx)
    if fmt == "bf16":
        assert torch.equal(ko, k) and torch.equal(vo, v)
        assert torch.equal(kc[1, 15], k[0]) and torch.equal(vc[0, 15], v[4])
    else:
        np.testing.assert_array_equal(P.f64(ko), P.dequantise(*P.quantise(P.f64(k))))
        np.testing.assert_array_equal(P.f64(vo), P.dequantise(*P.quantise(P.f64(v))))


def test_append_read_on_a_stream_and_in_a_graph():
    d, n, hkv, page = 128, 64, 2, 16
    ctx = make_ctx(d)
    k, v = (torch.randn((n, hkv, d), device=DEV).to(torch.bfloat16) for _ in range(2))
    cache = P.make_cache("bf16", 8, page, hkv, d, False)
    pages, slot = T.KVPages(*cache), up(np.random.default_rng(0).permutation(128)[:n].astype(np.int64))
    out = torch.empty((2, n, hkv, d), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    T.tq_append_kv_pages(ctx, pages, k, v, slot, stream=side)
    T.tq_read_kv_pages(ctx, pages, slot, hkv, k_out=out[0], v_out=out[1], stream=side)
    side.synchronize()
    assert torch.equal(out[0], k) and torch.equal(out[1], v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.tq_append_kv_pages(ctx, pages, k, v, slot)
        T.tq_read_kv_pages(ctx, pages, slot, hkv, k_out=out[0], v_out=out[1])
    for i in range(3):
        k.normal_(), v.normal_()
        slot.copy_(up(np.random.default_rng(i).permutation(128)[:n].astype(np.int64)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], k) and torch.equal(out[1], v)
    T.tq_check_device(ctx)


def test_append_and_read_refusals():
    d, hkv = 128, 2
    ctx = make_ctx(d)
    cache = P.make_cache("bf16", 4, 16, hkv, d, False)
    pages = T.KVPages(*cache)
    k = torch.zeros((3, hkv, d), dtype=torch.bfloat16, device=DEV)
    slot = up(np.arange(3))
    with pytest.raises(ValueError):
        T.tq_append_kv_pages(ctx, pages, k.half(), k.half(), slot)               # another type than the cache
    with pytest.raises(ValueError):
        T.tq_append_kv_pages(ctx, pages, k, k, slot.int())                       # slot type
    with pytest.raises(ValueError):
        T.tq_append_kv_pages(ctx, pages, k, k, up(np.zeros((3, hkv), np.int64)))  # slot shape
    with pytest.raises(ValueError):
        T.tq_append_kv_pages(ctx, pages, k[:, :1], k[:, :1], slot)               # KV heads
    with pytest.raises(ValueError):
        T.tq_append_kv_pages(make_ctx(64), pages, k, k, slot)                    # d
    with pytest.raises(ValueError):
        T.KVPages(cache[0], cache[1].transpose(0, 1))
    with pytest.raises(ValueError):
        T.KVPages(cache[0].view(torch.uint8), cache[1].view(torch.uint8))        # MXFP4 without scales
    with pytest.raises(ValueError):
        T.KVPages(cache[0].float(), cache[1].float())
    pos, tab = up(np.zeros(3, np.int64)), torch.zeros((10, 24), device=DEV)
    for bad in (tab, torch.zeros((10, 144), device=DEV)):                        # rot_dim 24; above d
        with pytest.raises(T.TQError) as e:
            T.tq_append_kv_pages(ctx, pages, k, k, slot, cos_sin=bad, positions=pos)
        assert e.value.status == _lib.TQ_EUNSUPPORTED
    odd = torch.zeros(3 * 260 + 8, dtype=torch.bfloat16, device=DEV)
    for t in (odd[1:].as_strided((3, hkv, d), (264, d, 1)), odd.as_strided((3, hkv, d), (260, d, 1))):
        with pytest.raises(T.TQError) as e:                                      # unaligned rows
            T.tq_append_kv_pages(ctx, pages, t, k, slot)
        assert e.value.status == _lib.TQ_EINVAL
    st = _lib.tq_kv_pages.from_buffer_copy(pages._struct)
    st.hkv, st.token_stride = hkv, 8                                             # tokens overlap
    args = (_lib.TQ_BF16, 3, 0, None, 0, k.data_ptr(), 256, k.data_ptr(), 256, None, slot.data_ptr(), None, 0, None)
    assert _lib.lib.tq_append_kv_pages(ctx.handle, ctypes.byref(st), *args) == _lib.TQ_EINVAL
    assert b"strides" in _lib.lib.tq_last_error()
    T.tq_append_kv_pages(ctx, pages, k[:0], k[:0], slot[:0])                     # no rows: nothing to do
    T.tq_check_device(ctx)
    for t in cache[:2]:
        assert (t.view(torch.uint8) == P.SENTINEL).all()
