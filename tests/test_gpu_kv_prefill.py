"""GPU tests of tq_prefill_kv_pages (through the C ABI) against softmax attention in 64 bits.

Tolerances, beside the ones of the decode tests: a probability enters the product with the values
rounded to q's type (half a step of it, relative), so the output may move by that much of the
probability-weighted |v| (no more than max|v|), and by the same again through the sum."""
import numpy as np
import pytest

import _pages as P
from test_gpu_kv_decode import block_tables, random_cache, tokens
from test_gpu_kv_pages import make_ctx, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import kv_cache_vector_05_b200 as T  # noqa: E402
from kv_cache_vector_05_b200 import _lib  # noqa: E402

DEV = "cuda:0"


def check(cache, table, q_lens, kv_lens, cu, q, out, lse, page, per_head, hkv, window, fmt, scale=None, rows=None):
    total, hq, d = q.shape
    g, scale = hq // hkv, scale or d ** -0.5
    q64, out, lse = P.f64(q), P.f64(out), P.f64(lse)
    typ = "f16" if fmt == "f16" else "bf16"
    for b, (nq, n) in enumerate(zip(q_lens, kv_lens)):
        s = int(cu[b])
        pick = np.arange(nq) if rows is None else np.unique(np.clip(rows, 0, max(nq - 1, 0)))[: max(nq, 0)]
        for h in range(hkv):
            hs = slice(h * g, (h + 1) * g)
            k, v = (tokens(cache, table, b, h, int(n), page, per_head, hkv, w) for w in (0, 1))
            pos = pick + int(n) - int(nq)
            qq = q64[s + pick][:, hs]
            want, wl = P.attend(qq, k, v, pos, window, scale)
            o, ls = out[s + pick][:, hs], lse[s + pick][:, hs]
            none = np.isneginf(wl)
            assert np.isneginf(ls[none]).all() and (o[none] == 0).all()
            if n == 0:
                continue
            size = np.abs(qq).max(1) @ np.abs(k).T                        # [rows, n], an upper bound over the heads
            delta = scale * (d / 8 + 4) * 2.0 ** -23 * size.max(-1)
            steps = (n / 16 + 40) * 2.0 ** -23
            rel = 2 * (delta + P.EPS[typ] + 2.0 ** -21 + steps)
            vmax = np.abs(v).max(0)
            tol = rel[:, None, None] * vmax + n * 2.0 ** -37 * vmax + P.EPS[typ] * np.abs(want) + P.TINY[typ]
            assert (np.abs(o - want) <= tol).all(), (b, h, np.abs(o - want).max(), np.argmax((np.abs(o - want) / tol).max((1, 2))))
            with np.errstate(invalid="ignore"):
                tl = (delta + steps + 2.0 ** -20)[:, None] + np.abs(wl) * 2.0 ** -21
                assert (np.abs(ls - wl) <= tl)[~none].all(), (b, h, np.nanmax(np.abs(ls - wl)[~none]))


CASES = [
    # fmt, d, g, hkv, (q_len, kv_len)s, page, per_head, order, window
    ("bf16", 128, 4, 2, [(1, 1), (64, 64), (100, 333), (0, 50), (7, 200)], 16, False, "nhd", 0),
    ("bf16", 128, 1, 2, [(300, 300), (129, 1000)], 16, False, "hnd", 0),
    ("bf16", 128, 8, 1, [(33, 500)], 7, False, "gap", 0),
    ("bf16", 128, 3, 1, [(250, 251), (1, 129), (86, 128)], 48, True, "nhd", 40),
    ("bf16", 64, 5, 2, [(130, 777), (2, 3)], 16, False, "nhd", 0),
    ("bf16", 64, 1, 4, [(513, 513)], 1, False, "nhd", 100),
    ("bf16", 256, 2, 2, [(100, 150), (65, 65), (1, 700)], 16, False, "nhd", 0),
    ("bf16", 256, 4, 1, [(40, 300)], 33, True, "nhd", 65),
    ("f16", 128, 4, 2, [(200, 450), (17, 17)], 32, False, "nhd", 0),
    ("f16", 64, 8, 1, [(70, 600), (128, 128)], 24, True, "nhd", 128),
    ("f16", 256, 1, 1, [(140, 300)], 16, False, "gap", 1),
    ("mxfp4", 128, 8, 2, [(64, 300), (33, 33)], 16, False, "nhd", 0),
    ("mxfp4", 128, 2, 1, [(140, 1111)], 512, True, "nhd", 200),
    ("mxfp4", 64, 4, 2, [(77, 200), (1, 1)], 5, False, "hnd", 0),
    ("mxfp4", 256, 3, 1, [(50, 260)], 16, False, "nhd", 0),
    ("mxfp4", 128, 8, 2, [(140, 300), (3, 50), (0, 7), (129, 129)], 16, False, "nhd", 0),  # expanded first
    ("mxfp4", 64, 4, 1, [(300, 500), (1, 1)], 7, False, "gap", 150),
    ("mxfp4", 256, 4, 2, [(130, 400)], 64, True, "nhd", 0),
    ("mxfp4", 128, 64, 1, [(20, 3000), (9, 5)], 48, False, "hnd", 700),
    ("bf16", 128, 4, 1, [(5, 2), (3, 0), (200, 150)], 16, False, "nhd", 0),      # rows before the first token
    ("bf16", 128, 16, 1, [(16, 9000)], 16, False, "nhd", 0),                     # tokens split over CTAs
    ("f16", 64, 2, 1, [(3, 5000), (1, 1), (2, 4097)], 16, False, "nhd", 3000),
    ("mxfp4", 128, 6, 2, [(4, 7000)], 512, True, "nhd", 0),
    ("bf16", 256, 8, 1, [(2, 4200), (2, 10)], 16, False, "nhd", 0),
]


@pytest.mark.parametrize("fmt,d,g,hkv,lens,page,per_head,order,window", CASES)
def test_prefill(fmt, d, g, hkv, lens, page, per_head, order, window):
    rng = np.random.default_rng(d + g + len(lens))
    ctx = make_ctx(d)
    q_lens, kv_lens = np.array([x[0] for x in lens]), np.array([x[1] for x in lens])
    max_len, max_q = int(kv_lens.max()) + 2, int(q_lens.max())
    n_pages = int((-(-kv_lens // page)).sum()) * (hkv if per_head else 1) + 1
    cache = random_cache(rng, fmt, n_pages, page, hkv, d, per_head, order)
    table = block_tables(rng, kv_lens, page, hkv, per_head, -(-max_len // page), n_pages)
    bad = [float("nan"), float("inf"), float("-inf")]    # slots past the sequences hold anything
    for b, n in enumerate(kv_lens):
        for h in range(hkv if per_head else 1):
            row = table[b, h] if per_head else table[b]
            for t in range(n, -(-n // page) * page):
                for x in (cache[:2] if fmt != "mxfp4" else cache[2:]):
                    x[int(row[t // page]), t % page] = bad[t % 3] if fmt != "mxfp4" else 255
    dt = P.TORCH[fmt]
    total = int(q_lens.sum()) + 3                        # three rows of no sequence
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    qq = torch.randn((total, hkv * g + 2, d), device=DEV).to(dt)
    q = qq[:, 1:hkv * g + 1]                             # strided rows
    out = torch.full((total, hkv * g, d), 5.0, dtype=dt, device=DEV)
    lse = torch.full((total, hkv * g), 6.0, device=DEV)
    T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), max_len, up(cu), max_q,
                          seq_lens=up(kv_lens.astype(np.int32)), window=window, out=out, lse=lse)
    T.tq_check_device(ctx)
    assert (out[total - 3:] == 5.0).all() and (lse[total - 3:] == 6.0).all()
    check(cache, table, q_lens, kv_lens, cu, q, out, lse, page, per_head, hkv, window, fmt)


def simple(rng, fmt, d, g, hkv, lens, page=16, extra=1, max_len=None):
    q_lens, kv_lens = np.array([x[0] for x in lens]), np.array([x[1] for x in lens])
    n_pages = int((-(-kv_lens // page)).sum()) + extra
    cache = random_cache(rng, fmt, n_pages, page, hkv, d, False)
    max_len = max_len or int(kv_lens.max())
    table = block_tables(rng, kv_lens, page, hkv, False, -(-max_len // page), n_pages)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = torch.randn((int(q_lens.sum()), hkv * g, d), device=DEV).to(P.TORCH[fmt])
    return q_lens, kv_lens, cache, table, cu, q


@pytest.mark.parametrize("fmt,d,g,max_len", [("bf16", 128, 2, 500), ("f16", 64, 2, 500), ("bf16", 256, 2, 500),
                                             ("mxfp4", 128, 2, 500), ("mxfp4", 128, 8, 500), ("mxfp4", 128, 4, 1 << 21)])
def test_prefill_nonfinite_values_reach_only_rows_that_see_them(fmt, d, g, max_len):
    """Infinities and NaN in keys and values of single tokens (on the diagonal, at the window's
    edge, in the middle), and a NaN query: every other row keeps its bits."""
    hkv, window = 2, 150
    rng = np.random.default_rng(11)
    ctx = make_ctx(d)
    q_lens, kv_lens, cache, table, cu, q = simple(rng, fmt, d, g, hkv, [(200, 500), (90, 90)], max_len=max_len)
    args = (hkv, up(table), max_len, up(cu), 200)
    kw = dict(seq_lens=up(kv_lens.astype(np.int32)), window=window)
    ref, rl = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), *args, **kw)
    base = [None if t is None else t.clone() for t in cache]
    for b, t, which, kind in ((0, 380, 1, "inf"), (0, 380, 1, "nan"), (0, 250, 1, "-inf"), (1, 40, 1, "nan"),
                              (0, 499, 1, "inf"), (0, 420, 0, "nan"), (1, 0, 0, "nan"), (0, 200, 1, "nan")):
        for x, y in zip(cache, base):
            if x is not None:
                x.copy_(y)
        at = (int(table[b, t // 16]), t % 16, 1)         # KV head 1, coordinates 32 to 63
        if fmt == "mxfp4":
            cache[which + 2][at][1] = 255
        elif which:
            cache[1][at][40] = float(kind)
        else:
            cache[0][at][40] = float("nan")
        out, lse = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), *args, **kw)
        T.tq_check_device(ctx)
        pos = np.arange(q_lens[b]) + kv_lens[b] - q_lens[b]
        sees = torch.from_numpy((pos >= t) & (pos - window < t)).to(DEV)
        bad = torch.zeros_like(out, dtype=torch.bool)
        rows = torch.arange(int(cu[b]), int(cu[b + 1]), device=DEV)[sees]
        if which:
            bad[rows, g:, 32:64] = True if fmt == "mxfp4" else bad[rows, g:, 32:64]
            if fmt != "mxfp4":
                bad[rows, g:, 40] = True
                want = out[rows, g:, 40]
                assert (torch.isnan(want) if kind == "nan" else want == float(kind)).all()
        else:
            bad[rows, g:] = True
            assert torch.isnan(lse[rows, g:]).all()
        assert torch.equal(torch.isfinite(out), ~bad), (b, t, which, kind)
        assert torch.equal(out[~bad], ref[~bad])
    for x, y in zip(cache, base):
        if x is not None:
            x.copy_(y)
    q2 = q.clone()
    q2[7, 3, 5] = float("nan")
    out, lse = T.tq_prefill_kv_pages(ctx, q2, T.KVPages(*cache), *args, **kw)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[7, 3] = True
    assert torch.equal(torch.isnan(out), bad) and torch.equal(out[~bad], ref[~bad])


@pytest.mark.parametrize("fmt", ["bf16", "f16", "mxfp4"])
def test_prefill_large_and_rising_logits(fmt):
    """Peaked rows, tiny scales, and keys that raise the maximum tile after tile."""
    d, g, hkv = 128, 4, 1
    rng = np.random.default_rng(12)
    ctx = make_ctx(d)
    q_lens, kv_lens, cache, table, cu, q = simple(rng, fmt, d, g, hkv, [(130, 900), (70, 70)])
    q = (q.float() * 8).to(q.dtype)
    args = (hkv, up(table), 900, up(cu), 130)
    for scale in (0.0, 1e-4, 2.0):
        out, lse = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), *args, seq_lens=up(kv_lens.astype(np.int32)),
                                         softmax_scale=scale)
        check(cache, table, q_lens, kv_lens, cu, q, out, lse, 16, False, hkv, 0, fmt, scale or None)
    if fmt == "mxfp4":
        return
    for t in range(900):
        cache[0][int(table[0, t // 16]), t % 16] = (q[60, :1].float() * (t / 900)).to(q.dtype)
    out, lse = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), *args, seq_lens=up(kv_lens.astype(np.int32)))
    check(cache, table, q_lens, kv_lens, cu, q, out, lse, 16, False, hkv, 0, fmt)


@pytest.mark.parametrize("fmt,page,window", [("bf16", 16, 40), ("bf16", 20, 40), ("mxfp4", 16, 40), ("f16", 128, 1)])
def test_prefill_window_reads_no_entry_before_it(fmt, page, window):
    """Pages that lie wholly before the first new row's window may be gone, as may those of
    positions past the sequence."""
    d, g, hkv = 64, 2, 1
    rng = np.random.default_rng(18)
    ctx = make_ctx(d)
    q_lens, kv_lens, cache, table, cu, q = simple(rng, fmt, d, g, hkv, [(7, 400), (130, 900), (1, 129), (300, 300)],
                                                  page=page, max_len=1000)
    gone = table.copy()
    for b, (nq, n) in enumerate(zip(q_lens, kv_lens)):
        gone[b, :max(0, n - nq - window + 1) // page] = -1
    out, lse = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(gone), 1000, up(cu), 300,
                                     seq_lens=up(kv_lens.astype(np.int32)), window=window)
    T.tq_check_device(ctx)
    check(cache, table, q_lens, kv_lens, cu, q, out, lse, page, False, hkv, window, fmt)


@pytest.mark.parametrize("d,g,hkv,page,window", [(128, 8, 2, 16, 0), (64, 8, 4, 5, 0), (256, 3, 1, 48, 90)])
def test_prefill_mxfp4_too_long_to_expand(d, g, hkv, page, window):
    """Several row blocks over MXFP4 pages where the call's longest sequence allows no workspace for
    all its tokens as bf16: each block turns the records itself."""
    rng = np.random.default_rng(19)
    ctx = make_ctx(d)
    max_len = (1 << 21) + 5
    lens = [(150, 700), (1, 1), (97, 97), (30, 20)]
    q_lens, kv_lens, cache, table, cu, q = simple(rng, "mxfp4", d, g, hkv, lens, page=page, max_len=max_len)
    assert T.tq_prefill_kv_pages_workspace_bytes(ctx, len(q), 4, hkv * g, hkv, max_len, 150) < 1 << 28
    out, lse = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), max_len, up(cu), 150,
                                     seq_lens=up(kv_lens.astype(np.int32)), window=window)
    T.tq_check_device(ctx)
    check(cache, table, q_lens, kv_lens, cu, q, out, lse, page, False, hkv, window, "mxfp4")


def test_prefill_one_row_equals_decode():
    """A chunk of one token per sequence is a decode step (up to P's rounding)."""
    d, g, hkv = 128, 4, 2
    rng = np.random.default_rng(13)
    ctx = make_ctx(d)
    q_lens, kv_lens, cache, table, cu, q = simple(rng, "bf16", d, g, hkv, [(1, 300), (1, 1), (1, 77), (1, 4000)])
    ln = up(kv_lens.astype(np.int32))
    out, lse = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 4000, up(cu), 1, seq_lens=ln)
    dec, dl = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 4000, seq_lens=ln)
    assert (out.float() - dec).abs().max() <= 2.0 ** -7 * dec.abs().max() + 2.0 ** -7
    assert (lse - dl).abs().max() <= 1e-4


def test_prefill_bad_ranges_and_pages_are_reported():
    d, g, hkv = 128, 2, 1
    rng = np.random.default_rng(14)
    ctx = make_ctx(d)
    q_lens, kv_lens, cache, table, cu, q = simple(rng, "bf16", d, g, hkv, [(30, 100), (20, 50), (10, 10)])
    ln = up(kv_lens.astype(np.int32))
    ref, rl = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 100, up(cu), 30, seq_lens=ln)
    T.tq_check_device(ctx)
    for c2, ok in (([0, 30, 20, 60], [True, False, False]), ([0, 30, 50, 61], [True, True, False]),
                   ([-1, 30, 50, 60], [False, True, True]), ([0, 30, 50, 2 ** 31 - 1], [True, True, False])):
        out, lse = torch.full_like(ref, 3.0), torch.full_like(rl, 4.0)
        T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 100, up(np.array(c2, np.int32)), 30,
                              seq_lens=ln, out=out, lse=lse)
        with pytest.raises(T.TQError):
            T.tq_check_device(ctx)
        for b in range(3):
            if ok[b]:
                assert torch.equal(out[cu[b]:cu[b + 1]], ref[cu[b]:cu[b + 1]])
            elif c2 != [0, 30, 20, 60]:
                assert (out[cu[b]:cu[b + 1]] == 3.0).all() and (lse[cu[b]:cu[b + 1]] == 4.0).all()
    # more rows than max_q: that sequence is skipped
    out = torch.full_like(ref, 3.0)
    T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 100, up(cu), 20, seq_lens=ln, out=out)
    with pytest.raises(T.TQError):
        T.tq_check_device(ctx)
    assert (out[:30] == 3.0).all() and torch.equal(out[30:], ref[30:])
    t2, t3 = table.copy(), table.copy()
    t2[0, 3], t3[0, 3] = -5, 0
    out, _ = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(t2), 100, up(cu), 30, seq_lens=ln)
    with pytest.raises(T.TQError):
        T.tq_check_device(ctx)
    want, _ = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(t3), 100, up(cu), 30, seq_lens=ln)
    assert torch.equal(out, want)
    none, _ = T.tq_prefill_kv_pages(ctx, q[:0], T.KVPages(*cache), hkv, up(table), 100, up(cu * 0), 30, seq_lens=ln)
    assert none.shape[0] == 0
    T.tq_check_device(ctx)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_prefill_past_32_bit_offsets(fmt):
    d, hkv, g, page = 128, 2, 4, 16
    rng = np.random.default_rng(15)
    ctx = make_ctx(d)
    big = torch.zeros((1 << 32) + (1 << 20), dtype=torch.uint8, device=DEV)
    src = random_cache(rng, fmt, 2, page, hkv, d, False)
    if fmt == "bf16":
        f = big.view(torch.bfloat16)
        st = (1 << 31, hkv * d, d, 1)
        cache = (f.as_strided((2, page, hkv, d), st), f.as_strided((2, page, hkv, d), st, 1 << 16), None, None)
    else:
        cache = tuple(big.as_strided((2, page, hkv, w), (1 << 32, hkv * w, w, 1), i << 16)
                      for i, w in enumerate((64, 64, 4, 4)))
    for x, y in zip(cache, src):
        if x is not None:
            x.copy_(y)
    table, cu = np.array([[1, 0]], np.int32), np.array([0, 25], np.int32)
    q = torch.randn((25, hkv * g, d), device=DEV).to(torch.bfloat16)
    out, lse = T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 32, up(cu), 25,
                                     seq_lens=up(np.array([30], np.int32)))
    T.tq_check_device(ctx)
    check(src, table, [25], [30], cu, q, out, lse, page, False, hkv, 0, fmt)


def test_prefill_repeats_on_streams_and_in_graphs():
    """The same bits from every run; captured and replayed with other lengths; two graphs that
    share a workspace of a split call."""
    d, g, hkv = 128, 4, 1
    rng = np.random.default_rng(16)
    ctx = make_ctx(d)
    q_lens, kv_lens, cache, table, cu, q = simple(rng, "bf16", d, g, hkv, [(20, 5000), (44, 44), (64, 3000)])
    pages, tab, cuq, ln = T.KVPages(*cache), up(table), up(cu), up(kv_lens.astype(np.int32))
    need = T.tq_prefill_kv_pages_workspace_bytes(ctx, len(q), 3, hkv * g, hkv, 5000, 64)
    assert need > 0                                      # tokens are split over CTAs
    ref, rl = T.tq_prefill_kv_pages(ctx, q, pages, hkv, tab, 5000, cuq, 64, seq_lens=ln)
    check(cache, table, q_lens, kv_lens, cu, q, ref, rl, 16, False, hkv, 0, "bf16", rows=np.array([0, 7, 19, 43, 63]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = T.tq_prefill_kv_pages(ctx, q, pages, hkv, tab, 5000, cuq, 64, seq_lens=ln)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    made = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        o, ls = torch.empty_like(ref), torch.empty_like(rl)
        with torch.cuda.graph(gr):
            T.tq_prefill_kv_pages(ctx, q, pages, hkv, tab, 5000, cuq, 64, seq_lens=ln, out=o, lse=ls, workspace=ws)
        made.append((gr, o, ls))
    for i in range(3):
        q.normal_()
        ln.copy_(up(np.array([5000 - 1000 * i, 44 - i, 64 + 500 * i], np.int32)))
        want, wl = T.tq_prefill_kv_pages(ctx, q, pages, hkv, tab, 5000, cuq, 64, seq_lens=ln)
        for gr, o, ls in made:
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(ls, wl)
    T.tq_check_device(ctx)


def test_prefill_writes_only_its_outputs():
    d, g, hkv = 64, 3, 2
    rng = np.random.default_rng(17)
    ctx = make_ctx(d)
    q_lens, kv_lens, cache, table, cu, q = simple(rng, "f16", d, g, hkv, [(20, 5000), (3, 44)])
    keep = [t.clone() for t in cache[:2]]
    need = T.tq_prefill_kv_pages_workspace_bytes(ctx, 23, 2, hkv * g, hkv, 5000, 20)
    sizes = [23 * hkv * g * d * 2, 23 * hkv * g * 4, need]
    bufs = [torch.full((8192 + s,), 0xC3, dtype=torch.uint8, device=DEV) for s in sizes]
    mid = [b[4096:4096 + s] for b, s in zip(bufs, sizes)]
    out, lse = mid[0].view(torch.float16).view(23, hkv * g, d), mid[1].view(torch.float32).view(23, hkv * g)
    T.tq_prefill_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 5000, up(cu), 20,
                          seq_lens=up(kv_lens.astype(np.int32)), out=out, lse=lse, workspace=mid[2])
    T.tq_check_device(ctx)
    check(cache, table, q_lens, kv_lens, cu, q, out, lse, 16, False, hkv, 0, "f16")
    for b, s in zip(bufs, sizes):
        assert (b[:4096] == 0xC3).all() and (b[4096 + s:] == 0xC3).all()
    assert all(torch.equal(a, b) for a, b in zip(cache[:2], keep))


def test_prefill_refusals():
    d, hkv, g = 128, 2, 4
    ctx = make_ctx(d)
    cache = P.make_cache("bf16", 4, 16, hkv, d, False)
    pages = T.KVPages(*cache)
    q = torch.zeros((5, hkv * g, d), dtype=torch.bfloat16, device=DEV)
    table, cu = up(np.zeros((1, 400), np.int32)), up(np.array([0, 5], np.int32))

    def status(**kw):
        a = dict(q=q, table=table, max_len=32, cu=cu, max_q=5, ws=None, kw={})
        a.update(kw)
        try:
            T.tq_prefill_kv_pages(ctx, a["q"], pages, hkv, a["table"], a["max_len"], a["cu"], a["max_q"],
                                  workspace=a["ws"], **a["kw"])
        except T.TQError as e:
            return e.status
        except ValueError:
            return "value"
        return 0
    cache[0].zero_(), cache[1].zero_()
    assert status() == 0
    assert status(max_len=6401) == _lib.TQ_EINVAL
    assert status(max_q=-1) == _lib.TQ_EINVAL
    assert status(max_len=6400, ws=torch.zeros(64, dtype=torch.uint8, device=DEV)) == _lib.TQ_EINVAL  # needs one
    assert status(kw=dict(window=-3)) == _lib.TQ_EINVAL
    assert status(kw=dict(softmax_scale=float("inf"))) == _lib.TQ_EINVAL
    assert status(q=q.half()) == "value"
    assert status(cu=cu.long()) == "value"
    assert status(table=table.repeat(2, 1)) == "value"
    assert status(kw=dict(out=torch.zeros((5, 8, d), device=DEV))) == "value"          # fp32 out
    assert status(max_q=0) == 0
    T.tq_check_device(ctx)
