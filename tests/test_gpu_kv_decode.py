"""GPU tests of tq_decode_kv_pages (through the C ABI) against softmax attention in 64 bits.

Tolerances. The products q k are exact in fp32; a score sums them in d / 16 tensor-core steps,
each off by at most 2^-23 of the magnitudes it adds (two steps' worth is granted), and its
exponential adds 2^-21. P's two 16-bit terms leave 2^-17 (bf16) of a probability, the sums over n
tokens a 2^-23 per step of 16 tokens and per merge. A relative error e of every probability moves
the output by at most 2 e max|v|. The output's own rounding is half a step of its type."""
import ctypes

import numpy as np
import pytest

import _pages as P
from test_gpu_kv_pages import make_ctx, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import kv_cache_vector_05_b200 as T  # noqa: E402
from kv_cache_vector_05_b200 import _lib  # noqa: E402

DEV = "cuda:0"


def random_cache(rng, fmt, n_pages, page, hkv, d, per_head, order="nhd", k_exp=(124, 127), v_exp=(120, 127)):
    cache = P.make_cache(fmt, n_pages, page, hkv, d, per_head, order)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(rng.integers(1 << 31)))
    for i, t in enumerate(cache):
        if t is None:
            continue
        if fmt != "mxfp4":
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        elif i < 2:
            t.copy_(torch.randint(0, 256, t.shape, generator=gen, device=DEV, dtype=torch.uint8))
        else:
            lo, hi = k_exp if i == 2 else v_exp
            t.copy_(torch.randint(lo, hi, t.shape, generator=gen, device=DEV, dtype=torch.uint8))
    return cache


def block_tables(rng, lens, page, hkv, per_head, max_pages, n_pages):
    """Distinct pages for every used block; entries of unused blocks are out of range (never read)."""
    lead = (len(lens), hkv) if per_head else (len(lens),)
    table = np.full(lead + (max_pages,), 1 << 30, np.int32)
    order, at = rng.permutation(n_pages), 0
    for idx in np.ndindex(*lead):
        used = -(-int(lens[idx[0]]) // page)
        table[idx][:used] = order[at:at + used]
        at += used
    assert at <= n_pages
    return table


def tokens(cache, table, b, h, n, page, per_head, hkv, which):
    """float64 vectors of (sequence b, KV head h)'s tokens 0..n-1."""
    t = np.arange(n)
    row = table[b, h] if per_head else table[b]
    slot = row[t // page].astype(np.int64) * page + t % page

    def pick(w):
        x = cache[w]
        x = x.reshape(-1, x.shape[-1]) if x.dim() == 3 else x.reshape((-1,) + tuple(x.shape[2:]))[:, h]
        return x[torch.from_numpy(slot).to(x.device)]
    x = pick(which)
    return P.dequantise(x.cpu().numpy(), pick(which + 2).cpu().numpy()) if cache[2] is not None else P.f64(x)


def tolerance(q, k, v, scale, d, n, fmt, out_fmt, want, lse):
    """(out, lse) tolerances of one row group: q [g, d], k, v [n, d]."""
    size = np.abs(q) @ np.abs(k).T                                   # [g, n]
    delta = scale * (d / 8 + 4) * 2.0 ** -23 * size.max(-1)
    steps = (n / 16 + 40) * 2.0 ** -23
    rel = 2 * (delta + 2.0 ** -17 + 2.0 ** -21 + steps)
    vmax = np.abs(v).max(0)
    # f16 probabilities below 2^-38 of the largest vanish
    tol = rel[:, None] * vmax + n * 2.0 ** -37 * vmax + P.EPS[out_fmt] * np.abs(want) + P.TINY[out_fmt]
    return tol, delta + steps + 2.0 ** -20 + np.abs(lse) * 2.0 ** -21


def check(cache, table, lens, q, out, lse, page, per_head, hkv, window, fmt, out_fmt, scale=None):
    batch, hq, d = q.shape
    g, scale = hq // hkv, scale or d ** -0.5
    q64, out, lse = P.f64(q), P.f64(out), P.f64(lse)
    for b in range(batch):
        n = int(lens[b])
        for h in range(hkv):
            rows = slice(h * g, (h + 1) * g)
            if n == 0:
                assert (out[b, rows] == 0).all() and np.isneginf(lse[b, rows]).all()
                continue
            lo = max(0, n - window) if window else 0
            k, v = (tokens(cache, table, b, h, n, page, per_head, hkv, w)[lo:] for w in (0, 1))
            want, wl = P.attend(q64[b, rows][None], k, v, np.array([n - lo - 1]), 0, scale)
            tol, tl = tolerance(q64[b, rows], k, v, scale, d, n - lo, fmt, out_fmt, want[0], wl[0])
            assert (np.abs(out[b, rows] - want[0]) <= tol).all(), (b, h, n, np.abs(out[b, rows] - want[0]).max())
            assert (np.abs(lse[b, rows] - wl[0]) <= tl).all(), (b, h, n, np.abs(lse[b, rows] - wl[0]).max())


EDGE = [0, 1, 15, 16, 17, 33, 0, 250]
CASES = [
    # fmt, d, g, hkv, lens, page, per_head, order, window, out
    ("bf16", 128, 4, 2, EDGE, 16, False, "nhd", 0, "f32"),
    ("bf16", 128, 8, 1, [4096], 16, False, "nhd", 0, "bf16"),
    ("bf16", 128, 1, 3, EDGE + [1000], 7, False, "gap", 0, "f32"),
    ("bf16", 128, 5, 2, EDGE, 1, False, "hnd", 0, "f32"),
    ("bf16", 64, 4, 4, EDGE + [3000], 48, True, "nhd", 0, "bf16"),
    ("bf16", 64, 7, 1, [77] * 40, 16, False, "hnd", 20, "f32"),
    ("bf16", 256, 3, 2, EDGE, 24, False, "nhd", 0, "f32"),
    ("bf16", 256, 8, 1, EDGE + [2049], 512, True, "nhd", 33, "bf16"),
    ("bf16", 128, 12, 2, EDGE, 16, False, "nhd", 0, "f32"),            # two blocks of 6 heads
    ("bf16", 64, 17, 1, EDGE + [513], 32, False, "nhd", 0, "f32"),     # three blocks: 6, 6, 5
    ("f16", 128, 4, 2, EDGE + [700], 16, False, "nhd", 5, "f16"),
    ("f16", 128, 6, 1, [5000, 1, 0, 33], 64, True, "nhd", 0, "f32"),
    ("f16", 64, 2, 2, EDGE, 3, False, "gap", 0, "f32"),
    ("f16", 256, 8, 1, EDGE, 16, False, "nhd", 1, "f16"),
    ("mxfp4", 128, 4, 2, EDGE + [999], 16, False, "nhd", 0, "f32"),
    ("mxfp4", 128, 6, 4, [12000], 512, True, "nhd", 0, "f32"),
    ("mxfp4", 128, 8, 1, EDGE, 5, False, "gap", 18, "bf16"),
    ("mxfp4", 64, 3, 2, EDGE + [600], 16, False, "hnd", 0, "f32"),
    ("mxfp4", 64, 8, 1, EDGE, 9, True, "nhd", 0, "f32"),
    ("mxfp4", 256, 2, 2, EDGE + [400], 32, False, "nhd", 0, "f32"),
    ("mxfp4", 256, 5, 1, EDGE, 33, False, "nhd", 40, "bf16"),
    ("bf16", 128, 2, 8, [100] * 130 + [0] * 20 + [999] * 7, 16, False, "nhd", 0, "f32"),  # units inside warps
    ("bf16", 64, 1, 1, list(range(0, 700)), 16, False, "nhd", 0, "f32"),                   # batch above a block
    # long sequences: tiles split over the whole grid
    ("bf16", 64, 17, 1, [0, 9000, 33, 1], 24, False, "nhd", 0, "f32"),
    ("mxfp4", 64, 12, 2, [6000, 5, 0], 7, True, "nhd", 5001, "bf16"),
    ("mxfp4", 256, 4, 1, [7000, 640], 32, False, "hnd", 0, "f32"),
    ("f16", 256, 5, 1, [4100, 17, 2500], 16, False, "gap", 0, "f16"),
    ("bf16", 256, 9, 1, [5000, 1], 33, True, "nhd", 4500, "f32"),
    # one to eight CTAs per unit
    ("bf16", 128, 4, 8, [1999, 0, 3], 16, False, "nhd", 0, "f32"),
    ("bf16", 128, 4, 8, [400] * 9 + [0, 1, 17, 1000], 16, False, "nhd", 0, "bf16"),
    ("f16", 64, 8, 16, [500, 512, 1, 0, 77, 300, 16, 15], 8, False, "nhd", 100, "f32"),
]


@pytest.mark.parametrize("fmt,d,g,hkv,lens,page,per_head,order,window,out_fmt", CASES)
def test_decode(fmt, d, g, hkv, lens, page, per_head, order, window, out_fmt):
    rng = np.random.default_rng(len(lens) * d + g)
    ctx = make_ctx(d)
    lens = np.array(lens)
    max_len = int(lens.max()) + 3
    max_pages = -(-max_len // page)
    n_pages = int((-(-lens // page)).sum()) * (hkv if per_head else 1) + 1
    cache = random_cache(rng, fmt, n_pages, page, hkv, d, per_head, order)
    table = block_tables(rng, lens, page, hkv, per_head, max_pages, n_pages)
    if fmt != "mxfp4":                                  # slots outside the attended tokens hold anything
        bad = [float("nan"), float("inf"), float("-inf")]
        for b, n in enumerate(lens):
            for h in range(hkv if per_head else 1):
                row = table[b, h] if per_head else table[b]
                dead = list(range(n, -(-n // page) * page)) + list(range(0, max(0, n - window) if window else 0))
                for i, t in enumerate(dead):
                    for x in cache[:2]:
                        x[int(row[t // page]), t % page] = bad[i % 3]
    else:
        for b, n in enumerate(lens):
            for h in range(hkv if per_head else 1):
                row = table[b, h] if per_head else table[b]
                for t in range(n, -(-n // page) * page):
                    for x in cache[2:]:
                        x[int(row[t // page]), t % page] = 255
    dt = P.TORCH[fmt]
    qq = torch.randn((len(lens), hkv * g + 1, d), device=DEV).to(dt)
    q = qq[:, :hkv * g]                                  # strided rows
    out, lse = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), max_len,
                                    seq_lens=up(lens.astype(np.int32)), window=window,
                                    out_dtype=torch.float32 if out_fmt == "f32" else dt)
    T.tq_check_device(ctx)
    check(cache, table, lens, q, out, lse, page, per_head, hkv, window, fmt, out_fmt)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "mxfp4"])
def test_decode_large_and_peaked_logits(fmt):
    """Logits up to several hundred (a few tokens carry everything), one far above all the others
    at the start, in the middle or at the end, and rising ones that move the maximum every tile."""
    d, hkv, g, n, page = 128, 2, 4, 3000, 16
    rng = np.random.default_rng(3)
    ctx = make_ctx(d)
    cache = random_cache(rng, fmt, 2 * (-(-n // page)) + 200, page, hkv, d, False)
    lens = np.array([n, n - 5])
    table = block_tables(rng, lens, page, hkv, False, -(-n // page), cache[0].shape[0])
    q = (torch.randn((2, hkv * g, d), device=DEV) * 8).to(P.TORCH[fmt])
    if fmt != "mxfp4":
        for b, t in ((0, 0), (0, 1500), (1, 2990)):
            p, o = int(table[b, t // page]), t % page
            cache[0][p, o] = q[b, :2] / 4
    for scale in (0.0, 1e-3, 2.0):
        out, lse = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), n,
                                        seq_lens=up(lens.astype(np.int32)), softmax_scale=scale)
        check(cache, table, lens, q, out, lse, page, False, hkv, 0, fmt, "f32", scale or None)
    if fmt != "mxfp4":
        ramp = torch.linspace(0, 1, n, device=DEV)
        for t in range(n):
            cache[0][int(table[0, t // page]), t % page] = (q[0, :2].float() * ramp[t]).to(P.TORCH[fmt])
        out, lse = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), n,
                                        seq_lens=up(lens.astype(np.int32)))
        check(cache, table, lens, q, out, lse, page, False, hkv, 0, fmt, "f32")


def test_decode_mxfp4_full_scale_range():
    """Value blocks of every magnitude (each sequence one), keys of small and large scale, and
    queries far from 1: the block scales never meet a 16-bit type's range."""
    d, hkv, g, page = 128, 1, 4, 16
    rng = np.random.default_rng(4)
    ctx = make_ctx(d)
    exps = [1, 2, 20, 60, 100, 127, 140, 141, 142, 143, 144, 160, 200, 245]
    lens = np.full(len(exps), 70)
    cache = random_cache(rng, "mxfp4", 5 * len(exps), page, hkv, d, False)
    table = block_tables(rng, lens, page, hkv, False, 5, 5 * len(exps))
    q = torch.randn((len(exps), g, d), device=DEV).to(torch.bfloat16)
    for b, e in enumerate(exps):
        rows = up(table[b].astype(np.int64))
        cache[3][rows] = torch.randint(e, e + 2, (5, page, hkv, 4), device=DEV, dtype=torch.uint8)
        ke = 30 + 14 * b                                 # keys of 2^(ke - 127), queries to match
        cache[2][rows] = ke
        q[b] = (q[b].float() * 2.0 ** (126 - ke)).to(torch.bfloat16)
    cache[3][int(table[8, 1]), 3] = 1                    # a tiny block among large ones, and the reverse
    cache[3][int(table[2, 1]), 3] = 150
    out, lse = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 80, seq_lens=up(lens.astype(np.int32)))
    check(cache, table, lens, q, out, lse, page, False, hkv, 0, "mxfp4", "f32")
    # a block marked not finite reaches the rows that attend to it, and only those
    cache[3][int(table[0, 0]), 5, 0, 1] = 255
    cache[0][int(table[1, 2]), 1] = 0
    cache[2][int(table[1, 2]), 1, 0, 2] = 255
    out2, lse2 = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 80, seq_lens=up(lens.astype(np.int32)))
    assert torch.isnan(out2[0, :, 32:64]).all()
    # the other blocks of that row pass through the tile's other products: each is off by at most the
    # 2^-17 of P's terms, twice max|v| = 6 x 2^(2 - 127)
    assert (out2[0, :, :32] - out[0, :, :32]).abs().max() <= 2 * 2 * 2.0 ** -17 * 6 * 2.0 ** -125
    assert torch.isnan(out2[1]).all() and torch.isnan(lse2[1]).all()
    assert torch.equal(out2[2:], out[2:]) and torch.equal(lse2[2:], lse[2:])


def test_decode_nonfinite_inputs_stay_in_their_rows():
    d, hkv, g, page, n = 64, 2, 2, 16, 200
    rng = np.random.default_rng(5)
    ctx = make_ctx(d)
    lens = np.array([n, n, n])
    cache = random_cache(rng, "bf16", 60, page, hkv, d, False)
    table = block_tables(rng, lens, page, hkv, False, 13, 60)
    q = torch.randn((3, hkv * g, d), device=DEV).to(torch.bfloat16)
    args = dict(seq_lens=up(lens.astype(np.int32)))
    ref, rl = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), n, **args)
    q2 = q.clone()
    q2[0, 1, 3] = float("nan")
    cache[1][int(table[1, 3]), 4, 0, 7] = float("inf")       # a value of KV head 0
    cache[0][int(table[2, 3]), 4, 1, 7] = float("nan")       # a key of KV head 1
    out, lse = T.tq_decode_kv_pages(ctx, q2, T.KVPages(*cache), hkv, up(table), n, **args)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 1] = True
    bad[1, :g, 7] = True
    bad[2, g:] = True
    assert torch.equal(torch.isfinite(out), ~bad) and torch.equal(out[~bad], ref[~bad])
    assert torch.isposinf(out[1, :g, 7]).all() and torch.isnan(lse[2, g:]).all()


def test_decode_bad_page_is_reported_and_lengths_are_clamped():
    d, hkv, g, page = 128, 2, 4, 16
    rng = np.random.default_rng(6)
    ctx = make_ctx(d)
    lens = np.array([100, 50])
    cache = random_cache(rng, "bf16", 30, page, hkv, d, False)
    table = block_tables(rng, lens, page, hkv, False, 7, 30)
    q = torch.randn((2, hkv * g, d), device=DEV).to(torch.bfloat16)
    ref, _ = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 100, seq_lens=up(lens.astype(np.int32)))
    big, _ = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 100,
                                  seq_lens=up(np.array([1 << 30, 50], np.int32)))
    assert torch.equal(ref, big)
    neg, nl = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 100,
                                   seq_lens=up(np.array([100, -7], np.int32)))
    none, _ = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 100,
                                   seq_lens=up(np.array([100, 0], np.int32)))   # the split follows all lengths
    assert torch.equal(none, neg) and (neg[1] == 0).all() and torch.isneginf(nl[1]).all()
    T.tq_check_device(ctx)
    for page_id in (30, -1, 2 ** 31 - 1):
        t2, t3 = table.copy(), table.copy()
        t2[1, 2], t3[1, 2] = page_id, 0
        out, _ = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(t2), 100, seq_lens=up(lens.astype(np.int32)))
        with pytest.raises(T.TQError):
            T.tq_check_device(ctx)
        want, _ = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(t3), 100,
                                       seq_lens=up(lens.astype(np.int32)))
        assert torch.equal(out, want)


@pytest.mark.parametrize("fmt,page,window", [("mxfp4", 16, 20), ("mxfp4", 16, 1), ("mxfp4", 48, 70), ("mxfp4", 5, 33),
                                             ("bf16", 16, 17), ("f16", 24, 30)])
def test_decode_window_reads_no_entry_before_it(fmt, page, window):
    """Pages that lie wholly before the window may be gone: their table entries are never read."""
    d, hkv, g = 64, 1, 2
    rng = np.random.default_rng(10)
    ctx = make_ctx(d)
    lens = np.arange(1, 140)
    cache = random_cache(rng, fmt, int((-(-lens // page)).sum()), page, hkv, d, False)
    table = block_tables(rng, lens, page, hkv, False, -(-140 // page), cache[0].shape[0])
    gone = table.copy()
    for b, n in enumerate(lens):
        gone[b, :max(0, n - window) // page] = -1
    q = torch.randn((len(lens), hkv * g, d), device=DEV).to(P.TORCH[fmt])
    out, lse = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(gone), 139, seq_lens=up(lens.astype(np.int32)),
                                    window=window)
    T.tq_check_device(ctx)
    check(cache, table, lens, q, out, lse, page, False, hkv, window, fmt, "f32")


def test_decode_without_lengths_and_max_len_zero():
    d, hkv, g, page = 128, 1, 2, 16
    rng = np.random.default_rng(7)
    ctx = make_ctx(d)
    cache = random_cache(rng, "f16", 30, page, hkv, d, False)
    lens = np.array([90, 90])
    table = block_tables(rng, lens, page, hkv, False, 6, 30)
    q = torch.randn((2, g, d), device=DEV).half()
    out, lse = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 90)
    check(cache, table, lens, q, out, lse, page, False, hkv, 0, "f16", "f32")
    out, lse = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 0)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = T.tq_decode_kv_pages(ctx, q[:0], T.KVPages(*cache), hkv, up(table)[:0], 90)
    assert out.shape == (0, g, d)
    T.tq_check_device(ctx)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_decode_past_32_bit_offsets(fmt):
    """Pages more than 2^32 bytes apart, in one sequence."""
    d, hkv, g, page = 128, 2, 4, 16
    ctx = make_ctx(d)
    big = torch.zeros((1 << 32) + (1 << 20), dtype=torch.uint8, device=DEV)
    if fmt == "bf16":
        f = big.view(torch.bfloat16)
        st, off = (1 << 31, hkv * d, d, 1), 1 << 16
        cache = (f.as_strided((2, page, hkv, d), st), f.as_strided((2, page, hkv, d), st, off), None, None)
        for t in cache[:2]:
            t.copy_(torch.randn(t.shape, device=DEV))
    else:
        cache = tuple(big.as_strided((2, page, hkv, w), (1 << 32, hkv * w, w, 1), i << 16)
                      for i, w in enumerate((64, 64, 4, 4)))
        for i, t in enumerate(cache):
            t.copy_(torch.randint(0, 256, t.shape, device=DEV) if i < 2 else torch.randint(124, 128, t.shape, device=DEV))
    table, lens = np.array([[1, 0]], np.int32), np.array([30])
    q = torch.randn((1, hkv * g, d), device=DEV).to(torch.bfloat16)
    out, lse = T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 32, seq_lens=up(lens.astype(np.int32)))
    T.tq_check_device(ctx)
    small = tuple(None if t is None else t.contiguous() for t in cache)
    check(small, table, lens, q, out, lse, page, False, hkv, 0, fmt, "f32")


@pytest.mark.parametrize("cut", [1, 10])     # tiles split over the grid; a cluster per unit
def test_decode_repeats_on_streams_and_in_graphs(cut):
    """The same bits from every run, on another stream, captured and replayed with other lengths
    and queries, and from two graphs that share a workspace but run one after the other."""
    d, hkv, g, page, batch = 128, 2, 4, 16, 5
    rng = np.random.default_rng(8)
    ctx = make_ctx(d)
    top = 3000 // cut
    lens = np.array([top, 17, 0, 801 // cut, 1600 // cut])
    cache = random_cache(rng, "bf16", 400, page, hkv, d, False)
    table = up(block_tables(rng, lens, page, hkv, False, 188, 400))
    pages = T.KVPages(*cache)
    q = torch.randn((batch, hkv * g, d), device=DEV).to(torch.bfloat16)
    ln = up(lens.astype(np.int32))
    ref, rl = T.tq_decode_kv_pages(ctx, q, pages, hkv, table, top, seq_lens=ln)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            out, lse = T.tq_decode_kv_pages(ctx, q, pages, hkv, table, top, seq_lens=ln)
        side.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, rl)
    out, lse = T.tq_decode_kv_pages(ctx, q, pages, hkv, table, top, seq_lens=ln, stream=side)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    ws = torch.empty(T.tq_decode_kv_pages_workspace_bytes(ctx, batch, hkv * g, hkv), dtype=torch.uint8, device=DEV)
    ws.fill_(255)
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        o, ls = torch.empty_like(ref), torch.empty_like(rl)
        with torch.cuda.graph(gr):
            T.tq_decode_kv_pages(ctx, q, pages, hkv, table, top, seq_lens=ln, out=o, lse=ls, workspace=ws)
        graphs.append(gr)
        outs.append((o, ls))
    for i in range(4):
        q.normal_()
        ln.copy_(up(np.minimum(lens, [top - 7 * i, 17, i, 800, 1000 * i // 2]).astype(np.int32)))
        want, wl = T.tq_decode_kv_pages(ctx, q, pages, hkv, table, top, seq_lens=ln)
        for gr, (o, ls) in zip(graphs, outs):
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(ls, wl)


def test_decode_writes_only_its_outputs():
    """Guard bytes around out, lse and an exactly sized workspace stay as they were."""
    d, hkv, g, page = 128, 2, 5, 16
    rng = np.random.default_rng(9)
    ctx = make_ctx(d)
    lens = np.array([0, 1, 700, 2500])
    cache = random_cache(rng, "bf16", 210, page, hkv, d, False)
    keep = [t.clone() for t in cache[:2]]
    table = block_tables(rng, lens, page, hkv, False, 160, 210)
    q = torch.randn((4, hkv * g, d), device=DEV).to(torch.bfloat16)
    need = T.tq_decode_kv_pages_workspace_bytes(ctx, 4, hkv * g, hkv)
    sizes = [4 * hkv * g * d * 2, 4 * hkv * g * 4, need]
    bufs = [torch.full((4096 + s + 4096,), 0xC3, dtype=torch.uint8, device=DEV) for s in sizes]
    mid = [b[4096:4096 + s] for b, s in zip(bufs, sizes)]
    out, lse = mid[0].view(torch.bfloat16).view(4, hkv * g, d), mid[1].view(torch.float32).view(4, hkv * g)
    T.tq_decode_kv_pages(ctx, q, T.KVPages(*cache), hkv, up(table), 2560, seq_lens=up(lens.astype(np.int32)), out=out,
                         lse=lse, workspace=mid[2])
    T.tq_check_device(ctx)
    check(cache, table, lens, q, out, lse, page, False, hkv, 0, "bf16", "bf16")
    for b, s in zip(bufs, sizes):
        assert (b[:4096] == 0xC3).all() and (b[4096 + s:] == 0xC3).all()
    assert all(torch.equal(a, b) for a, b in zip(cache[:2], keep))


def test_decode_refusals():
    d, hkv, g = 128, 2, 4
    ctx = make_ctx(d)
    cache = P.make_cache("bf16", 4, 16, hkv, d, False, "nhd")
    pages = T.KVPages(*cache)
    q = torch.zeros((2, hkv * g, d), dtype=torch.bfloat16, device=DEV)
    table = up(np.zeros((2, 2), np.int32))

    def status(**kw):
        a = dict(q=q, table=table, max_len=32, ws=None, kw={})
        a.update(kw)
        try:
            T.tq_decode_kv_pages(ctx, a["q"], pages, hkv, a["table"], a["max_len"], workspace=a["ws"], **a["kw"])
        except T.TQError as e:
            return e.status
        except ValueError:
            return "value"
        return 0
    assert status() == 0
    assert status(max_len=33) == _lib.TQ_EINVAL                                     # beyond the block table
    assert status(max_len=-1) == _lib.TQ_EINVAL
    assert status(kw=dict(window=-1)) == _lib.TQ_EINVAL
    assert status(kw=dict(softmax_scale=float("nan"))) == _lib.TQ_EINVAL
    assert status(kw=dict(softmax_scale=-1.0)) == _lib.TQ_EINVAL
    assert status(q=q[:, :7].contiguous()) == _lib.TQ_EINVAL                        # 7 heads over 2
    assert status(kw=dict(out_dtype=torch.float16)) == _lib.TQ_EUNSUPPORTED
    assert status(ws=torch.zeros(64, dtype=torch.uint8, device=DEV)) == _lib.TQ_EINVAL
    assert status(q=q.half()) == "value" and status(q=q.float()) == "value"
    assert status(table=table.long()) == "value"
    assert status(kw=dict(seq_lens=up(np.zeros(3, np.int32)))) == "value"
    assert status(q=q.cpu()) == "value"
    T.tq_check_device(ctx)
    st = pages.struct(ctx, hkv)
    need = T.tq_decode_kv_pages_workspace_bytes(ctx, 2, 8, hkv)
    ws = torch.zeros(need + 16, dtype=torch.uint8, device=DEV)
    out = torch.zeros((2, 8, d), device=DEV)

    def raw(qs=8 * d, o=out.data_ptr(), w=ws.data_ptr(), n=need):
        return _lib.lib.tq_decode_kv_pages(ctx.handle, st, q.data_ptr(), _lib.TQ_BF16, qs, 2, 8, table.data_ptr(), 2,
                                           None, 32, 0, 0.0, o, _lib.TQ_F32, None, w, n,
                                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert raw() == 0
    assert raw(qs=8 * d - 8) == raw(qs=8 * d + 4) == _lib.TQ_EINVAL
    assert raw(o=out.data_ptr() + 4) == raw(w=ws.data_ptr() + 8) == raw(n=need - 1) == raw(w=None) == _lib.TQ_EINVAL
    assert T.tq_decode_kv_pages_workspace_bytes(ctx, 2, 7, 2) == 0
