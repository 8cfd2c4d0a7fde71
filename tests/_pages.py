"""Plain 64-bit restatement of the page-cache operators for the tests (numpy, on the CPU), and the
construction of caches with chosen layouts. Shares no code with the library."""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SENTINEL = 0x5A
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "mxfp4": torch.bfloat16}
# half a step relative to the value (torch.finfo(t).eps / 2: bf16 has 7 stored mantissa bits, so its
# step is 2^-7 of the power of two below the value), and half the smallest step
EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "mxfp4": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "mxfp4": 2.0 ** -134, "f32": 2.0 ** -150}


def f64(t):
    return t.detach().cpu().double().numpy()


def rotate(x, table, pos, interleaved, dtype=np.float64):
    """The position rotation of x [n, heads, d] with `table` [n_pos, rot] (cosines, then sines)."""
    x = x.astype(dtype).copy()
    half = table.shape[1] // 2
    c, s = (table[pos][:, None, i * half:(i + 1) * half].astype(dtype) for i in (0, 1))
    i0 = np.arange(half) * 2 if interleaved else np.arange(half)
    i1 = i0 + (1 if interleaved else half)
    a, b = x[..., i0], x[..., i1]
    x[..., i0], x[..., i1] = a * c - b * s, b * c + a * s
    return x


def rotate_abs(x, table, pos, interleaved):
    """|a cos| + |b sin| and |b cos| + |a sin| in the places of the rotated pairs."""
    x = np.abs(x.astype(np.float64))
    half = table.shape[1] // 2
    c, s = (np.abs(table[pos][:, None, i * half:(i + 1) * half].astype(np.float64)) for i in (0, 1))
    i0 = np.arange(half) * 2 if interleaved else np.arange(half)
    i1 = i0 + (1 if interleaved else half)
    a, b = x[..., i0], x[..., i1]
    x[..., i0], x[..., i1] = a * c + b * s, b * c + a * s
    return x


def quantise(x):
    """MXFP4 of float32 values [..., d]: (codes uint8 [..., d/2], scales uint8 [..., d/32])."""
    x = x.astype(np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    finite = np.isfinite(b).all(-1)
    b = np.where(finite[..., None], b, 0.0)
    amax = np.abs(b).max(-1)
    e = np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1 - 2
    e = np.where(amax > 0, np.maximum(e, -126), -126)
    y = np.abs(b) * 2.0 ** -e[..., None].astype(np.float64)
    mid = (GRID[:-1] + GRID[1:]) / 2
    code = np.zeros(y.shape, np.uint8)
    for i, m in enumerate(mid):                     # a tie goes to the even code
        code += ((y > m) | ((y == m) & (i % 2 == 1))).astype(np.uint8)
    code |= np.signbit(b).astype(np.uint8) << 3
    code = np.where(finite[..., None], code, 0).astype(np.uint8).reshape(x.shape)
    scales = np.where(finite, e + 127, 255).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def dequantise(codes, scales):
    """float64 values of MXFP4 codes [..., d/2] and scales [..., d/32]."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    v = GRID[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    f = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(f, 32, axis=-1)


def attend(q, k, v, pos, window, scale):
    """softmax(q k^T scale) v in float64: q [rows, g, d] at positions pos [rows], k, v [n, d].
    Tokens after a row's position, or `window` or more before it, are left out of the sums."""
    rows, g, d = q.shape
    out, lse = np.zeros((rows, g, d)), np.full((rows, g), -np.inf)
    for i in range(rows):
        lo = max(0, pos[i] - window + 1) if window else 0
        hi = max(lo, pos[i] + 1)
        if hi == lo:
            continue
        x = q[i] @ k[lo:hi].T * scale
        m = x.max(-1, keepdims=True)
        with np.errstate(invalid="ignore"):
            e = np.exp(x - m)
            out[i] = e @ v[lo:hi] / e.sum(-1, keepdims=True)
            lse[i] = (m + np.log(e.sum(-1, keepdims=True)))[:, 0]
    return out, lse


def make_tensor(shape, dtype, order, device, fill=SENTINEL):
    """A tensor [n_pages, page_size(, hkv), width] laid out in `order` ("nhd": as the shape says,
    "hnd": heads outside tokens, "gap": nhd with a record's gap after every token), every byte `fill`."""
    if len(shape) == 3 or order == "nhd":
        t = torch.empty(shape, dtype=dtype, device=device)
        t.view(torch.uint8).fill_(fill)
        return t
    p, s, h, w = shape
    if order == "hnd":
        t = torch.empty((p, h, s, w), dtype=dtype, device=device)
        t.view(torch.uint8).fill_(fill)
        return t.transpose(1, 2)
    t = torch.empty((p, s, h + 1, w), dtype=dtype, device=device)
    t.view(torch.uint8).fill_(fill)
    return t[:, :, :h]


def make_cache(fmt, n_pages, page, hkv, d, per_head, order="nhd", device="cuda:0"):
    """(k, v, k_scales, v_scales) filled with SENTINEL bytes."""
    lead = (n_pages, page) if per_head else (n_pages, page, hkv)
    if fmt == "mxfp4":
        return tuple(make_tensor(lead + (w,), torch.uint8, order, device) for w in (d // 2, d // 2, d // 32, d // 32))
    return tuple(make_tensor(lead + (d,), TORCH[fmt], order, device) for _ in range(2)) + (None, None)


def slots_for(rng, n, n_pages, page, hkv, per_head):
    """Distinct random cache rows for n tokens: [n], or [n, hkv] with per-head pages."""
    m = n * hkv if per_head else n
    s = rng.permutation(n_pages * page)[:m].astype(np.int64)
    return s.reshape(n, hkv) if per_head else s


def gather(cache, slot, hkv, which):
    """Raw records of cache rows `slot`, [n, hkv, width] on the CPU (which: 0 k, 1 v, 2/3 scales)."""
    t = cache[which].cpu()
    if t.dim() == 3:
        return t.reshape(-1, t.shape[-1])[torch.from_numpy(slot)]
    return t.reshape(-1, hkv, t.shape[-1])[torch.from_numpy(slot)]
