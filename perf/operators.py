"""Cases of the page-cache operators: a paged key/value cache of 16-bit or MXFP4 records, filled
with rotated keys, read back, and attended by one new token or by a chunk of new tokens.

A cache holds pages of ``page_size`` tokens. Either a page holds every KV head of its tokens
(``[n_pages, page_size, hkv, width]``, block table ``[batch, max_pages]``) or it belongs to one
(sequence, KV head) pair (``[n_pages, page_size, width]``, block table ``[batch, hkv, max_pages]``),
the layout of the packed caches. 16-bit caches hold the vectors; MXFP4 caches hold two e2m1 codes a
byte (coordinate j in nibble j % 2 of byte j // 2) and one E8M0 scale byte per 32 coordinates.

``own`` False computes every operator in its plain form; True calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "mxfp4": torch.bfloat16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)          # e2m1 magnitudes


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch of 32 sequences: 32 new tokens, latency counts
        dict(name="append_step_b32", op="append", fmt="bf16", n=32, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, page=16, per_head=False, fused=True, spare=512),
        # the prompt of a Qwen2.5-3B-shaped layer (16 query heads, 2 KV heads), ragged length
        dict(name="append_prompt_8k", op="append", fmt="bf16", n=8111, hq=16, hkv=2, d=128, rot=128,
             interleaved=False, page=16, per_head=False, fused=True, spare=40),
        # prompts of several sequences quantised on the way into pages of one KV head each
        dict(name="append_mxfp4_16k", op="append", fmt="mxfp4", n=16384, hq=32, hkv=8, d=128, rot=64,
             interleaved=True, page=512, per_head=True, fused=True, spare=3),
        # a recent window taken out of small odd pages, to be compressed
        dict(name="read_window_f16", op="read", fmt="f16", n=513, hkv=8, d=64, page=24, per_head=False, spare=7),
        # a long prefix read out of an MXFP4 cache
        dict(name="read_mxfp4_32k", op="read", fmt="mxfp4", n=32768, hkv=8, d=128, page=512, per_head=True, spare=3),
        # one sequence, one KV head, 8 query heads, 4096 tokens: the smallest attention call
        dict(name="decode_b1_4k", op="decode", fmt="bf16", batch=1, hq=8, hkv=1, d=128, max_len=4096,
             min_len=4096, page=16, per_head=False, window=0, out="f32", zero=0),
        # Llama-8B-shaped layer: 32 sequences of 32768 tokens
        dict(name="decode_b32_32k", op="decode", fmt="bf16", batch=32, hq=32, hkv=8, d=128, max_len=32768,
             min_len=32768, page=16, per_head=False, window=0, out="bf16", zero=0),
        # a batch of very different lengths, some slots empty, small odd pages, sliding window
        dict(name="decode_ragged_f16", op="decode", fmt="f16", batch=48, hq=24, hkv=4, d=64, max_len=5003,
             min_len=1, page=24, per_head=False, window=4001, out="f16", zero=5),
        # one sequence of 1,048,576 tokens, 4 KV heads, 24 query heads, MXFP4 cache
        dict(name="decode_mxfp4_1m", op="decode", fmt="mxfp4", batch=1, hq=24, hkv=4, d=128, max_len=1 << 20,
             min_len=1 << 20, page=512, per_head=True, window=0, out="f32", zero=0),
        # short chunks of several sequences over caches of odd lengths
        dict(name="prefill_ragged_f16", op="prefill", fmt="f16", batch=6, hq=8, hkv=8, d=64, max_len=777,
             max_q=130, page=16, per_head=False, window=0, pad=3),
        # a whole prompt of 8192 tokens, Llama-8B-shaped layer
        dict(name="prefill_8k", op="prefill", fmt="bf16", batch=1, hq=32, hkv=8, d=128, max_len=8192,
             max_q=8192, page=16, per_head=False, window=0, pad=0),
        # the next chunk of a long prompt over an MXFP4 cache
        dict(name="prefill_mxfp4_chunk", op="prefill", fmt="mxfp4", batch=1, hq=16, hkv=2, d=128, max_len=32768,
             max_q=2048, page=512, per_head=True, window=0, pad=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "decode", "decode", "decode", "prefill", "prefill"])
    fmt = rng.choice(["bf16", "f16", "mxfp4"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    per_head = rng.random() < 0.4
    page = rng.choice([1, 16, 24, 48, 64, 128, 512])
    c = dict(op=op, fmt=fmt, d=d, hkv=hkv, page=page, per_head=per_head)
    if op == "append":
        n = _log_int(rng, 1, 16384)
        rot = rng.choice([0, 32, d // 2, d])
        c.update(n=n, hq=hkv * g if rng.random() < 0.8 else 0, rot=rot, interleaved=rng.random() < 0.5,
                 fused=rng.random() < 0.5, spare=rng.randint(0, 50))
    elif op == "read":
        c.update(n=_log_int(rng, 1, 32768), spare=rng.randint(0, 50))
    elif op == "decode":
        batch = _log_int(rng, 1, 128)
        budget = 32 * 8 * 32768 * 128 // (batch * hkv * d)
        max_len = _log_int(rng, 1, min(1 << 17, max(1, budget // 4)))
        c.update(batch=batch, hq=hkv * g, max_len=max_len,
                 min_len=max_len if rng.random() < 0.3 else 1,
                 window=_log_int(rng, 1, max_len) if rng.random() < 0.25 else 0,
                 out="f32" if rng.random() < 0.5 else ("f16" if fmt == "f16" else "bf16"),
                 zero=rng.randint(0, batch // 4))
    else:
        batch = _log_int(rng, 1, 12)
        max_len = _log_int(rng, 1, 8192)
        while batch * hkv * g * max_len * max_len > 8 * 8192 * 8192:
            max_len = (max_len + 1) // 2
        c.update(batch=batch, hq=hkv * g, max_len=max_len, max_q=_log_int(rng, 1, max_len),
                 window=_log_int(rng, 1, max_len) if rng.random() < 0.25 else 0, pad=rng.randint(0, 5))
    return c


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """(q_lens, kv_lens) of an attention case, from the case alone (work() needs them too)."""
    r = np.random.RandomState(7)
    if case["op"] == "decode":
        lens = r.randint(case["min_len"], case["max_len"] + 1, size=case["batch"])
        lens[r.randint(case["batch"])] = case["max_len"]
        if case["zero"]:
            lens[r.permutation(case["batch"])[: case["zero"]]] = 0
        return np.ones(case["batch"], np.int64), lens.astype(np.int64)
    q = r.randint(1, case["max_q"] + 1, size=case["batch"])
    q[r.randint(case["batch"])] = case["max_q"]
    kv = np.array([r.randint(x, case["max_len"] + 1) for x in q])
    kv[int(np.argmax(q))] = case["max_len"]
    return q.astype(np.int64), kv.astype(np.int64)


def _cache(case, n_pages, gen, fill):
    """Page tensors; `fill` "values" draws every slot, "stale" leaves what a reused page holds."""
    heads = () if case["per_head"] else (case["hkv"],)
    shape = (n_pages, case["page"]) + heads
    d = case["d"]
    if case["fmt"] == "mxfp4":
        def codes():
            return torch.randint(0, 256, shape + (d // 2,), dtype=torch.uint8, device=DEV, generator=gen)

        def scales(lo, hi):
            return torch.randint(lo, hi, shape + (d // 32,), dtype=torch.uint8, device=DEV, generator=gen)
        # key blocks of amplitude around 1, value blocks over a wider range
        return codes(), codes(), scales(124, 127), scales(120, 127)
    dt = DT[case["fmt"]]
    if fill == "stale":
        return tuple(torch.full(shape + (d,), float("nan"), dtype=dt, device=DEV) for _ in range(2)) + (None, None)

    def vals():
        out = torch.empty(shape + (d,), dtype=dt, device=DEV)
        flat = out.view(-1)
        for i in range(0, flat.numel(), 1 << 28):
            part = flat[i:i + (1 << 28)]
            part.copy_(torch.randn(part.numel(), device=DEV, generator=gen, dtype=torch.float32))
        return out
    return vals(), vals(), None, None


def _handle(state, case):
    """What a program of the library keeps beside the data: the context and the page views."""
    import kv_cache_vector_05_b200 as T
    c, t = T.tq_lloyd_max_codebook(case["d"], 2)
    state["T"] = T
    state["ctx"] = T.tq_codebook_load(case["d"], 2, 4, c, t, None, hadamard_signs=np.ones(case["d"], np.int8))
    state["pages"] = T.KVPages(*state["cache"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    cpu = np.random.RandomState(seed % (1 << 31))
    s = {"case": case}
    d, hkv, page = case["d"], case["hkv"], case["page"]
    dt = DT[case["fmt"]]
    if case["op"] in ("append", "read"):
        n = case["n"]
        used = -(-n // page)
        units = hkv if case["per_head"] else 1
        n_pages = used * units + case["spare"]
        s["cache"] = _cache(case, n_pages, gen, "values" if case["op"] == "read" else "stale")
        order = cpu.permutation(n_pages)[: used * units].reshape(units, used)
        tok = np.arange(n)
        slot = order[:, tok // page] * page + tok % page                  # [units, n]
        slot = np.ascontiguousarray(slot.T) if case["per_head"] else slot[0]
        s["slot"] = torch.from_numpy(slot.astype(np.int64)).to(DEV)
        if case["op"] == "append":
            hq, width = case["hq"], case["hq"] + 2 * hkv
            if case["fused"]:                                              # one projection's output rows
                qkv = torch.randn((n, width, d), device=DEV, generator=gen).to(dt)
                s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            else:
                s["q"], s["k"], s["v"] = (torch.randn((n, h, d), device=DEV, generator=gen).to(dt)
                                          for h in (hq, hkv, hkv))
            if hq == 0:
                s["q"] = None
            s["table"] = s["pos"] = None
            if case["rot"]:
                half = case["rot"] // 2
                n_pos = 2 * n + 100
                freq = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
                ang = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * freq
                s["table"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
                s["pos"] = torch.from_numpy(cpu.randint(0, n_pos, size=n).astype(np.int64)).to(DEV)
            if s["q"] is not None:
                s["q_out"] = torch.empty((n, hq, d), dtype=dt, device=DEV)
        if case["op"] == "read" or case["fmt"] == "mxfp4":
            s["k_out"], s["v_out"] = (torch.empty((n, hkv, d), dtype=dt, device=DEV) for _ in range(2))
    else:
        q_lens, kv_lens = _lengths(case)
        batch, hq = case["batch"], case["hq"]
        max_pages = max(1, -(-case["max_len"] // page))
        used = -(-kv_lens // page)
        units = hkv if case["per_head"] else 1
        n_pages = int(used.sum()) * units + 2
        s["cache"] = _cache(case, n_pages, gen, "values")
        order = cpu.permutation(n_pages)
        table = np.zeros((batch, units, max_pages), np.int32)
        at = 0
        for b in range(batch):
            for u in range(units):
                table[b, u, : used[b]] = order[at:at + used[b]]
                at += int(used[b])
        s["q_lens"], s["kv_lens"] = q_lens, kv_lens
        if case["fmt"] != "mxfp4":                                          # what a reused page still holds
            for b in range(batch):
                if kv_lens[b] % page:
                    last = torch.from_numpy(table[b, :, used[b] - 1].astype(np.int64)).to(DEV)
                    for x in s["cache"][:2]:
                        x[last, int(kv_lens[b] % page):] = float("nan")
        s["block_table"] = torch.from_numpy(table if case["per_head"] else table[:, 0].copy()).to(DEV)
        s["seq_lens"] = torch.from_numpy(kv_lens.astype(np.int32)).to(DEV)
        if case["op"] == "decode":
            s["q"] = torch.randn((batch, hq, d), device=DEV, generator=gen).to(dt)
            out_dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[case["out"]]
            s["out"] = torch.empty((batch, hq, d), dtype=out_dt, device=DEV)
            s["lse"] = torch.empty((batch, hq), dtype=torch.float32, device=DEV)
        else:
            total = int(q_lens.sum())
            s["q"] = torch.randn((total + case["pad"], hq, d), device=DEV, generator=gen).to(dt)
            s["out"] = torch.zeros((total + case["pad"], hq, d), dtype=dt, device=DEV)   # pad rows stay
            s["lse"] = torch.zeros((total + case["pad"], hq), dtype=torch.float32, device=DEV)
            s["cu_q"] = torch.from_numpy(np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)).to(DEV)
    if own:
        _handle(s, case)
        T = s["T"]
        if case["op"] == "decode":
            need = T.tq_decode_kv_pages_workspace_bytes(s["ctx"], case["batch"], case["hq"], hkv)
            s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
        elif case["op"] == "prefill":
            need = T.tq_prefill_kv_pages_workspace_bytes(s["ctx"], s["q"].shape[0], case["batch"], case["hq"], hkv,
                                                         case["max_len"], case["max_q"])
            s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ the passes

def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(state, case)


def _run_own(s, case):
    T = s["T"]
    if case["op"] == "append":
        T.tq_append_kv_pages(s["ctx"], s["pages"], s["k"], s["v"], s["slot"], q=s["q"], q_out=s.get("q_out"),
                             cos_sin=s["table"], positions=s["pos"], interleaved=case["interleaved"])
        if case["fmt"] != "mxfp4":
            return s.get("q_out"), s["cache"][0], s["cache"][1]
        k, v = T.tq_read_kv_pages(s["ctx"], s["pages"], s["slot"], case["hkv"], k_out=s["k_out"], v_out=s["v_out"])
        return s.get("q_out"), k, v
    if case["op"] == "read":
        return T.tq_read_kv_pages(s["ctx"], s["pages"], s["slot"], case["hkv"], k_out=s["k_out"], v_out=s["v_out"])
    if case["op"] == "decode":
        return T.tq_decode_kv_pages(s["ctx"], s["q"], s["pages"], case["hkv"], s["block_table"], case["max_len"],
                                    seq_lens=s["seq_lens"], window=case["window"], out=s["out"], lse=s["lse"],
                                    workspace=s["ws"])
    return T.tq_prefill_kv_pages(s["ctx"], s["q"], s["pages"], case["hkv"], s["block_table"], case["max_len"],
                                 s["cu_q"], case["max_q"], seq_lens=s["seq_lens"], window=case["window"],
                                 out=s["out"], lse=s["lse"], workspace=s["ws"])


def _dequant(codes, scales, dtype):
    """MXFP4 codes [..., d/2] and scales [..., d/32] as values of `dtype` (fp32 or fp64)."""
    grid = torch.tensor(GRID + tuple(-x for x in GRID), dtype=dtype, device=codes.device)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    x = grid[nib.int()].unflatten(-1, (-1, 32))
    e = torch.ldexp(torch.ones((), dtype=torch.float64, device=codes.device), scales.double() - 127).to(dtype)
    return (x * e[..., None]).flatten(-2)


def _quant(x):
    """fp32 values [..., d] through MXFP4 (scale 2^(floor(log2 amax) - 2), ties to the even code)."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(min=-126)
    e = torch.where(amax > 0, e, torch.full_like(e, -126))
    y = torch.ldexp(b, -e).abs()
    code = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int() + (y > 2.5).int()
            + (y >= 3.5).int() + (y > 5).int())
    grid = torch.tensor(GRID, dtype=torch.float32, device=x.device)
    return (torch.ldexp(grid[code], e) * torch.sign(b)).flatten(-2)


def _rotate(x, table, pos, interleaved):
    """The position rotation of x [n, heads, d] in x's type: pairs (i, i + rot/2), or (2i, 2i + 1)."""
    if table is None:
        return x
    half = table.shape[1] // 2
    cs = table[pos].to(x.dtype)
    c, s = cs[:, None, :half], cs[:, None, half:]
    out = x.clone()
    i0, i1 = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., i0], x[..., i1]
    out[..., i0] = a * c - b * s
    out[..., i1] = b * c + a * s
    return out


def _flat(x):
    return x.flatten(0, 1)                                                  # [slots, (hkv,) width]


def _tokens(case, cache, rows, unit, which, dtype):
    """Vectors of KV head `unit` at cache slots `rows`, in `dtype` (which: 0 keys, 1 values)."""
    x = _flat(cache[which])
    x = x[rows] if case["per_head"] else x[rows, unit]
    if case["fmt"] != "mxfp4":
        return x.to(dtype)
    sc = _flat(cache[2 + which])
    return _dequant(x, sc[rows] if case["per_head"] else sc[rows, unit], dtype)


def _rows(s, case, b, unit):
    n = int(s["kv_lens"][b])
    tab = s["block_table"][b, unit] if case["per_head"] else s["block_table"][b]
    t = torch.arange(n, device=DEV)
    return tab[t // case["page"]].long() * case["page"] + t % case["page"]


def _read_plain(s, case):
    outs = []
    for which in (0, 1):
        cols = []
        for u in range(case["hkv"]):
            rows = s["slot"][:, u] if case["per_head"] else s["slot"]
            cols.append(_tokens(case, s["cache"], rows, u, which, torch.float32).to(DT[case["fmt"]]))
        outs.append(torch.stack(cols, 1))
    return outs[0], outs[1]


def _attend(q, k, v, pos, window, scale):
    """q [rows, g, d] at positions pos [rows] over k, v [n, d]: (out [rows, g, d], lse [rows, g]), in
    q's type; rows are taken in blocks that keep the score matrix near 1 GB."""
    n = k.shape[0]
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=q.dtype, device=q.device)
    if n == 0:
        return out, lse
    t = torch.arange(n, device=q.device)
    step = max(1, (1 << 30) // (q.element_size() * n * q.shape[1]))
    for i in range(0, q.shape[0], step):
        logit = (q[i:i + step].flatten(0, 1) @ k.T * scale).unflatten(0, (-1, q.shape[1]))
        p = pos[i:i + step, None]
        seen = t[None] <= p
        if window:
            seen &= t[None] > p - window
        logit = logit.masked_fill(~seen[:, None], -math.inf)
        m = logit.amax(-1, keepdim=True).clamp(min=torch.finfo(q.dtype).min)
        e = torch.exp(logit - m)
        total = e.sum(-1, keepdim=True)
        o = (e.flatten(0, 1) @ v).unflatten(0, (-1, q.shape[1]))
        out[i:i + step] = torch.where(total > 0, o / total.clamp(min=1e-300 if q.dtype == torch.float64 else 1e-30), 0)
        lse[i:i + step] = (m + torch.log(total)).squeeze(-1)
    return out, lse


def _attention(s, case, dtype, out, lse):
    """Every (sequence, KV head) of an attention case in `dtype`, written into out and lse."""
    g, scale = case["hq"] // case["hkv"], 1.0 / math.sqrt(case["d"])
    at = 0
    for b in range(case["batch"]):
        nq, n = int(s["q_lens"][b]), int(s["kv_lens"][b])
        pos = torch.arange(n - nq, n, device=DEV)
        for u in range(case["hkv"]):
            rows = _rows(s, case, b, u)
            k, v = (_tokens(case, s["cache"], rows, u, w, dtype) for w in (0, 1))
            h = slice(u * g, (u + 1) * g)
            o, l_ = _attend(s["q"][at:at + nq, h].to(dtype), k, v, pos, case["window"], scale)
            out[at:at + nq, h], lse[at:at + nq, h] = o.to(out.dtype), l_.to(lse.dtype)
        at += nq
    return out, lse


def _run_plain(s, case):
    if case["op"] == "read":
        return _read_plain(s, case)
    if case["op"] != "append":
        return _attention(s, case, torch.float32, s["out"], s["lse"])
    k32 = _rotate(s["k"].float(), s["table"], s["pos"], case["interleaved"])
    v32 = s["v"].float()
    q = None if s["q"] is None else _rotate(s["q"].float(), s["table"], s["pos"], case["interleaved"]).to(s["q"].dtype)
    if case["fmt"] == "mxfp4":
        return q, _quant(k32).to(s["k"].dtype), _quant(v32).to(s["v"].dtype)
    for x, c in ((k32, s["cache"][0]), (v32, s["cache"][1])):
        x = x.to(c.dtype)
        if case["per_head"]:
            _flat(c)[s["slot"].flatten()] = x.flatten(0, 1)
        else:
            _flat(c)[s["slot"]] = x
    return q, s["cache"][0], s["cache"][1]


def work(case):
    d, hkv = case["d"], case["hkv"]
    rec = d // 2 + d // 32 if case["fmt"] == "mxfp4" else 2 * d            # bytes of a cached vector
    if case["op"] == "append":
        n, hq = case["n"], case["hq"]
        units = hkv if case["per_head"] else 1
        nbytes = n * (2 * hq * d * 2 + 2 * hkv * (2 * d + rec) + 8 * units) + (n * (4 * case["rot"] + 8) if case["rot"] else 0)
        if case["fmt"] == "mxfp4":                                          # read back
            nbytes += n * 2 * hkv * (rec + 2 * d)
        return {"bytes": nbytes, "flops": n * (hq + hkv) * 3 * case["rot"]}
    if case["op"] == "read":
        return {"bytes": case["n"] * (2 * hkv * (rec + 2 * d) + 8 * (hkv if case["per_head"] else 1)),
                "flops": case["n"] * 2 * hkv * d if case["fmt"] == "mxfp4" else 0}
    q_lens, kv_lens = _lengths(case)
    g, w = case["hq"] // hkv, case["window"]
    seen = pairs = 0
    for nq, n in zip(q_lens.tolist(), kv_lens.tolist()):
        nq = min(nq, n)
        first = n - nq
        seen += n if not w else n - max(0, first - w + 1)
        p = np.arange(first, n, dtype=np.float64) + 1
        pairs += float((np.minimum(p, w) if w else p).sum())
    rows = int(q_lens.sum())
    out_bytes = {"f32": 4}.get(case.get("out"), 2)
    return {"bytes": 2 * seen * hkv * rec + rows * case["hq"] * (2 * d + out_bytes * d + 4),
            "flops": 4 * d * g * hkv * pairs}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "read" and case["fmt"] != "mxfp4":                     # a copy
        return tuple(c.flatten(0, 1)[s["slot"]].to(f64) for c in s["cache"][:2])
    if case["op"] == "read":
        outs = []
        for which in (0, 1):
            c, sc = _flat(s["cache"][which]), _flat(s["cache"][2 + which])
            c, sc = c[s["slot"]], sc[s["slot"]]                             # [n, hkv, .] in both layouts
            mag = (c.unsqueeze(-1) >> torch.tensor([0, 4], dtype=torch.uint8, device=DEV) & 15).flatten(-2).long()
            ex, man = (mag & 7) >> 1, (mag & 1).to(f64)
            val = torch.where(ex > 0, (1 + man / 2) * 2.0 ** (ex - 1).to(f64), man / 2)
            val = torch.where(mag >= 8, -val, val)
            outs.append(val * torch.repeat_interleave(2.0 ** (sc.to(f64) - 127), 32, dim=-1))
        return outs[0], outs[1]
    if case["op"] == "append":
        def turn(x):
            if x is None or s["table"] is None:
                return None if x is None else x.to(f64)
            half = case["rot"] // 2
            x = x.to(f64)
            z = x[..., : 2 * half]
            z = z.unflatten(-1, (half, 2)) if case["interleaved"] else z.unflatten(-1, (2, half)).transpose(-1, -2)
            cs = s["table"][s["pos"]].to(f64)
            w = torch.view_as_complex(z.contiguous()) * torch.complex(cs[:, :half], cs[:, half:])[:, None]
            w = torch.view_as_real(w)
            w = w.flatten(-2) if case["interleaved"] else w.transpose(-1, -2).flatten(-2)
            return torch.cat([w, x[..., 2 * half:]], -1)
        q, k, v = turn(s["q"]), turn(s["k"]), s["v"].to(f64)
        if case["fmt"] == "mxfp4":
            # the keys' codes follow the rotated value's last bits at a tie: no 64-bit counterpart
            b = v.unflatten(-1, (-1, 32))
            amax = b.abs().amax(-1, keepdim=True)
            step = 2.0 ** (torch.floor(torch.log2(amax.clamp(min=2.0 ** -126))) - 2)
            y = (b / step).abs()
            e = torch.floor(torch.log2(y.clamp(min=1.0)))
            y = torch.clamp(torch.round(y * 2.0 ** (1 - e)) * 2.0 ** (e - 1), max=6.0)
            return q, None, (y * step * torch.sign(b)).flatten(-2)
        outs = []
        for x, c in ((k, s["cache"][0]), (v, s["cache"][1])):
            c = c.to(f64)
            if case["per_head"]:
                for u in range(case["hkv"]):
                    c.flatten(0, 1)[s["slot"][:, u]] = x[:, u]
            else:
                c.flatten(0, 1)[s["slot"]] = x
            outs.append(c)
        return q, outs[0], outs[1]
    # attention: probabilities from log-softmax over each row's own tokens, in blocks of rows
    out = torch.zeros(s["out"].shape, dtype=f64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=f64, device=DEV)
    g, at = case["hq"] // case["hkv"], 0
    for b in range(case["batch"]):
        nq, n = int(s["q_lens"][b]), int(s["kv_lens"][b])
        for u in range(case["hkv"]):
            rows = _rows(s, case, b, u)
            k, v = (_tokens(case, s["cache"], rows, u, w, f64) for w in (0, 1))
            blk = max(1, (1 << 26) // max(1, n * g))
            for i in range(0, nq, blk):
                j = min(nq, i + blk)
                pos = torch.arange(n - nq + i, n - nq + j, device=DEV)
                lo = max(0, int(pos[0]) - case["window"] + 1) if case["window"] else 0
                hi = max(lo, int(pos[-1]) + 1)
                x = torch.einsum("rgd,nd->rgn", s["q"][at + i:at + j, u * g:(u + 1) * g].to(f64), k[lo:hi])
                x = x / math.sqrt(case["d"])
                t = torch.arange(lo, hi, device=DEV)
                hide = t[None] > pos[:, None]
                if case["window"]:
                    hide |= t[None] <= pos[:, None] - case["window"]
                x = x.masked_fill(hide[:, None], -math.inf)
                z = torch.logsumexp(x, -1) if hi > lo else torch.full(x.shape[:2], -math.inf, dtype=f64, device=DEV)
                p = torch.exp(x - z.clamp(min=-1e300)[..., None])
                out[at + i:at + j, u * g:(u + 1) * g] = torch.einsum("rgn,nd->rgd", p, v[lo:hi])
                lse[at + i:at + j, u * g:(u + 1) * g] = z
        at += nq
    return out, lse
