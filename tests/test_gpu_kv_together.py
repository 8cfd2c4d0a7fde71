"""The page caches and the packed cache used together, as a serving loop does: prompts appended
and attended in chunks, decode steps that append one token per sequence, full pages moved into the
packed cache (read, tq_compress_kv_slots) and the two attentions merged (tq_merge_attention).
Checked after every step against softmax attention in 64 bits over what the caches hold."""
import numpy as np
import pytest

import _pages as P
from _parity import make_ctx
from test_gpu_kv_decode import tolerance
from test_gpu_kv_pages import table_for, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import kv_cache_vector_05_b200 as T  # noqa: E402

DEV = "cuda:0"
PAGE, D, HKV, G, BATCH, ROT = 512, 128, 2, 4, 2, 64


class Server:
    """Per-head pages, so that a full page is a run of one head's records in both caches."""

    def __init__(self, fmt, seed):
        self.rng = np.random.default_rng(seed)
        self.fmt, self.dt = fmt, P.TORCH[fmt]
        self.ctx = make_ctx(T, D, 2, 4)
        self.n_pages = 40
        self.cache = P.make_cache(fmt, self.n_pages, PAGE, HKV, D, True)
        self.pages = T.KVPages(*self.cache)
        self.free = list(self.rng.permutation(self.n_pages))
        self.table = [[[] for _ in range(HKV)] for _ in range(BATCH)]
        self.len = [0] * BATCH
        self.moved = [0] * BATCH                        # leading tokens that live in the packed cache
        self.cos_sin = up(table_for(self.rng, 8192, ROT))

    def slots(self, b, t0, t1):
        """Cache rows [t1 - t0, HKV] of a sequence's tokens, new pages taken as needed."""
        out = np.empty((t1 - t0, HKV), np.int64)
        for h in range(HKV):
            pages = self.table[b][h]
            while len(pages) * PAGE < t1 - self.moved[b]:
                pages.append(self.free.pop())
            t = np.arange(t0, t1) - self.moved[b]
            out[:, h] = np.array(pages)[t // PAGE] * PAGE + t % PAGE
        return out

    def block_table(self):
        width = max(len(p) for row in self.table for p in row)
        tab = np.full((BATCH, HKV, width), 1 << 30, np.int32)
        for b in range(BATCH):
            for h in range(HKV):
                tab[b, h, :len(self.table[b][h])] = self.table[b][h]
        return up(tab), width * PAGE

    def append(self, counts):
        """New tokens of every sequence in one call, with one padding row at the end; their queries."""
        n = sum(counts) + 1
        qkv = torch.randn((n, HKV * (G + 2), D), device=DEV).to(self.dt)
        slot, pos = np.full((n, HKV), -1, np.int64), np.zeros(n, np.int64)
        at = 0
        for b, c in enumerate(counts):
            slot[at:at + c] = self.slots(b, self.len[b], self.len[b] + c)
            pos[at:at + c] = np.arange(self.len[b], self.len[b] + c)
            self.len[b] += c
            at += c
        hq = HKV * G
        T.tq_append_kv_pages(self.ctx, self.pages, qkv[:, hq:hq + HKV], qkv[:, hq + HKV:], up(slot), q=qkv[:, :hq],
                             q_out=qkv[:, :hq], cos_sin=self.cos_sin, positions=up(pos))
        return qkv[:, :hq]

    def held(self, b, h):
        """Values of a sequence's tokens in the pages, as the attention sees them."""
        s = up(self.slots(b, self.moved[b], self.len[b]))
        k, v = T.tq_read_kv_pages(self.ctx, self.pages, s, HKV)
        return P.f64(k[:, h]), P.f64(v[:, h])

    def lens(self):
        return up(np.array([n - m for n, m in zip(self.len, self.moved)], np.int32))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_serving_loop(fmt):
    s = Server(fmt, 21)
    scale, hq = D ** -0.5, HKV * G
    # prompts in two chunks
    for counts in ((1300, 611), (240, 90)):
        q = s.append(counts)
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        tab, cap = s.block_table()
        out, lse = T.tq_prefill_kv_pages(s.ctx, q, s.pages, HKV, tab, cap, up(cu), max(counts), seq_lens=s.lens())
        T.tq_check_device(s.ctx)
        for b in range(BATCH):
            rows = np.array([0, counts[b] // 2, counts[b] - 1])
            for h in range(HKV):
                k, v = s.held(b, h)
                qq = P.f64(q[int(cu[b]) + rows][:, h * G:(h + 1) * G])
                want, wl = P.attend(qq, k, v, rows + s.len[b] - counts[b], 0, scale)
                got = P.f64(out[int(cu[b]) + rows][:, h * G:(h + 1) * G])
                for i in range(len(rows)):
                    tol, _ = tolerance(qq[i], k, v, scale, D, len(k), fmt, "bf16", want[i], wl[i])
                    tol = tol + 2 * P.EPS["bf16"] * np.abs(v).max(0)              # P in one 16-bit term
                    assert (np.abs(got[i] - want[i]) <= tol).all(), (b, h, rows[i])

    def decode_step(packed, max_packed):
        q = s.append((1, 1))[:BATCH]
        tab, cap = s.block_table()
        outs, lses = torch.empty((2, BATCH, hq, D), device=DEV), torch.empty((2, BATCH, hq), device=DEV)
        T.tq_decode_kv_pages(s.ctx, q, s.pages, HKV, tab, cap, seq_lens=s.lens(), out=outs[0], lse=lses[0])
        got = outs[0]
        if packed is not None:
            T.tq_decode_attention_partial(s.ctx, q.contiguous(), packed, BATCH, hq, HKV, max_packed,
                                          seq_lens=up(np.array(s.moved, np.int32)), out=outs[1], lse=lses[1])
            got, _ = T.tq_merge_attention(outs, lses)
            kp, vp = T.tq_decompress(s.ctx, packed, BATCH * HKV * max_packed)
        T.tq_check_device(s.ctx)
        for b in range(BATCH):
            for h in range(HKV):
                k, v = s.held(b, h)
                if s.moved[b]:
                    at = (b * HKV + h) * max_packed
                    k = np.concatenate([P.f64(kp[at:at + s.moved[b]]), k])
                    v = np.concatenate([P.f64(vp[at:at + s.moved[b]]), v])
                qq = P.f64(q[b, h * G:(h + 1) * G])
                want, wl = P.attend(qq[None], k, v, np.array([len(k) - 1]), 0, scale)
                tol, _ = tolerance(qq, k, v, scale, D, len(k), fmt, "f32", want[0], wl[0])
                if s.moved[b]:
                    tol = tol + 1e-4 + 1e-3 * np.abs(want[0])                       # the packed decode's bound
                assert (np.abs(P.f64(got[b, h * G:(h + 1) * G]) - want[0]) <= tol).all(), (b, h)

    for _ in range(3):
        decode_step(None, 0)
    # the two leading pages of sequence 0 and the first of sequence 1 move into the packed cache
    max_packed = 1024
    rows = BATCH * HKV * max_packed
    packed = {"k_codes": torch.zeros((rows, s.ctx.k_code_bytes), dtype=torch.uint8, device=DEV),
              "k_signs": torch.zeros((rows, s.ctx.m // 8), dtype=torch.uint8, device=DEV),
              "k_norms": torch.zeros((rows, 2), dtype=torch.int16, device=DEV),
              "v_codes": torch.zeros((rows, s.ctx.v_code_bytes), dtype=torch.uint8, device=DEV),
              "v_params": torch.zeros((rows, D // 32, 2), dtype=torch.int16, device=DEV)}
    for b, n in ((0, 1024), (1, 512)):
        k, v = T.tq_read_kv_pages(s.ctx, s.pages, up(s.slots(b, 0, n)), HKV)
        slot = (b * HKV + np.arange(HKV)[None]) * max_packed + np.arange(n)[:, None]
        T.tq_compress_kv_slots(s.ctx, k.view(-1, D), v.view(-1, D), up(slot.reshape(-1)), packed)
        for h in range(HKV):
            s.free += s.table[b][h][:n // PAGE]
            s.table[b][h] = s.table[b][h][n // PAGE:]
        s.moved[b] = n
    for _ in range(3):
        decode_step(packed, max_packed)
