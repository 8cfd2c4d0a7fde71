// Causal attention of chunks of new tokens over a page cache that holds them.
//
// Work. The G query heads of a KV head see the same keys, so a sequence's rows are packed as
// (token, head) pairs, row i = (token i / G, head i % G): a CTA takes 256 packed rows (128 at
// d = 256) of one (sequence, KV head) as two M = 128 tiles and streams the cache once for all of
// them, up to its last row's position. 4 d flop per (row, token) pair against 4 d bytes per 256
// rows: bound by the tensor cores and by the exponentials (one per pair, at 16 a clock and SM
// exactly as long as the two products of d = 128). Blocks of late rows, which see the most
// tokens, are launched first. Short chunks over long caches leave SMs idle; then the tokens are
// split as well and combine_kernel joins the parts.
//
// One CTA of 12 warps per SM, in roles:
//   warps 0-3, 4-7  softmax of row tile 0, 1: thread = row = tensor-memory lane. S is read into
//                   registers, P = 2^(S' - m) written over it in 16 bits; while one tile's
//                   exponentials run, the tensor cores work for the other tile
//   warp 8          one thread issues the MMAs: S = Q K^T (both from shared memory, K-major), then
//                   O += P V with P from tensor memory and V as it lies in the cache (MN-major)
//   warps 9-11      bring K and V tiles into a ring of stages in the 128-byte-swizzled layout, by
//                   cp.async (pages of any size, records of any stride), or, for MXFP4, by loads
//                   one tile ahead that are turned into exact bf16 values on the way
// The accumulated O lives in tensor memory and is rescaled only when a row's maximum has grown
// by more than 2^kSlack, so almost every tile leaves it alone.
//
// Tokens a row does not see get p = 0 by a select on the score, whatever the score is. A value
// that is not finite would still spoil p = 0 rows in the product (0 x inf), so in tiles where
// rows differ in what they see (the diagonal, the window's edge) the producers replace such
// values by 0 and raise a flag; the epilogue then adds them to the rows that do see them.
#include <algorithm>

#include "kv_pages.cuh"
#include "tq_device.cuh"
#include "tq_sm100.cuh"

namespace tq {
namespace {

using namespace sm100;

constexpr int kThreads = 384, kLoaders = 96;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegHuge = -1.7e38f;  // maximum of no logits: finite, so that -inf - m is -inf

struct PreArgs {
  PageView pg;
  const char* q;
  int64_t q_b;
  int64_t total_q;
  int batch, hq, G;
  const int32_t* cu_q;
  int64_t max_q;
  const int32_t* table;
  int64_t max_pages;
  const int32_t* lens;
  int64_t max_len, window;
  float scale_log2;
  char* out;
  float* lse;
  float* part;    // splits > 1: [splits][total_q * hq][HD + 4]
  int splits;
  int blocks;     // row blocks of the longest sequence
  unsigned int* err;
};

template <bool MX, int HD>
struct Config {
  static constexpr int NQ = HD == 256 ? 1 : 2;    // row tiles
  static constexpr int BN = HD == 256 ? 64 : 128; // tokens per K / V tile
  static constexpr int kStage = BN * HD * 2;
  static constexpr int kStages = HD == 64 ? 8 : HD == 256 ? 4 : MX ? 4 : 5;
  static constexpr int kQ = NQ * 128 * HD * 2;
  static constexpr int kOffRow = kQ + kStages * kStage;        // int64 [BN] record offsets
  static constexpr int kOffScale = kOffRow + BN * 8;           // int64 [BN] scale offsets (MXFP4)
  static constexpr int kOffBar = kOffScale + (MX ? BN * 8 : 0);
  static constexpr int kSmem = 1024 + kOffBar + 256;
  static constexpr int kS = 128, kO = 256;        // tensor-memory columns: S tile t at t * kS, O at kO + t * HD
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void loaders_sync() { asm volatile("bar.sync 1, 96;" ::: "memory"); }

// Shared-memory operand of `rows` rows and HD 16-bit columns: byte of the 16-byte chunk ch of a
// row (panels of 64 columns, chunks permuted within 128 bytes by row % 8).
template <int ROWS>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) {
  return (uint32_t)((ch >> 3) * (ROWS * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
}

// Zero the elements of a 16-byte chunk that are not finite; true if there were any.
template <typename T>
__device__ __forceinline__ bool scrub(uint4& x) {
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  uint32_t* w = &x.x;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & kExp) == kExp) w[i] &= 0xffff0000u, any = true;
    if (((w[i] >> 16) & kExp) == kExp) w[i] &= 0x0000ffffu, any = true;
  }
  return any;
}

// What a block works on.
struct Block {
  int64_t q0;         // first row of the sequence in q
  int b, kvh, first;  // sequence, KV head, first packed row
  int rows;           // packed rows of the sequence
  int nq, n;          // its new tokens, its tokens in the cache
  bool ok;
};

template <int ROWS>
__device__ __forceinline__ Block locate(const PreArgs& a, bool report) {
  Block w;
  const int per = a.batch * a.pg.hkv;
  int x = blockIdx.x / per;
  const int rest = blockIdx.x - x * per;
  w.b = rest / a.pg.hkv;
  w.kvh = rest - w.b * a.pg.hkv;
  const int64_t s = __ldg(a.cu_q + w.b), e = __ldg(a.cu_q + w.b + 1);
  w.ok = s >= 0 && e >= s && e <= a.total_q && e - s <= a.max_q;
  if (!w.ok && report) atomicOr(a.err, kErrIndex);
  w.q0 = s;
  w.nq = w.ok ? (int)(e - s) : 0;
  w.rows = w.nq * a.G;
  w.first = (a.blocks - 1 - x) * ROWS;  // late rows first
  int64_t n = a.lens ? (int64_t)__ldg(a.lens + w.b) : a.max_len;
  w.n = (int)(n < 0 ? 0 : n > a.max_len ? a.max_len : n);
  return w;
}

template <typename T, bool MX, int HD>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(const PreArgs a) {
  using C = Config<MX, HD>;
  constexpr int NQ = C::NQ, BN = C::BN, NS = C::kStages, ROWS = NQ * 128;
  constexpr bool F16 = std::is_same<T, __half>::value;
  // P in f16: the largest p is 2^13 to 2^15, so that small ones keep their bits
  constexpr float kOff = F16 ? 13.f : 0.f, kSlack = F16 ? 2.f : 8.f;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Block w = locate<ROWS>(a, tid == 0);
  if (!w.ok || w.first >= w.rows) return;

  // positions: row i's token sits at p0 + i / G; tokens of this block's rows: [lo, hi)
  const int p0 = w.n - w.nq;
  int end_row = w.first + ROWS < w.rows ? w.first + ROWS : w.rows;
  const int pmin = p0 + w.first / a.G, pmax = p0 + (end_row - 1) / a.G;
  const int wnd = a.window && a.window < 0x7fffffff ? (int)a.window : 0;
  const int lo = wnd && pmin - wnd + 1 > 0 ? pmin - wnd + 1 : 0;
  const int hi = pmax + 1;  // <= n
  int t0 = lo / BN, t1 = hi > lo ? (hi - 1) / BN + 1 : t0;
  if (a.splits > 1) {
    const int nt = t1 - t0, s = blockIdx.y, base = t0;
    t0 = base + (int)((int64_t)nt * s / a.splits);
    t1 = base + (int)((int64_t)nt * (s + 1) / a.splits);
  }
  // tiles of each row tile: [t0, te[t]): a tile of rows stops at its own last position
  int cnt[2], tmin[2], tmax[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int f = w.first + t * 128;
    cnt[t] = 0, tmin[t] = tmax[t] = 0;
    if (t >= NQ || f >= end_row) continue;
    const int l = f + 127 < end_row - 1 ? f + 127 : end_row - 1;
    tmin[t] = p0 + f / a.G, tmax[t] = p0 + l / a.G;
    const int te = tmax[t] < 0 ? t0 : tmax[t] / BN + 1;
    cnt[t] = (te < t1 ? te : t1) - t0;
    if (cnt[t] < 0) cnt[t] = 0;
  }
  const int n_tiles = cnt[0] > cnt[1] ? cnt[0] : cnt[1];
  auto is_edge = [&](int kv0) { return kv0 + BN - 1 > pmin || (wnd && kv0 <= pmax - wnd); };

  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint64_t* b_q = bars;            // Q in shared memory
  uint64_t* b_s = bars + 1;        // [NQ] S of a row tile written (and its last P V done)
  uint64_t* b_p = bars + 3;        // [NQ] P of a row tile written
  uint64_t* b_o = bars + 5;        // [NQ] O of a row tile complete
  uint64_t* b_full = bars + 7;     // [NS]
  uint64_t* b_free = bars + 7 + NS;
  volatile uint32_t* ctl = reinterpret_cast<volatile uint32_t*>(bars + 7 + 2 * NS);  // tmem, dirty
  if (warp == 8) {
    tmem_alloc(const_cast<uint32_t*>(ctl), 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    ctl[1] = 0;
    mbar_init(b_q, kLoaders);
    for (int t = 0; t < 2; ++t) mbar_init(b_s + t, 1), mbar_init(b_p + t, 128), mbar_init(b_o + t, 1);
    for (int s = 0; s < NS; ++s) mbar_init(b_full + s, kLoaders), mbar_init(b_free + s, 1);
    mbar_init_fence();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = ctl[0];
  const uint32_t s_q = smem_u32(sm), s_ring = s_q + C::kQ;
  bool good = true;  // no wait has timed out; after one, the roles run out without waiting
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (good && !mbar_wait(bar, parity)) {
      good = false;
      atomicOr(a.err, 1u);
    }
    return good;
  };

  if (warp >= 9 && n_tiles > 0) {
    // ---- loaders ----------------------------------------------------------------------
    const int lt = tid - 288;
    constexpr int QC = HD / 8, QR = kLoaders / QC;  // 16-byte chunks per row, rows per pass
    {
      const int ch = lt % QC;
      for (int i = lt / QC; i < ROWS; i += QR) {
        const int row = w.first + i, tok = row / a.G, h = row - tok * a.G;
        const bool ok = row < end_row;
        const char* src = a.q + (ok ? (w.q0 + tok) * a.q_b + ((int64_t)w.kvh * a.G + h) * (HD * 2) : 0) + ch * 16;
        cp_async16(s_q + (i >> 7) * (128 * HD * 2) + chunk_at<128>(i & 127, ch), src, ok);
      }
      cp_commit();
    }
    // record offsets of a tile's tokens: table entries are loaded a tile ahead of their use
    int64_t* offs = reinterpret_cast<int64_t*>(sm + C::kOffRow);
    [[maybe_unused]] int64_t* soffs = reinterpret_cast<int64_t*>(sm + C::kOffScale);
    const int32_t* trow = a.table + (a.pg.per_head ? (int64_t)w.b * a.pg.hkv + w.kvh : (int64_t)w.b) * a.max_pages;
    int pid[2], pof[2];
    auto look = [&](int tile) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int tok = tile * BN + lt + i * kLoaders;
        tok = tok < lo ? lo : tok >= hi ? hi - 1 : tok;
        const int blk = tok / (int)a.pg.page_size;
        pof[i] = tok - blk * (int)a.pg.page_size;
        pid[i] = __ldg(trow + blk);
      }
    };
    auto place = [&]() {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = lt + i * kLoaders;
        if (r >= BN) break;
        int64_t p = pid[i];
        if (p < 0 || p >= a.pg.n_pages) {
          atomicOr(a.err, kErrIndex);
          p = 0;
        }
        offs[r] = p * a.pg.page_b + (int64_t)pof[i] * a.pg.tok_b + (int64_t)w.kvh * a.pg.head_b;
        if constexpr (MX) soffs[r] = p * a.pg.spage_b + (int64_t)pof[i] * a.pg.stok_b + (int64_t)w.kvh * a.pg.shead_b;
      }
    };
    look(t0);
    place();
    loaders_sync();
    bool dirty = false;
    if constexpr (!MX) {
      constexpr int kLag = 2;  // copies of this many stages stay in flight
      const int ch = lt % QC;
      // group g: 0 is Q, 1 + 2 j K tile j, 2 + 2 j V tile j; stage (g - 1) % NS
      auto arrive = [&](int g) {
        if (g == 0) {
          fence_async_smem();
          mbar_arrive(b_q);
          return;
        }
        const int st = (g - 1) % NS, kv0 = (t0 + (g - 1) / 2) * BN;
        if ((g & 1) == 0 && is_edge(kv0)) {  // this thread's own chunks of a V tile
          for (int r = lt / QC; r < BN; r += QR) {
            const uint32_t at = s_ring + st * C::kStage + chunk_at<BN>(r, ch);
            uint4 x = lds128(at);
            if (scrub<T>(x)) sts128(at, x), dirty = true;
          }
          if (dirty) ctl[1] = 1;
        }
        fence_async_smem();
        mbar_arrive(b_full + st);
      };
      const int groups = 1 + 2 * n_tiles;
      for (int g = 1; g < groups; ++g) {
        const int j = (g - 1) >> 1, st = (g - 1) % NS;
        if (g > NS) wait(b_free + st, ((g - 1) / NS - 1) & 1);
        if ((g & 1) && j + 1 < n_tiles) look(t0 + j + 1);
        const char* src = ((g & 1) ? a.pg.k : a.pg.v) + ch * 16;
        const int kv0 = (t0 + j) * BN;
        if (good)
          for (int r = lt / QC; r < BN; r += QR)
            cp_async16(s_ring + st * C::kStage + chunk_at<BN>(r, ch), src + offs[r], kv0 + r >= lo && kv0 + r < hi);
        cp_commit();
        if (!(g & 1) && j + 1 < n_tiles) {
          loaders_sync();  // the offsets have been used
          place();
          loaders_sync();
        }
        if (g >= kLag) {
          cp_wait<kLag>();
          arrive(g - kLag);
        }
      }
      cp_wait<0>();
      for (int g = groups - kLag; g < groups; ++g) arrive(g);  // groups >= 3
    } else {
      cp_wait<0>();
      fence_async_smem();
      mbar_arrive(b_q);
      constexpr int CPR = HD / 32, RS = kLoaders / CPR, NC = (BN + RS - 1) / RS;  // one chunk = one block of 32
      const int blk = lt % CPR, r0 = lt / CPR;
      uint4 code[NC];
      uint32_t sc[NC];
      auto fetch = [&](bool keys, int kv0) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int r = r0 + i * RS;
          code[i] = make_uint4(0, 0, 0, 0);
          sc[i] = 127;
          if (r < BN && kv0 + r >= lo && kv0 + r < hi) {
            code[i] = __ldg(reinterpret_cast<const uint4*>((keys ? a.pg.k : a.pg.v) + offs[r] + blk * 16));
            sc[i] = __ldg((keys ? a.pg.ks : a.pg.vs) + soffs[r] + blk);
          }
        }
      };
      fetch(true, t0 * BN);
      for (int h = 0; h < 2 * n_tiles; ++h) {  // K and V tiles in turn
        const int st = h % NS, kv0 = (t0 + (h >> 1)) * BN;
        const bool scan = (h & 1) && is_edge(kv0);
        uint4 cur[NC];
        uint32_t cs[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) cur[i] = code[i], cs[i] = sc[i];
        if (!(h & 1)) {
          fetch(false, kv0);
          if (h + 2 < 2 * n_tiles) look(t0 + (h >> 1) + 1);
        } else if (h + 1 < 2 * n_tiles) {
          loaders_sync();
          place();
          loaders_sync();
          fetch(true, kv0 + BN);
        }
        if (h >= NS) wait(b_free + st, (h / NS - 1) & 1);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int r = r0 + i * RS;
          if (r >= BN || !good) break;
          const uint32_t wd[4] = {cur[i].x, cur[i].y, cur[i].z, cur[i].w};
          const uint32_t f = e8m0_bf16(cs[i]) * 0x10001u, two112 = 0x77807780u;
          const __nv_bfloat162 f2 = *reinterpret_cast<const __nv_bfloat162*>(&f);
          const __nv_bfloat162 k2 = *reinterpret_cast<const __nv_bfloat162*>(&two112);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[4];
            e2m1x8_f16(wd[c], x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t y = (x[e] & 0x80008000u) | ((x[e] >> 3) & 0x0fff0fffu);  // code 2^-112 as bf16
              const __nv_bfloat162 v = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y), k2), f2);
              x[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            uint4 o = make_uint4(x[0], x[1], x[2], x[3]);
            if (scan && scrub<T>(o)) dirty = true;
            sts128(s_ring + st * C::kStage + chunk_at<BN>(r, blk * 4 + c), o);
          }
        }
        if (dirty) ctl[1] = 1;
        fence_async_smem();
        mbar_arrive(b_full + st);
      }
    }
  } else if (warp == 8 && n_tiles > 0) {
    // ---- MMA issue ----------------------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t kFmt = F16 ? 0u : 1u;
      constexpr uint32_t i_qk = idesc_f16_f32(128, BN) | (kFmt << 7) | (kFmt << 10);
      constexpr uint32_t i_pv = idesc_f16_f32(128, HD) | (kFmt << 7) | (kFmt << 10) | (1u << 16);  // B MN-major
      auto qk = [&](int t, int st) {
#pragma unroll
        for (int k = 0; k < HD; k += 16)
          umma_f16(tmem + t * C::kS, sw128_desc(s_q + t * (128 * HD * 2), k, 128),
                   sw128_desc(s_ring + st * C::kStage, k, BN), i_qk, k > 0);
        umma_commit(b_s + t);
      };
      auto pv = [&](int t, int st, bool acc) {
#pragma unroll
        for (int k = 0; k < BN; k += 16)
          umma_f16_ts(tmem + C::kO + t * HD, tmem + t * C::kS + k / 2, sw128_mn_desc(s_ring + st * C::kStage, k, BN),
                      i_pv, acc || k > 0);
      };
      if (wait(b_q, 0) && wait(b_full, 0)) {
        fence_after_sync();
#pragma unroll
        for (int t = 0; t < NQ; ++t)
          if (cnt[t] > 0) qk(t, 0);
        umma_commit(b_free);
        for (int j = 0; j < n_tiles && good; ++j) {
          const int sv = (2 * j + 1) % NS, sk = (2 * j + 2) % NS;
          if (!wait(b_full + sv, ((2 * j + 1) / NS) & 1)) break;
          if (j + 1 < n_tiles && !wait(b_full + sk, ((2 * j + 2) / NS) & 1)) break;
#pragma unroll
          for (int t = 0; t < NQ; ++t) {
            if (j >= cnt[t]) continue;
            if (!wait(b_p + t, j & 1)) break;
            fence_after_sync();
            pv(t, sv, j > 0);
            if (j + 1 < cnt[t]) qk(t, sk);
            else umma_commit(b_o + t);
          }
          umma_commit(b_free + sv);
          if (j + 1 < n_tiles) umma_commit(b_free + sk);
        }
        // the last arrival of a commit must not outlive the block's shared memory
        const int last = 2 * n_tiles - 1;
        wait(b_free + last % NS, (last / NS) & 1);
      }
    }
    __syncwarp();
  } else if (warp < 4 * NQ) {
    // ---- softmax ------------------------------------------------------------------------
    const int t = warp >> 2, i = w.first + t * 128 + (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + t * C::kS + lanes, to = tmem + C::kO + t * HD + lanes;
    const int tok = i / a.G, pos = p0 + tok;
    const int n = t == 0 ? cnt[0] : cnt[1], fmin = t == 0 ? tmin[0] : tmin[1], fmax = t == 0 ? tmax[0] : tmax[1];
    const float sl = a.scale_log2;
    float m = kNegHuge, l = 0.f;
    for (int j = 0; j < n; ++j) {
      if (!__all_sync(kFull, wait(b_s + t, j & 1))) break;
      fence_after_sync();
      uint32_t s[BN];
#pragma unroll
      for (int c = 0; c < BN; c += 32) tmem_ld32(ts + c, *reinterpret_cast<uint32_t(*)[32]>(s + c));
      tmem_ld_wait();
      const int kv0 = (t0 + j) * BN;
      if (kv0 + BN - 1 > fmin || (wnd && kv0 <= fmax - wnd)) {
        const int last = pos - kv0, from = wnd ? last - wnd + 1 : -1;  // columns seen: [from, last]
#pragma unroll
        for (int c = 0; c < BN; ++c)
          if (c > last || c < from) s[c] = 0xff800000u;
      }
      float mx = __uint_as_float(s[0]), my = __uint_as_float(s[1]);
#pragma unroll
      for (int c = 2; c < BN; c += 2)
        mx = fmaxf(mx, __uint_as_float(s[c])), my = fmaxf(my, __uint_as_float(s[c + 1]));
      mx = fmaxf(mx, my) * sl;
      if (__any_sync(kFull, mx > m + (kOff + kSlack))) {
        const float mn = fmaxf(m, mx - kOff), f = ex2(m - mn);
        m = mn;
        l *= f;
        if (j > 0) {
#pragma unroll
          for (int c = 0; c < HD; c += 32) {
            uint32_t o[32];
            tmem_ld32(to + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(to + c, o);
          }
        }
      }
      const float2 sl2 = make_float2(sl, sl), nm2 = make_float2(-m, -m);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < BN; c += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = fma2(make_float2(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1])), sl2, nm2);
          const float2 p = make_float2(ex2(x.x), ex2(x.y));
          sum = add2(sum, p);
          pk[e / 2] = Half2<T>::pack(p.x, p.y);
        }
        tmem_st16(ts + c / 2, pk);
      }
      l += sum.x + sum.y;
      tmem_st_wait();
      fence_before_sync();
      mbar_arrive(b_p + t);
    }
    // epilogue: O / l in q's type, or the parts of a split
    if (n > 0) good = __all_sync(kFull, wait(b_o + t, 0));
    fence_after_sync();
    const bool mine = i < end_row;
    const int64_t row = (w.q0 + tok) * a.hq + (int64_t)w.kvh * a.G + (i - tok * a.G);
    const bool fix = n > 0 && ctl[1] != 0;
    const float inv = l == 0.f ? 0.f : 1.f / l;  // no token (or no finite logit): zeros
    if (good) {
      float* part = a.splits > 1 ? a.part + ((int64_t)blockIdx.y * a.total_q * a.hq + row) * (HD + 4) : nullptr;
#pragma unroll 1
      for (int c = 0; c < HD; c += 32) {
        uint32_t o[32];
        __syncwarp();
        if (n > 0) {
          tmem_ld32(to + c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (!mine) continue;
        if (fix) {
          // add the values that are not finite (zeroed in edge tiles) of the tokens this row sees
          for (int j = 0; j < n; ++j) {
            const int kv0 = (t0 + j) * BN;
            if (!is_edge(kv0)) continue;
            for (int x = kv0 < lo ? lo : kv0; x < kv0 + BN && x <= pos; ++x) {
              if (wnd && x <= pos - wnd) continue;
              const int blk = x / (int)a.pg.page_size, off = x - blk * (int)a.pg.page_size;
              int64_t p = __ldg(a.table + (a.pg.per_head ? (int64_t)w.b * a.pg.hkv + w.kvh : (int64_t)w.b) * a.max_pages +
                                blk);
              p = p < 0 || p >= a.pg.n_pages ? 0 : p;
              const char* v = a.pg.v + p * a.pg.page_b + (int64_t)off * a.pg.tok_b + (int64_t)w.kvh * a.pg.head_b;
              if constexpr (MX) {
                const uint8_t* vs = a.pg.vs + p * a.pg.spage_b + (int64_t)off * a.pg.stok_b +
                                    (int64_t)w.kvh * a.pg.shead_b;
                const float f = e8m0(vs[c / 32]);
                for (int q4 = 0; q4 < 4; ++q4) {
                  uint32_t hx[4];
                  e2m1x8_f16(*reinterpret_cast<const uint32_t*>(v + c / 2 + q4 * 4), hx);
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const float2 z = Half2<__half>::unpack(hx[e >> 1]);
                    const float u = __bfloat162float(__float2bfloat16((e & 1 ? z.y : z.x) * f));
                    if (!isfinite(u)) {
#pragma unroll
                      for (int d = 0; d < 32; ++d)
                        if (d == q4 * 8 + e) o[d] = __float_as_uint(__uint_as_float(o[d]) + u);
                    }
                  }
                }
              } else {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  const float2 z = Half2<T>::unpack(*reinterpret_cast<const uint32_t*>(v + (c + e) * 2));
                  if (!isfinite(z.x)) o[e] = __float_as_uint(__uint_as_float(o[e]) + z.x);
                  if (!isfinite(z.y)) o[e + 1] = __float_as_uint(__uint_as_float(o[e + 1]) + z.y);
                }
              }
            }
          }
        }
        if (part) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(part + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(a.out + (row * HD + c) * 2);
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = __uint_as_float(o[e + u]) * inv;
            dst[e / 8] = make_uint4(Half2<T>::pack(x[0], x[1]), Half2<T>::pack(x[2], x[3]), Half2<T>::pack(x[4], x[5]),
                                    Half2<T>::pack(x[6], x[7]));
          }
        }
      }
      if (mine) {
        if (part) *reinterpret_cast<float2*>(part + HD) = make_float2(m, l);
        else if (a.lse) a.lse[row] = (m + log2f(l)) * kLn2;
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// Join the parts of split rows: one warp per row of the same blocks.
template <typename T, int HD, int ROWS>
__global__ void __launch_bounds__(256) kv_prefill_combine_kernel(const PreArgs a) {
  constexpr int E = HD / 32;  // values per lane
  const Block w = locate<ROWS>(a, false);
  if (!w.ok) return;
  const int lane = threadIdx.x & 31;
  const int64_t stride = a.total_q * a.hq * (HD + 4);
  for (int i = w.first + (threadIdx.x >> 5); i < w.first + ROWS && i < w.rows; i += 8) {
    const int tok = i / a.G;
    const int64_t row = (w.q0 + tok) * a.hq + (int64_t)w.kvh * a.G + (i - tok * a.G);
    const float* p = a.part + row * (HD + 4);
    float m = kNegHuge, l = 0.f, o[E];
    for (int s = 0; s < a.splits; ++s) m = fmaxf(m, p[s * stride + HD]);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int s = 0; s < a.splits; ++s) {
      const float f = ex2(p[s * stride + HD] - m);
      l = fmaf(f, p[s * stride + HD + 1], l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f, p[s * stride + lane * E + e], o[e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(a.out + (row * HD + lane * E + e) * 2) = Half2<T>::pack(o[e] * inv, o[e + 1] * inv);
    if (a.lse && lane == 0) a.lse[row] = (m + log2f(l)) * kLn2;
  }
}

template <typename T, bool MX, int HD>
cudaError_t run(const PreArgs& a, cudaStream_t st) {
  using C = Config<MX, HD>;
  auto kern = kv_prefill_kernel<T, MX, HD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (int64_t)a.blocks * a.batch * a.pg.hkv;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  kern<<<dim3((unsigned)blocks, a.splits), kThreads, C::kSmem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.splits == 1) return e;
  kv_prefill_combine_kernel<T, HD, C::NQ * 128><<<(unsigned)blocks, 256, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, bool MX>
cudaError_t pick(int d, const PreArgs& a, cudaStream_t st) {
  if (d == 64) return run<T, MX, 64>(a, st);
  if (d == 128) return run<T, MX, 128>(a, st);
  return run<T, MX, 256>(a, st);
}

int block_rows(int d) { return d == 256 ? 128 : 256; }

// Parts a call's tokens are split into: none while the row blocks fill the SMs; otherwise as
// many as fit on them, each of at least 1024 tokens (a part costs a pass of its rows through
// the workspace, about as much as 100 tokens).
int split_count(const tq_ctx* ctx, int batch, int G, int hkv, int64_t max_len, int64_t max_q) {
  const int64_t rows = block_rows(ctx->shape.d);
  const int64_t blocks = (max_q * G + rows - 1) / rows * batch * hkv;
  if (blocks <= 0 || blocks * 2 > ctx->num_sms) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(ctx->num_sms / blocks, max_len / 1024));
}

}  // namespace

size_t kv_prefill_workspace(const tq_ctx* ctx, int64_t total_q, int batch, int hq, int hkv, int64_t max_len,
                            int64_t max_q) {
  const int s = split_count(ctx, batch, hq / hkv, hkv, max_len, max_q);
  return s > 1 ? (size_t)s * total_q * hq * (ctx->shape.d + 4) * sizeof(float) : 0;
}

cudaError_t launch_kv_prefill(const tq_ctx* ctx, const PageView& pg, int format, const void* q, int64_t q_stride,
                              int64_t total_q, int batch, int hq, const int32_t* cu_q, int64_t max_q,
                              const int32_t* table, int64_t max_pages, const int32_t* seq_lens, int64_t max_len,
                              int64_t window, float scale, void* out, float* lse, void* workspace,
                              cudaStream_t stream) {
  PreArgs a{};
  a.pg = pg;
  a.q = static_cast<const char*>(q), a.q_b = q_stride * 2, a.total_q = total_q;
  a.batch = batch, a.hq = hq, a.G = hq / pg.hkv;
  a.cu_q = cu_q, a.max_q = max_q, a.table = table, a.max_pages = max_pages, a.lens = seq_lens;
  a.max_len = max_len, a.window = window, a.scale_log2 = scale * 1.4426950408889634f;
  a.out = static_cast<char*>(out), a.lse = lse, a.err = ctx->d_err;
  a.splits = split_count(ctx, batch, a.G, pg.hkv, max_len, max_q);
  a.part = static_cast<float*>(workspace);
  const int rows = block_rows(ctx->shape.d);
  a.blocks = (int)((max_q * a.G + rows - 1) / rows);
  const int d = ctx->shape.d;
  if (format == TQ_KV_MXFP4) return pick<__nv_bfloat16, true>(d, a, stream);
  if (format == TQ_KV_BF16) return pick<__nv_bfloat16, false>(d, a, stream);
  return pick<__half, false>(d, a, stream);
}

}  // namespace tq
