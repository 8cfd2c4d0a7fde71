// Append to and read from a page cache.
//
// append: y = R(position) x for the heads of q and k (pairs (a, b) -> (a cos - b sin,
// b cos + a sin) with fp32 cosines and sines from the caller's table, every product and sum
// rounded to fp32, so the result does not depend on how the work is laid out), then one
// rounding to the 16-bit type or to MXFP4. read: records back to dense rows.
//
// Both move each byte once and are bound by HBM, or by launch latency for a decode step.
// A lane owns one 16-byte chunk (8 coordinates) of a vector, so a vector is d / 8 lanes and
// its loads and stores are whole lines; the partner chunk of the half-split rotation is a
// second load of the same lines (an L1 hit), which costs less than exchanging 4 registers.
// A warp keeps the 8 cosines and 8 sines of its chunk in registers and walks the heads of
// one token with them: the table's 4 rot_dim bytes per token are read once per warp and not
// once per head (the table bytes of a chunk are four times its data).
#include <algorithm>

#include "kv_pages.cuh"
#include "tq_device.cuh"

namespace tq {
namespace {

struct AppendArgs {
  PageView pg;
  const char* q;
  const char* k;
  const char* v;
  char* q_out;
  int64_t q_b, k_b, v_b, qo_b;  // row strides in bytes
  const float* table;
  const int64_t* pos;
  int64_t n_pos;
  int half;  // rot_dim / 2; 0: no rotation
  int interleaved;
  const int64_t* slot;
  int64_t n;
  int hq;       // 0: no queries
  int splits;   // warps that share a token
  int iters;    // vectors each lane handles
  unsigned int* err;
};

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // vectors in flight per lane: 8 16-byte loads

// The rotated (or copied) chunk `ch` of one vector as fp32.
template <typename T>
__device__ __forceinline__ void turn(const uint4& own, const uint4& par, int mode, const float (&c)[8],
                                     const float (&s)[8], float (&y)[8]) {
  const uint32_t w[4] = {own.x, own.y, own.z, own.w}, p[4] = {par.x, par.y, par.z, par.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = Half2<T>::unpack(w[i]);
    y[2 * i] = a.x;
    y[2 * i + 1] = a.y;
  }
  if (mode == 0) return;
  if (mode == 3) {  // pairs (2i, 2i + 1) lie in the chunk; c, s hold their four angles
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1];
      y[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
      y[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
    }
    return;
  }
  // mode 1: this chunk holds the pairs' first coordinates, 2: the second ones
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 b = Half2<T>::unpack(p[i]);
    const float b0 = __fmul_rn(b.x, s[2 * i]), b1 = __fmul_rn(b.y, s[2 * i + 1]);
    const float a0 = __fmul_rn(y[2 * i], c[2 * i]), a1 = __fmul_rn(y[2 * i + 1], c[2 * i + 1]);
    y[2 * i] = mode == 1 ? __fsub_rn(a0, b0) : __fadd_rn(a0, b0);
    y[2 * i + 1] = mode == 1 ? __fsub_rn(a1, b1) : __fadd_rn(a1, b1);
  }
}

// MXFP4 of 8 coordinates; the 4 lanes of an aligned quad hold one block of 32. The scale
// comes from the largest magnitude's exponent alone, read off its bits (as integers, NaN >
// infinity > every finite value), so it is exact; x 2^-e is exact as well unless it falls
// far below the smallest code.
__device__ __forceinline__ uint32_t quantise8(const float (&y)[8], uint32_t& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(kFull, m, 1));
  m = max(m, __shfl_xor_sync(kFull, m, 2));
  if (m >= 0x7f800000u) {
    scale = 255;
    return 0;
  }
  const int e = max((int)(m >> 23) - 127 - 2, -126);
  scale = (uint32_t)(e + 127);
  const float r = __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= e2m1_pair(y[2 * i] * r, y[2 * i + 1] * r) << (8 * i);
  return w;
}

template <typename T, bool MX, int LPV>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  constexpr int VP = 32 / LPV;  // vectors a warp holds at once
  const int lane = threadIdx.x & 31;
  const int64_t wid = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t tok = wid / a.splits;
  if (tok >= a.n) return;
  const int split = (int)(wid - tok * a.splits);
  const int ch = lane % LPV, sub = lane / LPV;
  const PageView& pg = a.pg;
  const int64_t* slots = a.slot + (pg.per_head ? tok * pg.hkv : tok);
  const int64_t slot0 = __ldg(slots);
  if (!pg.per_head && slot0 == -1) return;
  const int heads = a.hq + 2 * pg.hkv;

  // the rotation of this lane's chunk
  int mode = 0, pch = ch;
  float c[8], s[8];
  if (a.half) {
    if (pg.per_head) {  // a row whose every slot is padding has no position
      bool any = false;
      for (int h = 0; h < pg.hkv; ++h) any |= __ldg(slots + h) != -1;
      if (!any) return;
    }
    const int64_t pos = __ldg(a.pos + tok);
    if (pos < 0 || pos >= a.n_pos) {
      if (lane == 0) atomicOr(a.err, kErrIndex);
      return;
    }
    if (ch * 8 < 2 * a.half) {
      const float* row = a.table + pos * 2 * a.half;
      if (a.interleaved) {
        mode = 3;
        const float4 x = __ldg(reinterpret_cast<const float4*>(row + ch * 4));
        const float4 y = __ldg(reinterpret_cast<const float4*>(row + a.half + ch * 4));
        c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
        s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
      } else {
        mode = ch * 8 < a.half ? 1 : 2;
        pch = mode == 1 ? ch + a.half / 8 : ch - a.half / 8;
        const int t0 = (mode == 1 ? ch : pch) * 8;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(row + t0 + i));
          const float4 y = __ldg(reinterpret_cast<const float4*>(row + a.half + t0 + i));
          c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
          s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
        }
      }
    }
  }

  int64_t soff0 = 0;  // the row's place in the cache, where its heads share one
  const bool in0 = slot0 >= 0 && slot0 < pg.n_slots;
  const int64_t off0 = !pg.per_head && in0 ? record_offset(pg, slot0, 0, soff0) : 0;

  const int first = split * a.iters * VP + sub;
  for (int i0 = 0; i0 < a.iters; i0 += kUnroll) {
    uint4 own[kUnroll], par[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = first + (i0 + u) * VP;
      own[u] = par[u] = make_uint4(0, 0, 0, 0);
      if (i0 + u >= a.iters || h >= heads) continue;
      const char* src = h < a.hq                ? a.q + tok * a.q_b + (int64_t)h * (LPV * 16)
                        : h < a.hq + pg.hkv     ? a.k + tok * a.k_b + (int64_t)(h - a.hq) * (LPV * 16)
                                                : a.v + tok * a.v_b + (int64_t)(h - a.hq - pg.hkv) * (LPV * 16);
      own[u] = *reinterpret_cast<const uint4*>(src + ch * 16);
      if (h < a.hq + pg.hkv && (mode == 1 || mode == 2)) par[u] = *reinterpret_cast<const uint4*>(src + pch * 16);
    }
    __syncwarp();  // q_out may be q: every chunk is read before any is written
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = first + (i0 + u) * VP;
      const bool live = i0 + u < a.iters && h < heads;
      const bool is_q = h < a.hq;
      float y[8];
      turn<T>(own[u], par[u], h < a.hq + pg.hkv ? mode : 0, c, s, y);
      uint32_t word = 0, scale = 0;
      if constexpr (MX) word = quantise8(y, scale);  // warp-wide: before any lane leaves
      if (!live) continue;
      const uint4 packed = make_uint4(Half2<T>::pack(y[0], y[1]), Half2<T>::pack(y[2], y[3]),
                                      Half2<T>::pack(y[4], y[5]), Half2<T>::pack(y[6], y[7]));
      if (is_q) {
        if (slot0 != -1)
          *reinterpret_cast<uint4*>(a.q_out + tok * a.qo_b + (int64_t)h * (LPV * 16) + ch * 16) = packed;
        continue;
      }
      const bool is_k = h < a.hq + pg.hkv;
      const int kh = is_k ? h - a.hq : h - a.hq - pg.hkv;
      const int64_t slot = pg.per_head ? __ldg(slots + kh) : slot0;
      if (slot < 0 || slot >= pg.n_slots) {
        if (slot != -1 && ch == 0) atomicOr(a.err, kErrIndex);
        continue;
      }
      int64_t off = off0 + (int64_t)kh * pg.head_b, soff = soff0 + (int64_t)kh * pg.shead_b;
      if (pg.per_head) off = record_offset(pg, slot, kh, soff);
      char* base = is_k ? pg.k : pg.v;
      if constexpr (MX) {
        *reinterpret_cast<uint32_t*>(base + off + ch * 4) = word;
        if ((ch & 3) == 0) (is_k ? pg.ks : pg.vs)[soff + ch / 4] = (uint8_t)scale;
      } else {
        *reinterpret_cast<uint4*>(base + off + ch * 16) = packed;
      }
    }
  }
}

struct ReadArgs {
  PageView pg;
  const int64_t* slot;
  int64_t n;
  char* k_out;
  char* v_out;
  unsigned int* err;
};

// One lane per 16-byte chunk of the dense rows; blockIdx.y 0: keys, 1: values (or the one
// output asked for). kUnroll chunks of a lane lie a grid apart and are in flight together.
template <bool MX, int LPV>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs a) {
  const PageView& pg = a.pg;
  const bool keys = a.k_out && (blockIdx.y == 0);
  const char* base = keys ? pg.k : pg.v;
  const uint8_t* sbase = keys ? pg.ks : pg.vs;
  char* out = keys ? a.k_out : a.v_out;
  const int64_t total = a.n * pg.hkv * LPV, step = (int64_t)gridDim.x * kThreads;
  for (int64_t c0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; c0 < total; c0 += step * kUnroll) {
    int64_t slot[kUnroll];
    uint4 x[kUnroll];
    uint32_t sc[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t vec = (c0 + u * step) / LPV;
      slot[u] = c0 + u * step < total ? __ldg(a.slot + (pg.per_head ? vec : quotient(vec, pg.hkv))) : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      x[u] = make_uint4(0, 0, 0, 0);
      sc[u] = 0;
      if (slot[u] < 0 || slot[u] >= pg.n_slots) {
        if (slot[u] != -1) atomicOr(a.err, kErrIndex);
        slot[u] = -1;
        continue;
      }
      const int64_t c = c0 + u * step, vec = c / LPV;
      const int ch = (int)(c - vec * LPV);
      int64_t soff;
      const int64_t off = record_offset(pg, slot[u], (int)(vec - quotient(vec, pg.hkv) * pg.hkv), soff);
      if constexpr (MX) {
        x[u].x = *reinterpret_cast<const uint32_t*>(base + off + ch * 4);
        sc[u] = sbase[soff + ch / 4];
      } else {
        x[u] = *reinterpret_cast<const uint4*>(base + off + ch * 16);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (slot[u] < 0) continue;
      if constexpr (MX) {
        uint32_t h[4], r[4];
        e2m1x8_f16(x[u].x, h);
        const float f = e8m0(sc[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 t = Half2<__half>::unpack(h[i]);
          r[i] = Half2<__nv_bfloat16>::pack(t.x * f, t.y * f);
        }
        x[u] = make_uint4(r[0], r[1], r[2], r[3]);
      }
      *reinterpret_cast<uint4*>(out + (c0 + u * step) * 16) = x[u];
    }
  }
}

template <typename T, bool MX>
cudaError_t run_append(int d, const AppendArgs& a, unsigned blocks, cudaStream_t st) {
  if (d == 64) append_kernel<T, MX, 8><<<blocks, kThreads, 0, st>>>(a);
  else if (d == 128) append_kernel<T, MX, 16><<<blocks, kThreads, 0, st>>>(a);
  else append_kernel<T, MX, 32><<<blocks, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const tq_ctx* ctx, const PageView& pg, int format, int dtype, int64_t n, int hq,
                             const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, const tq_rope* rope, const int64_t* slot, void* q_out,
                             int64_t q_out_stride, cudaStream_t stream) {
  AppendArgs a{};
  a.pg = pg;
  a.q = static_cast<const char*>(q), a.k = static_cast<const char*>(k), a.v = static_cast<const char*>(v);
  a.q_out = static_cast<char*>(q_out);
  a.q_b = q_stride * 2, a.k_b = k_stride * 2, a.v_b = v_stride * 2, a.qo_b = q_out_stride * 2;
  if (rope && rope->rot_dim > 0) {
    a.table = rope->cos_sin, a.pos = rope->positions, a.n_pos = rope->n_positions;
    a.half = rope->rot_dim / 2, a.interleaved = rope->interleaved;
  }
  a.slot = slot, a.n = n, a.hq = q ? hq : 0, a.err = ctx->d_err;
  // Heads per warp: one group of 32 / (d / 8) vectors each while that leaves the SMs short of
  // warps (a decode step is latency), more as tokens grow, up to 8 groups, so that a warp's
  // table row serves several heads.
  const int vp = 256 / ctx->shape.d, groups = (a.hq + 2 * pg.hkv + vp - 1) / vp;
  const int64_t want = (int64_t)ctx->num_sms * 64;
  a.iters = (int)std::max<int64_t>(1, std::min<int64_t>(8, n * groups / want));
  a.splits = (groups + a.iters - 1) / a.iters;
  const int64_t blocks = (n * a.splits + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (format == TQ_KV_MXFP4) return run_append<__nv_bfloat16, true>(ctx->shape.d, a, (unsigned)blocks, stream);
  if (dtype == TQ_BF16) return run_append<__nv_bfloat16, false>(ctx->shape.d, a, (unsigned)blocks, stream);
  return run_append<__half, false>(ctx->shape.d, a, (unsigned)blocks, stream);
}

cudaError_t launch_kv_read(const tq_ctx* ctx, const PageView& pg, int format, int64_t n, const int64_t* slot,
                           void* k_out, void* v_out, cudaStream_t stream) {
  const ReadArgs a{pg, slot, n, static_cast<char*>(k_out), static_cast<char*>(v_out), ctx->d_err};
  const int lpv = ctx->shape.d / 8;
  const int64_t chunks = n * pg.hkv * lpv;
  // one chunk per lane until the grid holds 8 blocks per SM, then up to kUnroll
  const int64_t most = (int64_t)ctx->num_sms * 8;
  const int64_t need = (chunks + kThreads - 1) / kThreads;
  const int64_t blocks = std::min(need, std::max(most, (need + kUnroll - 1) / kUnroll));
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks, k_out && v_out ? 2 : 1);
  const bool mx = format == TQ_KV_MXFP4;
  if (lpv == 8) (mx ? read_kernel<true, 8> : read_kernel<false, 8>)<<<grid, kThreads, 0, stream>>>(a);
  else if (lpv == 16) (mx ? read_kernel<true, 16> : read_kernel<false, 16>)<<<grid, kThreads, 0, stream>>>(a);
  else (mx ? read_kernel<true, 32> : read_kernel<false, 32>)<<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace tq
