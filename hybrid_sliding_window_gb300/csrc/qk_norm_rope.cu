// RMSNorm of every query and key head, the position rotation, and the store of
// K and V into one layer's pool, in one pass over the projections' outputs.
//
// For a head row x of D values with weight w:
//   y = x * w / sqrt(mean(x^2) + eps)            (no weight given: y = x)
// and for the rot_dim leading values, in pairs (a, b) = (y_i, y_{i + rot/2})
// or (y_2i, y_{2i+1}), with the token's cosine and sine c_i, s_i:
//   (a, b) -> (a c - b s, b c + a s).
// All of it in float32, rounded once: to the queries' type, and to the pool's
// (E4M3: of the float32 quotient by the scale).  V is only stored.
//
// The pass should be bound by HBM: (Hq + 2 Hkv) D values read, Hq D + 2 Hkv D
// written per token.  A token's query heads are contiguous (as are its key and
// its value heads), so a persistent CTA - two per SM - streams whole tokens
// through a ring of shared-memory stages with bulk copies (one for each of q, k
// and v, and the token's row of the angle table): a hundred KB in flight per SM
// without a register for it.  A producer warp looks positions and slots up 32
// units ahead; eight warps take the rows from shared memory.  A row is held by
// D / 8 lanes (bf16) or D / 4 (f32), each with two 8-byte words that hold the
// two halves of its pairs: no value crosses lanes but the row's sum of squares.
// With 1 / rms = rs the pair is
//   rs * (x_a (w_a c) + x_b (-w_b s)),  rs * (x_b (w_b c) + x_a (w_a s)),
// whose bracketed factors a lane computes once per token (its dims are the same
// in every row), so an element costs a product, a fused product-sum and the
// product with rs, two elements at a time (f32x2).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_codec.cuh"
#include "spec_internal.h"
#include "tc_ptx.cuh"

namespace swa {
namespace {

constexpr int kNormWarps = 8;      // and a producer warp
constexpr int kNormStages = 4;
constexpr int kStageRows = 24576;  // bytes of head rows of a stage
constexpr int kStageTable = 512;   // bytes of an angle row (rot_dim <= 128)

struct NormParams {
  const char *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;   // bytes
  const int64_t *positions;
  const float *qw, *kw;
  float eps;
  const float *cos_sin;
  int64_t max_pos;
  int rot;
  const int64_t *full_loc, *swa_loc, *mapping;
  int64_t map_len;
  int in_full;
  int64_t pool_rows;
  KvAddr addr;
  int hq, hkv;
  float k_scale, v_scale;
  char *q_out;
  int32_t *err;
  int64_t units;         // chunks of all tokens
  int chunks;            // chunks of a token
  int chunk_rows;        // rows of a chunk
};

struct NormStage {
  int64_t base;          // pool byte offset of the token's K and V rows, -1: none
  int32_t ok;            // 0: bad position, nothing loaded
};

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// An 8-byte word of a row as pairs of floats, and back.
template <typename T> struct Word;
template <> struct Word<float> {
  static constexpr int kN = 2;
  static __device__ __forceinline__ void get(const uint2 &w, uint64_t (&x)[1]) {
    x[0] = tc::f2pack(__uint_as_float(w.x), __uint_as_float(w.y));
  }
  static __device__ __forceinline__ uint2 put(const uint64_t (&x)[1]) {
    float a, b;
    tc::f2unpack(x[0], a, b);
    return make_uint2(__float_as_uint(a), __float_as_uint(b));
  }
};
template <> struct Word<__nv_bfloat16> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint2 &w, uint64_t (&x)[2]) {
    x[0] = tc::f2pack(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
    x[1] = tc::f2pack(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  }
  static __device__ __forceinline__ uint2 put(const uint64_t (&x)[2]) {
    float a, b, c, d;
    tc::f2unpack(x[0], a, b);
    tc::f2unpack(x[1], c, d);
    return make_uint2(tc::pack_p<false>(a, b), tc::pack_p<false>(c, d));
  }
};

// Four values (a word of a bf16 row) as the E4M3 bytes of their quotients.
__device__ __forceinline__ uint32_t encode4(const uint64_t (&x)[2], float sc) {
  float a, b, c, d;
  tc::f2unpack(x[0], a, b);
  tc::f2unpack(x[1], c, d);
  return pack_e4m3x4(__fdiv_rn(a, sc), __fdiv_rn(b, sc), __fdiv_rn(c, sc), __fdiv_rn(d, sc));
}

// Bytes of global memory into shared memory (16-byte aligned both, a multiple
// of 16), completion counted on the barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// A unit is a chunk of one token's rows, counted through its query heads, key
// heads and value heads (an absent input has none).
template <typename T, int D, bool kF8, bool kInter>
__global__ void __launch_bounds__((kNormWarps + 1) * 32, 2) k_qk_norm_rope_store(NormParams P) {
  using Wd = Word<T>;
  constexpr int kEsz = (int)sizeof(T), kRow = D * kEsz;
  constexpr int W = Wd::kN, H = W / 2;    // values and pairs of a word
  constexpr int LPR = D / (2 * W);        // lanes of a row
  constexpr int RPW = 32 / LPR;           // rows of a warp's pass
  extern __shared__ __align__(128) char smem[];
  __shared__ uint64_t s_bar[2 * kNormStages];     // full, empty
  __shared__ NormStage s_info[kNormStages];
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nq = P.q ? P.hq : 0, nk = P.k ? P.hkv : 0, rows = nq + 2 * nk;
  auto full = [&](int s) { return tc::smem_u32(&s_bar[s]); };
  auto empty = [&](int s) { return tc::smem_u32(&s_bar[kNormStages + s]); };
  auto data = [&](int s) { return smem + s * (kStageRows + kStageTable); };
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < kNormStages; ++s) {
      tc::mbar_init(full(s), 1);
      tc::mbar_init(empty(s), kNormWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  __syncthreads();
  const int64_t step = gridDim.x;
  int issued = 0;                         // stages filled (producer)

  if (warp == kNormWarps) {
    // ===================== producer =====================
    int64_t pos = 0, base = -1;           // of unit k0 + lane
    for (int64_t u0 = blockIdx.x, k = 0; u0 < P.units; u0 += step, ++k) {
      if ((k & 31) == 0) {
        const int64_t u = u0 + lane * step;
        pos = 0;
        base = -1;
        if (u < P.units) {
          const int64_t t = u / P.chunks;
          if (P.rot > 0) {
            pos = P.positions[t];
            if (pos < 0 || pos >= P.max_pos) {
              set_error(P.err, SWA_DEVERR_RANGE);
              pos = -1;
            }
          }
          if (nk) {
            int64_t slot;
            if (P.in_full) {
              slot = P.full_loc[t];
            } else if (P.swa_loc) {
              slot = P.swa_loc[t];
            } else {
              int64_t f = P.full_loc[t];
              if (f < 0) f += P.map_len;
              slot = (f >= 0 && f < P.map_len) ? P.mapping[f] : -1;
            }
            if (slot < 0 || slot >= P.pool_rows) set_error(P.err, SWA_DEVERR_RANGE);
            else base = kv_row(P.addr, slot) * P.addr.row_bytes;
          }
        }
      }
      const int64_t upos = __shfl_sync(0xffffffffu, pos, (int)(k & 31));
      const int64_t ubase = __shfl_sync(0xffffffffu, base, (int)(k & 31));
      int good = 1;
      if (lane == 0) {
        const int s = issued % kNormStages, f = issued / kNormStages;
        if (f >= 1) good = tc::mbar_wait(empty(s), (f - 1) & 1, &s_abort);
        if (good) {
          const int64_t t = u0 / P.chunks;
          const int r0 = (int)(u0 % P.chunks) * P.chunk_rows, r1 = min(r0 + P.chunk_rows, rows);
          s_info[s] = NormStage{ubase, upos >= 0};
          if (upos < 0) {
            tc::mbar_arrive(full(s));
          } else {
            const uint32_t dst = tc::smem_u32(data(s));
            tc::mbar_expect_tx(full(s), (uint32_t)((r1 - r0) * kRow + P.rot * 4));
            auto part = [&](const char *src, int lo, int n) {   // rows lo .. lo + n - 1 of the token
              const int a = max(r0, lo), b = min(r1, lo + n);
              if (a < b)
                bulk_load(dst + (a - r0) * kRow, src + (int64_t)(a - lo) * kRow, (b - a) * kRow,
                          full(s));
            };
            part(P.q + t * P.q_stride, 0, nq);
            part(P.k + t * P.k_stride, nq, nk);
            part(P.v + t * P.v_stride, nq + nk, nk);
            if (P.rot > 0)
              bulk_load(dst + kStageRows, P.cos_sin + upos * P.rot, P.rot * 4, full(s));
          }
          ++issued;
        }
      }
      if (!__shfl_sync(0xffffffffu, good, 0)) break;
    }
  } else {
    // ===================== rows =====================
    const int sub = lane / LPR, li = lane % LPR;
    // First value of this lane's two words: of a turned lane the same place of
    // both halves (halves paired) or neighbouring words, else neighbouring words.
    const int half = P.rot >> 1;
    const bool turned = li * 2 * W < P.rot; // rot is a multiple of 2 W
    const bool split = turned && !kInter;
    const int da = split ? li * W : li * 2 * W, db = split ? half + li * W : li * 2 * W + W;
    int64_t k = 0;
    for (int64_t u0 = blockIdx.x; u0 < P.units; u0 += step, ++k) {
      const int s = (int)(k % kNormStages);
      if (!__all_sync(0xffffffffu,
                      tc::mbar_wait(full(s), (uint32_t)(k / kNormStages) & 1, &s_abort)))
        break;
      const NormStage info = s_info[s];
      const int64_t t = u0 / P.chunks;
      const int r0 = (int)(u0 % P.chunks) * P.chunk_rows, r1 = min(r0 + P.chunk_rows, rows);
      const char *tile = data(s);
      const float *angles = reinterpret_cast<const float *>(tile + kStageRows);
      // Rows of each kind in the chunk, in passes of RPW rows.
      const int q1 = min(r1, nq), k0 = max(r0, nq), k1 = min(r1, nq + nk), v0 = max(r0, nq + nk);
      const int pq = max(0, (q1 - r0 + RPW - 1) / RPW), pk = max(0, (k1 - k0 + RPW - 1) / RPW);
      const int pv = max(0, (r1 - v0 + RPW - 1) / RPW);
      const int total = info.ok ? pq + pk + pv : 0;
      // Factors of a kind: out_a = x_a fa + z_a ga, out_b = x_b fb + z_b gb, z the
      // pair's other values (halves: the other word; neighbours: swapped in place).
      uint64_t fa[H], ga[H], fb[H], gb[H];
      int have = -1;                      // kind whose factors are held
#pragma unroll 2
      for (int p = warp; p < total; p += kNormWarps) {
        const int kd = p < pq ? 0 : p < pq + pk ? 1 : 2;
        const int r = (kd == 0 ? r0 + p * RPW : kd == 1 ? k0 + (p - pq) * RPW
                                                        : v0 + (p - pq - pk) * RPW) + sub;
        const bool live = r < (kd == 0 ? q1 : kd == 1 ? k1 : r1);
        const char *src = tile + (live ? r - r0 : 0) * kRow;
        const uint2 ra = *reinterpret_cast<const uint2 *>(src + da * kEsz);
        const uint2 rb = *reinterpret_cast<const uint2 *>(src + db * kEsz);
        uint64_t a[H], b[H];
        Wd::get(ra, a);
        Wd::get(rb, b);
        if (kd != 2) {
          const float *w = kd == 0 ? P.qw : P.kw;
          if (have != kd) {
            have = kd;
            float xa[W], xb[W], ca[W], sa[W], cb[W], sb[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
              xa[i] = w ? w[da + i] : 1.f;
              xb[i] = w ? w[db + i] : 1.f;
              const int ia = kInter ? (da + i) >> 1 : da + i, ib = kInter ? (db + i) >> 1 : da + i;
              ca[i] = turned ? angles[ia] : 1.f;
              cb[i] = turned ? angles[ib] : 1.f;
              sa[i] = turned ? angles[half + ia] : 0.f;
              sb[i] = turned ? angles[half + ib] : 0.f;
            }
            float qa[W], qb[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
              const float za = kInter ? xa[i ^ 1] : xb[i], zb = kInter ? xb[i ^ 1] : xa[i];
              qa[i] = (kInter && (i & 1)) ? za * sa[i] : -za * sa[i];
              qb[i] = (kInter && !(i & 1)) ? -zb * sb[i] : zb * sb[i];
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
              fa[i] = tc::f2pack(xa[2 * i] * ca[2 * i], xa[2 * i + 1] * ca[2 * i + 1]);
              fb[i] = tc::f2pack(xb[2 * i] * cb[2 * i], xb[2 * i + 1] * cb[2 * i + 1]);
              ga[i] = tc::f2pack(qa[2 * i], qa[2 * i + 1]);
              gb[i] = tc::f2pack(qb[2 * i], qb[2 * i + 1]);
            }
          }
          uint64_t rs2 = tc::f2pack(1.f, 1.f);
          if (w) {
            uint64_t s2 = mul2(a[0], a[0]);
#pragma unroll
            for (int i = 1; i < H; ++i) s2 = tc::fma2(a[i], a[i], s2);
#pragma unroll
            for (int i = 0; i < H; ++i) s2 = tc::fma2(b[i], b[i], s2);
            float s0, s1;
            tc::f2unpack(s2, s0, s1);
            float ss = s0 + s1;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float rs = rsqrtf(ss * (1.f / D) + P.eps);
            rs2 = tc::f2pack(rs, rs);
          }
          uint64_t ya[H], yb[H];
#pragma unroll
          for (int i = 0; i < H; ++i) {
            ya[i] = mul2(a[i], fa[i]);
            yb[i] = mul2(b[i], fb[i]);
          }
          if (turned) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
              uint64_t za = b[i], zb = a[i];
              if (kInter) {
                float lo, hi;
                tc::f2unpack(a[i], lo, hi);
                za = tc::f2pack(hi, lo);
                tc::f2unpack(b[i], lo, hi);
                zb = tc::f2pack(hi, lo);
              }
              ya[i] = tc::fma2(za, ga[i], ya[i]);
              yb[i] = tc::fma2(zb, gb[i], yb[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < H; ++i) {
            a[i] = mul2(ya[i], rs2);
            b[i] = mul2(yb[i], rs2);
          }
        }
        if (kd == 0) {
          if (live) {
            char *dst = P.q_out + (t * P.hq + r) * kRow;
            *reinterpret_cast<uint2 *>(dst + da * kEsz) = Wd::put(a);
            *reinterpret_cast<uint2 *>(dst + db * kEsz) = Wd::put(b);
          }
        } else if (live && info.base >= 0) {
          const int h = r - nq - (kd == 2 ? nk : 0);
          char *dst = (kd == 2 ? P.addr.v : P.addr.k) + info.base;
          if constexpr (kF8) {
            const float sc = kd == 2 ? P.v_scale : P.k_scale;
            *reinterpret_cast<uint32_t *>(dst + h * D + da) = encode4(a, sc);
            *reinterpret_cast<uint32_t *>(dst + h * D + db) = encode4(b, sc);
          } else {
            *reinterpret_cast<uint2 *>(dst + h * kRow + da * kEsz) = kd == 2 ? ra : Wd::put(a);
            *reinterpret_cast<uint2 *>(dst + h * kRow + db * kEsz) = kd == 2 ? rb : Wd::put(b);
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty(s));
    }
  }
  __syncthreads();
  if (s_abort && threadIdx.x == kNormWarps * 32) {
    // A role gave up a wait: copies in flight still write this CTA's stages.
    set_error(P.err, SWA_DEVERR_TIMEOUT);
    for (int s = 0; s < kNormStages; ++s) {
      const int fills = (issued + kNormStages - 1 - s) / kNormStages;
      if (fills) tc::mbar_drain(full(s), (fills - 1) & 1);
    }
  }
}

template <typename T, int D, bool kF8, bool kInter>
cudaError_t launch_one(const Ctx &c, NormParams P, int64_t n, cudaStream_t s) {
  constexpr int kRow = D * (int)sizeof(T), kSmem = kNormStages * (kStageRows + kStageTable);
  const int rows = (P.q ? P.hq : 0) + (P.k ? 2 * P.hkv : 0);
  const int64_t ctas = 2LL * (c.num_sms > 0 ? c.num_sms : 148);
  // A chunk is a whole token where that fits a stage and there are tokens for
  // all CTAs; fewer tokens are cut finer, down to 16 rows.
  const int64_t even = (n * rows + ctas - 1) / ctas;
  P.chunk_rows = (int)(even < 16 ? 16 : even < kStageRows / kRow ? even : kStageRows / kRow);
  P.chunks = (rows + P.chunk_rows - 1) / P.chunk_rows;
  P.chunk_rows = (rows + P.chunks - 1) / P.chunks;
  P.units = n * P.chunks;
  cudaError_t e = cudaFuncSetAttribute(k_qk_norm_rope_store<T, D, kF8, kInter>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t grid = P.units < ctas ? P.units : ctas;
  k_qk_norm_rope_store<T, D, kF8, kInter><<<(unsigned)grid, (kNormWarps + 1) * 32, kSmem, s>>>(P);
  return cudaGetLastError();
}

template <typename T, int D, bool kF8>
cudaError_t launch_norm(const Ctx &c, bool inter, int64_t n, const NormParams &P, cudaStream_t s) {
  return inter ? launch_one<T, D, kF8, true>(c, P, n, s) : launch_one<T, D, kF8, false>(c, P, n, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope_store(Ctx &c, int layer, const QkNormArgs &a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  const LayerInfo &L = c.layers[layer];
  const int64_t esz = c.cfg.kv_dtype == SWA_DTYPE_F32 ? 4 : 2;
  NormParams P{};
  P.q = static_cast<const char *>(a.q);
  P.k = static_cast<const char *>(a.k);
  P.v = static_cast<const char *>(a.v);
  P.q_stride = a.q_stride * esz;
  P.k_stride = a.k_stride * esz;
  P.v_stride = a.v_stride * esz;
  P.positions = a.positions;
  P.qw = a.q_weight;
  P.kw = a.k_weight;
  P.eps = a.eps;
  P.cos_sin = a.cos_sin;
  P.max_pos = a.max_pos;
  P.rot = a.rot_dim;
  P.full_loc = a.full_loc;
  P.swa_loc = a.swa_loc;
  P.mapping = c.mapping;
  P.map_len = c.mapping_len;
  P.in_full = L.in_full ? 1 : 0;
  P.pool_rows = (L.in_full ? c.cfg.size_full : c.cfg.size_swa) + c.cfg.page_size;
  P.addr = L.addr;
  P.hq = c.cfg.num_q_heads;
  P.hkv = L.hkv;
  P.k_scale = a.k_scale;
  P.v_scale = a.v_scale;
  P.q_out = static_cast<char *>(a.q_out);
  P.err = c.err_word;
  const int d = c.cfg.head_dim;
  const bool in = a.interleaved;
  using bf = __nv_bfloat16;
  if (c.cfg.kv_dtype == SWA_DTYPE_F32) {
    if (d == 32) return launch_norm<float, 32, false>(c, in, a.n, P, s);
    if (d == 64) return launch_norm<float, 64, false>(c, in, a.n, P, s);
    return launch_norm<float, 128, false>(c, in, a.n, P, s);
  }
  if (c.cfg.kv_dtype == SWA_DTYPE_BF16) {
    if (d == 32) return launch_norm<bf, 32, false>(c, in, a.n, P, s);
    if (d == 64) return launch_norm<bf, 64, false>(c, in, a.n, P, s);
    return launch_norm<bf, 128, false>(c, in, a.n, P, s);
  }
  if (d == 32) return launch_norm<bf, 32, true>(c, in, a.n, P, s);
  if (d == 64) return launch_norm<bf, 64, true>(c, in, a.n, P, s);
  return launch_norm<bf, 128, true>(c, in, a.n, P, s);
}

}  // namespace swa
