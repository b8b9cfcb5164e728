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
// its value heads), so a persistent CTA - four per SM - streams whole tokens
// through a ring of shared-memory stages with bulk copies (one for each of q, k
// and v, and the token's row of the angle table): a hundred KB in flight per SM
// without a register for it.  A producer warp looks positions and slots up 32
// units ahead; four warps take the rows from shared memory.  A row is held by
// D / 8 lanes (bf16) or D / 4 (f32), each with two 8-byte words that hold the
// two halves of its pairs: no value crosses lanes but the row's sum of squares.
// With 1 / rms = rs the pair is
//   rs * (x_a (w_a c) + x_b (-w_b s)),  rs * (x_b (w_b c) + x_a (w_a s)),
// whose bracketed factors a lane computes once per token (its dims are the same
// in every row), so an element costs a product, a fused product-sum and the
// product with rs, two elements at a time (f32x2).
// Measured: 32768 tokens of 64 + 8 + 8 heads, bf16 D = 128 (1.36 GB): 239 us, 5.7
// TB/s (84 % of the copy peak; issue slots 65 % busy); 512 tokens of 64 + 4 + 4:
// 6.3 us; 4099 tokens of 40 + 8 + 8, E4M3 pool: 26.0-26.5 us (its 110 MB take 19 us
// at the first case's rate, the last round of 6.7 tokens per CTA 4 %; the rest is
// start and drain, which nothing overlaps; with products that enclose the quotient
// in place of the divisions by the scale 25.7 us, not worth the second path); f32,
// 32768 tokens of 4 + 1 + 1 heads of 64 (109 MB): 50.6 us, a CTA's two stages
// holding two tokens of 1.5 KB in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_codec.cuh"
#include "spec_internal.h"
#include "tc_ptx.cuh"

namespace swa {
namespace {

constexpr int kNormWarps = 4;      // and a producer warp
constexpr int kNormCtas = 4;       // per SM
constexpr int kNormStages = 2;
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
  int step_t, step_c;    // the grid as tokens and chunks
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
__global__ void __launch_bounds__((kNormWarps + 1) * 32, kNormCtas) k_qk_norm_rope_store(NormParams P) {
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
    const int oa = da * kEsz, ob = db * kEsz;
    float wq[2 * W], wk[2 * W];           // norm weights of the lane's values
#pragma unroll
    for (int i = 0; i < W; ++i) {
      wq[i] = P.qw ? P.qw[da + i] : 1.f;
      wq[W + i] = P.qw ? P.qw[db + i] : 1.f;
      wk[i] = P.kw ? P.kw[da + i] : 1.f;
      wk[W + i] = P.kw ? P.kw[db + i] : 1.f;
    }
    int64_t t = blockIdx.x / P.chunks;
    int c = (int)(blockIdx.x % P.chunks), s = 0;
    uint32_t phase = 0;
    for (int64_t u0 = blockIdx.x; u0 < P.units; u0 += step) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(full(s), phase, &s_abort))) break;
      const NormStage info = s_info[s];
      const int r0 = c * P.chunk_rows, r1 = info.ok ? min(r0 + P.chunk_rows, rows) : 0;
      const char *tile = data(s) - r0 * kRow;           // row r at tile + r * kRow
      // The token's angles at the lane's values (cosine 1, sine 0 where nothing turns).
      float cs[2 * W], sn[2 * W];
      if (turned) {
        const float *ang = reinterpret_cast<const float *>(data(s) + kStageRows);
        if (kInter) {
#pragma unroll
          for (int i = 0; i < 2 * W; i += 2) {
            cs[i] = cs[i + 1] = ang[(da + i) >> 1];
            sn[i + 1] = ang[half + ((da + i) >> 1)];
            sn[i] = -sn[i + 1];
          }
        } else {
#pragma unroll
          for (int i = 0; i < W; i += 2) {
            const float2 x = *reinterpret_cast<const float2 *>(ang + da + i);
            const float2 y = *reinterpret_cast<const float2 *>(ang + half + da + i);
            cs[i] = cs[W + i] = x.x;
            cs[i + 1] = cs[W + i + 1] = x.y;
            sn[W + i] = y.x;
            sn[W + i + 1] = y.y;
            sn[i] = -y.x;
            sn[i + 1] = -y.y;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {
          cs[i] = 1.f;
          sn[i] = 0.f;
        }
      }
      // Rows [lo, hi) of a kind, RPW per pass, the passes of all kinds dealt to
      // the warps in turn: `pass` counts those before, this warp's first row
      // follows.
      int pass = 0;
      auto first_row = [&](int lo, int hi) {
        const int mine = lo + ((warp - pass) & (kNormWarps - 1)) * RPW;
        if (hi > lo) pass += (hi - lo + RPW - 1) / RPW;
        return mine;
      };
#pragma unroll 1
      for (int kd = 0; kd < 2; ++kd) {    // query heads, key heads
        const int lo = kd ? max(r0, nq) : r0, hi = min(r1, kd ? nq + nk : nq);
        int rw = first_row(lo, hi);
        if (rw >= hi) continue;
        // Factors: out_a = x_a fa + z_a ga, out_b = x_b fb + z_b gb, z the pair's
        // other values (halves: the other word; neighbours: swapped in place).
        uint64_t fa[H], ga[H], fb[H], gb[H];
        {
          float f[2 * W], g[2 * W];
#pragma unroll
          for (int i = 0; i < 2 * W; ++i) {
            const int other = kInter ? i ^ 1 : (i + W) % (2 * W);
            f[i] = (kd ? wk[i] : wq[i]) * cs[i];
            g[i] = (kd ? wk[other] : wq[other]) * sn[i];
          }
#pragma unroll
          for (int i = 0; i < H; ++i) {
            fa[i] = tc::f2pack(f[2 * i], f[2 * i + 1]);
            fb[i] = tc::f2pack(f[W + 2 * i], f[W + 2 * i + 1]);
            ga[i] = tc::f2pack(g[2 * i], g[2 * i + 1]);
            gb[i] = tc::f2pack(g[W + 2 * i], g[W + 2 * i + 1]);
          }
        }
        const bool norm = kd ? P.kw != nullptr : P.qw != nullptr;
        const bool keep = kd == 0 || info.base >= 0;
        char *out = kd ? P.addr.k + info.base - (int64_t)nq * (kF8 ? D : kRow)
                       : P.q_out + t * P.hq * kRow;
        const int out_row = kd && kF8 ? D : kRow;
#pragma unroll 2
        for (; rw < hi; rw += kNormWarps * RPW) {
          const int r = rw + sub;
          const bool live = r < hi && keep;
          const char *src = tile + (r < hi ? r : rw) * kRow;
          uint64_t a[H], b[H];
          Wd::get(*reinterpret_cast<const uint2 *>(src + oa), a);
          Wd::get(*reinterpret_cast<const uint2 *>(src + ob), b);
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
          const float rs = norm ? rsqrtf(ss * (1.f / D) + P.eps) : 1.f;
          const uint64_t rs2 = tc::f2pack(rs, rs);
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
                float x, y;
                tc::f2unpack(a[i], x, y);
                za = tc::f2pack(y, x);
                tc::f2unpack(b[i], x, y);
                zb = tc::f2pack(y, x);
              }
              ya[i] = tc::fma2(za, ga[i], ya[i]);
              yb[i] = tc::fma2(zb, gb[i], yb[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < H; ++i) {
            ya[i] = mul2(ya[i], rs2);
            yb[i] = mul2(yb[i], rs2);
          }
          if (live) {
            char *dst = out + r * out_row;
            if (kF8 && kd) {
              if constexpr (kF8) {
                *reinterpret_cast<uint32_t *>(dst + da) = encode4(ya, P.k_scale);
                *reinterpret_cast<uint32_t *>(dst + db) = encode4(yb, P.k_scale);
              }
            } else {
              *reinterpret_cast<uint2 *>(dst + oa) = Wd::put(ya);
              *reinterpret_cast<uint2 *>(dst + ob) = Wd::put(yb);
            }
          }
        }
      }
      {                                   // value heads: stored as they are
        const int lo = max(r0, nq + nk), hi = info.base >= 0 ? r1 : 0;
        for (int rw = first_row(lo, hi); rw < hi; rw += kNormWarps * RPW) {
          const int r = rw + sub;
          if (r >= hi) continue;
          const char *src = tile + r * kRow;
          const uint2 ra = *reinterpret_cast<const uint2 *>(src + oa);
          const uint2 rb = *reinterpret_cast<const uint2 *>(src + ob);
          char *dst = P.addr.v + info.base;
          if constexpr (kF8) {
            dst += (r - nq - nk) * D;
            uint64_t a[H], b[H];
            Wd::get(ra, a);
            Wd::get(rb, b);
            *reinterpret_cast<uint32_t *>(dst + da) = encode4(a, P.v_scale);
            *reinterpret_cast<uint32_t *>(dst + db) = encode4(b, P.v_scale);
          } else {
            dst += (r - nq - nk) * kRow;
            *reinterpret_cast<uint2 *>(dst + oa) = ra;
            *reinterpret_cast<uint2 *>(dst + ob) = rb;
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty(s));
      if (++s == kNormStages) {
        s = 0;
        phase ^= 1;
      }
      t += P.step_t;
      c += P.step_c;
      if (c >= P.chunks) {
        c -= P.chunks;
        ++t;
      }
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
  const int64_t ctas = (int64_t)kNormCtas * (c.num_sms > 0 ? c.num_sms : 148);
  // A chunk is a whole token where that fits a stage and there are tokens for
  // all CTAs; fewer tokens are cut finer, down to 16 rows.
  const int64_t even = (n * rows + ctas - 1) / ctas;
  P.chunk_rows = (int)(even < 16 ? 16 : even < kStageRows / kRow ? even : kStageRows / kRow);
  P.chunks = (rows + P.chunk_rows - 1) / P.chunk_rows;
  P.chunk_rows = (rows + P.chunks - 1) / P.chunks;
  P.units = n * P.chunks;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_qk_norm_rope_store<T, D, kF8, kInter>, kSmem, c.device, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = P.units < ctas ? P.units : ctas;
  P.step_t = (int)(grid / P.chunks);
  P.step_c = (int)(grid % P.chunks);
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
