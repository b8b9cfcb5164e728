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
// The pass is bound by HBM: (Hq + 2 Hkv) D values read, Hq D + 2 Hkv D
// written per token.  One CTA per token: a row is held by D / 8 lanes (bf16;
// 16 bytes each) or D / 4 (f32), so a warp takes 32 / that many head rows at a
// time and its lanes keep the same dims of every row they meet: the angle
// table's row and the norm weights are loaded once per token into registers.
// The row's sum of squares and, for halves paired across lanes, the partner
// values come by shuffle.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_codec.cuh"
#include "spec_internal.h"

namespace swa {
namespace {

constexpr int kNormThreads = 256;
constexpr int kRows = 4;           // rows of one lane group in flight

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
};

template <typename T> struct Lane;      // the values of one 16-byte word
template <> struct Lane<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4 &w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <> struct Lane<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4 &w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// One token: rows 0 .. hq - 1 are query heads, then the key heads, then the
// value heads (an absent input has no rows).
template <typename T, int D, bool kF8, bool kInter>
__global__ void __launch_bounds__(kNormThreads) k_qk_norm_rope_store(NormParams P) {
  using Ln = Lane<T>;
  constexpr int N = Ln::kN;
  constexpr int LPR = D / N;              // lanes of a row
  constexpr int RPW = 32 / LPR;           // rows of a warp
  constexpr int kGroups = kNormThreads / 32 * RPW;
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, li = lane % LPR, d0 = li * N;
  const int nq = P.q ? P.hq : 0, nk = P.k ? P.hkv : 0, nv = P.v ? P.hkv : 0;

  // The token's angles, for this lane's dims.
  float cs[N], sn[N];
  const int half = P.rot >> 1;
  const bool turned = d0 < P.rot;         // rot is a multiple of 2 N: whole words
  int partner = lane;                     // lane with the other value of each pair
  if (P.rot > 0) {
    const int64_t pos = P.positions[t];
    if (pos < 0 || pos >= P.max_pos) {
      if (threadIdx.x == 0) set_error(P.err, SWA_DEVERR_RANGE);
      return;                             // block-uniform
    }
    const float *row = P.cos_sin + pos * P.rot;
    if (turned) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int a = kInter ? (d0 + i) >> 1 : (d0 < half ? d0 + i : d0 + i - half);
        const bool second = kInter ? (i & 1) : d0 >= half;
        cs[i] = row[a];
        sn[i] = second ? row[half + a] : -row[half + a];
      }
      if (!kInter) partner = lane + (d0 < half ? half : -half) / N;
    }
  }
  float wq[N], wk[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    wq[i] = P.qw ? P.qw[d0 + i] : 1.f;
    wk[i] = P.kw ? P.kw[d0 + i] : 1.f;
  }
  // The pool row of the token's K and V.
  int64_t base = -1;
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
    if (slot < 0 || slot >= P.pool_rows) {
      if (threadIdx.x == 0) set_error(P.err, SWA_DEVERR_RANGE);
    } else {
      base = kv_row(P.addr, slot) * P.addr.row_bytes;
    }
  }
  const int total = nq + nk + nv;
  // Rows r0, r0 + kGroups, ... of this lane group, kRows of them loaded together.
  for (int r0 = warp * RPW; r0 < total; r0 += kRows * kGroups) {
    uint4 w[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * kGroups + sub;
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < total) {
        const char *src = r < nq ? P.q + t * P.q_stride + (int64_t)r * D * sizeof(T)
                          : r < nq + nk
                              ? P.k + t * P.k_stride + (int64_t)(r - nq) * D * sizeof(T)
                              : P.v + t * P.v_stride + (int64_t)(r - nq - nk) * D * sizeof(T);
        w[u] = *reinterpret_cast<const uint4 *>(src + d0 * sizeof(T));
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int ru = r0 + u * kGroups;     // warp-uniform
      if (ru >= total) break;
      const int r = ru + sub;
      const bool is_v = r >= nq + nk, is_k = r >= nq && !is_v;
      float x[N];
      Ln::get(w[u], x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) ss += x[i] * x[i];
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      float y[N];
      const bool norm = is_k ? P.kw != nullptr : P.qw != nullptr;
      const float rs = norm ? rsqrtf(ss * (1.f / D) + P.eps) : 1.f;
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = x[i] * rs * (is_k ? wk[i] : wq[i]);
      if (P.rot > 0) {
        float z[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
          z[i] = kInter ? y[i ^ 1] : __shfl_sync(0xffffffffu, y[i], partner);
        if (turned) {
#pragma unroll
          for (int i = 0; i < N; ++i) y[i] = y[i] * cs[i] + z[i] * sn[i];
        }
      }
      if (r >= total) continue;
      if (r < nq) {
        *reinterpret_cast<uint4 *>(P.q_out + ((t * P.hq + r) * D + d0) * (int64_t)sizeof(T)) =
            Ln::put(y);
      } else if (base >= 0) {
        if (is_v) {
#pragma unroll
          for (int i = 0; i < N; ++i) y[i] = x[i];
        }
        const int h = is_v ? r - nq - nk : r - nq;
        char *dst = (is_v ? P.addr.v : P.addr.k) + base;
        if constexpr (kF8) {
          const float sc = is_v ? P.v_scale : P.k_scale;
          uint32_t o[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            o[j] = pack_e4m3x4(__fdiv_rn(y[4 * j], sc), __fdiv_rn(y[4 * j + 1], sc),
                               __fdiv_rn(y[4 * j + 2], sc), __fdiv_rn(y[4 * j + 3], sc));
          *reinterpret_cast<uint2 *>(dst + h * D + d0) = make_uint2(o[0], o[1]);
        } else {
          *reinterpret_cast<uint4 *>(dst + (h * D + d0) * (int64_t)sizeof(T)) =
              is_v ? w[u] : Ln::put(y);
        }
      }
    }
  }
}

template <typename T, int D, bool kF8>
void launch_norm(bool inter, int64_t n, const NormParams &P, cudaStream_t s) {
  if (inter) k_qk_norm_rope_store<T, D, kF8, true><<<(unsigned)n, kNormThreads, 0, s>>>(P);
  else k_qk_norm_rope_store<T, D, kF8, false><<<(unsigned)n, kNormThreads, 0, s>>>(P);
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
    if (d == 32) launch_norm<float, 32, false>(in, a.n, P, s);
    else if (d == 64) launch_norm<float, 64, false>(in, a.n, P, s);
    else launch_norm<float, 128, false>(in, a.n, P, s);
  } else if (c.cfg.kv_dtype == SWA_DTYPE_BF16) {
    if (d == 32) launch_norm<bf, 32, false>(in, a.n, P, s);
    else if (d == 64) launch_norm<bf, 64, false>(in, a.n, P, s);
    else launch_norm<bf, 128, false>(in, a.n, P, s);
  } else {
    if (d == 32) launch_norm<bf, 32, true>(in, a.n, P, s);
    else if (d == 64) launch_norm<bf, 64, true>(in, a.n, P, s);
    else launch_norm<bf, 128, true>(in, a.n, P, s);
  }
  return cudaGetLastError();
}

}  // namespace swa
