// k_rows_packed.cu — the row-wise operators of packed batches: QK-RMSNorm with
// rotary positions of several axes per token, and the residual addition with
// the norm behind it (output in fp32, bf16, or e4m3 with one scale per row).
// Both read every element once and hold the row in registers; both are bound
// by HBM.  Measured (B200, graph replays; a copy runs at 6.5 TB/s): QK-norm + rotary of 65520
// rows of 12 + 12 heads 140 us (5.8 TB/s), of 7801 rows of 40 + 40 heads 67 us (4.8); without gains 6.5
// TB/s.  Add + norm of 43745 x 1536, fp32 + bf16 -> fp32 and e4m3, 120 us (6.2 TB/s).
#include "wd_internal.cuh"

#include <cuda_fp8.h>

#include <cmath>

namespace wd {
namespace rows {

// A row is held by wpr = 1 .. 8 warps, each lane with NV <= 4 chunks of 8 elements: few
// registers a thread, so that several blocks share an SM and their loads cover one
// another's arithmetic.  A block has as many rows as fit into 8 warps.
constexpr int THREADS = 256, WARPS = THREADS / 32;   // at most
constexpr int MAX_NV = 4, ROW_MAX = MAX_NV * 8 * THREADS;   // widest row: 8192

// Waits for the wpr warps of one row (barrier 1 + the row's place in the block).
__device__ __forceinline__ void row_sync(int group, int wpr) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(wpr * 32) : "memory");
}

// Eight consecutive elements of type T as fp32 (16-byte accesses; the cache
// hint is "streaming": nothing here is read twice).
template <typename T> struct Chunk;
template <> struct Chunk<float> {
  uint4 u[2];
  __device__ __forceinline__ void load(const float* p) {
    u[0] = __ldcs(reinterpret_cast<const uint4*>(p));
    u[1] = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
  __device__ static __forceinline__ void store(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <> struct Chunk<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_bf16x2(w[i]);
      v[2 * i] = f.x; v[2 * i + 1] = f.y;
    }
  }
  __device__ static __forceinline__ void store(bf16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};
template <> struct Chunk<f16> {
  uint4 u;
  __device__ __forceinline__ void load(const f16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x; v[2 * i + 1] = f.y;
    }
  }
  __device__ static __forceinline__ void store(f16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                                              pack_f16x2(v[6], v[7]));
  }
};

__device__ __forceinline__ void load8f(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Sum (or maximum) of one value per lane over the wpr warps of a row; `red` has one
// float per warp and serves one reduction.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red, int warp, int wpr) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  if (wpr > 1) {
    const int group = warp / wpr;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    row_sync(group, wpr);
    v = red[group * wpr];
    for (int i = 1; i < wpr; ++i) v = MAX ? fmaxf(v, red[group * wpr + i]) : v + red[group * wpr + i];
  }
  return v;
}

// ============================================================ QK-RMSNorm + rotary positions of three axes
// For each token and head, pair p of the head's channels (2p, 2p+1) = (re, im)
// turns by pos[axis(p)] * step[axis] * theta^(-2 p_s / d_s), with p_s counted
// inside the axis's section of d_s channels; before that, with gains, the row
// (all heads) is RMS-normalised.
//
// Angles: one position's share of a turn, f = step * theta^(-2 p_s / d_s) / 2 pi
// mod 1, is held as a 64-bit fraction (made on the host in extended precision).
// pos * f mod 2^64 is then the angle in 2^-64 turns, exact but for f's own
// rounding (|pos| 2^-65 turns), so far positions lose nothing; the quadrant is
// its two leading bits.
constexpr int MAX_PAIRS = 128;   // head width up to 256
struct RopeArgs {
  const int* pos;                     // [rows, 3]
  const void* in[2];
  void* out[2];
  const float* gain[2];
  int64_t in_rs[2], out_rs[2];
  int D[2];                           // heads * dh of each tensor; 0: not given
  float inv_D[2];
  int64_t rows;
  int dh, p1, p2;                     // pairs [0, p1) frame, [p1, p2) row, [p2, dh / 2) column
  float eps;
  uint64_t freq[MAX_PAIRS];
};

// Within an eighth of a turn, |x| <= pi / 4, Taylor's series to x^9 and x^10 leave 1.8e-9
// (x^11 / 11!) and 1.1e-10 (x^12 / 12!), below the fp32 rounding of the sums.
__device__ __forceinline__ float2 turn(int pos, uint64_t f) {
  const uint32_t u = static_cast<uint32_t>((static_cast<uint64_t>(static_cast<int64_t>(pos)) * f) >> 32);
  const uint32_t quad = (u + 0x20000000u) >> 30;                       // nearest quarter turn
  const int rest = static_cast<int>(u - (quad << 30));                 // 2^-32 turns
  const float x = static_cast<float>(rest) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float y = x * x;
  const float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  const float c4 = fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f);
  const float c = fmaf(y, fmaf(y, c4, -0.5f), 1.f);
  const float a = (quad & 1u) ? -s : c, b = (quad & 1u) ? c : s;
  return (quad & 2u) ? make_float2(-a, -b) : make_float2(a, b);
}

// Shapes tried at 65520 x (1536 + 1536): three chunks a lane and two warps 140 us, two chunks and
// three warps 182, one and six 278, six and one 152; two tokens a group of warps, which share
// each load of the gains, 164 and more (fewer blocks an SM); a ring of bulk copies in
// shared memory with 24 computing warps 197 (7801 x (5120 + 5120): 67, 86 with the ring).
// wpr warps take one token, q and then k in the same lanes, and compute the token's
// cosines and sines once into shared memory: dh / 2 of them against heads * dh / 2
// rotations each in q and k.  The rows' loads are issued first.  With SAME (dh
// divides wpr * 256) all chunks of a lane lie at one place of their heads: its four
// cosines and sines are read once, with the row's 1 / rms multiplied in.  FULL: every
// given row has exactly NV chunks a lane, so nothing is compared against its width.
template <typename T, int NV, bool SAME, bool FULL>
__global__ void __launch_bounds__(THREADS, sizeof(T) == 4 ? 2 : (NV == 4 ? 3 : 4))
k_qknorm_rope_axes(const __grid_constant__ RopeArgs a, int wpr) {
  __shared__ __align__(16) float2 cs[WARPS * MAX_PAIRS];   // [token][pair]
  __shared__ float red[2][WARPS];
  const int half = a.dh >> 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = warp / wpr, in_row = (warp - mine * wpr) * 32 + lane;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (WARPS / wpr) + mine;
  if (row >= a.rows) return;   // the token's warps leave together
  Chunk<T> ch[2][NV];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const T* x = static_cast<const T*>(a.in[t]) + row * a.in_rs[t] + in_row * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (FULL ? a.D[t] > 0 : (i * wpr * 32 + in_row) * 8 < a.D[t]) ch[t][i].load(x + i * wpr * 256);
  }
  float2* tab = cs + mine * half;
  for (int p = in_row; p < half; p += wpr * 32)
    tab[p] = turn(a.pos[row * 3 + (p < a.p1 ? 0 : (p < a.p2 ? 1 : 2))], a.freq[p]);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if (!a.gain[t]) continue;
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (FULL || (i * wpr * 32 + in_row) * 8 < a.D[t]) {
        float v[8];
        ch[t][i].get(v);
#pragma unroll
        for (int k = 0; k < 8; k += 2) ss = ffma2(make_float2(v[k], v[k + 1]), make_float2(v[k], v[k + 1]), ss);
      }
    }
    float s = ss.x + ss.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) red[t][warp] = s;
  }
  row_sync(mine, wpr);   // the angles, and the warps' sums
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float* gain = a.gain[t] ? a.gain[t] + in_row * 8 : nullptr;
    float r = 1.f;
    if (gain) {
      float s = 0.f;
      for (int i = 0; i < wpr; ++i) s += red[t][mine * wpr + i];
      r = rsqrtf(fmaf(s, a.inv_D[t], a.eps));
    }
    // cos, sin of the four pairs at channel c of a head, times r
    auto angles = [&](int c, float2 (&w)[4]) {
      const float4* t4 = reinterpret_cast<const float4*>(tab + (c >> 1));
      const float4 x = t4[0], y = t4[1];
      w[0] = make_float2(x.x * r, x.y * r);
      w[1] = make_float2(x.z * r, x.w * r);
      w[2] = make_float2(y.x * r, y.y * r);
      w[3] = make_float2(y.z * r, y.w * r);
    };
    float2 w[4];
    if constexpr (SAME) angles((in_row * 8) % a.dh, w);
    T* y = static_cast<T*>(a.out[t]) + row * a.out_rs[t] + in_row * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * wpr * 32 + in_row) * 8;
      if (FULL ? a.D[t] == 0 : c >= a.D[t]) break;
      if constexpr (!SAME) angles(c % a.dh, w);
      float v[8];
      ch[t][i].get(v);
      if (gain) {
        float g[8];
        load8f(gain + i * wpr * 256, g);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float2 n = fmul2(make_float2(v[k], v[k + 1]), make_float2(g[k], g[k + 1]));
          v[k] = n.x;
          v[k + 1] = n.y;
        }
      }
      float o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[2 * k] = v[2 * k] * w[k].x - v[2 * k + 1] * w[k].y;
        o[2 * k + 1] = v[2 * k] * w[k].y + v[2 * k + 1] * w[k].x;
      }
      Chunk<T>::store(y + i * wpr * 256, o);
    }
  }
}

// ============================================================ residual addition + norm
// s = x + y; n = norm(s) * gain + beta per row, with the statistics and n taken
// from the fp32 sum; s is stored in x's type, n in fp32, bf16 or e4m3 (codes
// e4m3(n / scale), scale = amax / 448, as k_quant_rows_e4m3).  LayerNorm's
// variance is summed after the mean is known (the row is in registers), so no
// difference of large numbers is taken.
struct AddNormArgs {
  const void *x, *y;      // y null: no addition
  const float *gain, *beta;
  void *sum, *out;        // sum null: not stored
  float* scale;
  int64_t rows;
  int D, rms;
  float eps;
};

template <typename TX, typename TY, typename TO, int NV>
__global__ void __launch_bounds__(THREADS) k_add_norm(const AddNormArgs a, int wpr) {
  constexpr bool Q = std::is_same<TO, uint8_t>::value;
  __shared__ float red[3][WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int in_row = (warp % wpr) * 32 + lane;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (WARPS / wpr) + warp / wpr;
  if (row >= a.rows) return;        // the row's warps leave together
  const int D = a.D;
  const int64_t base = row * D;
  float v[NV][8];
  {
    Chunk<TX> cx[NV];
    Chunk<TY> cy[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * wpr * 32 + in_row) * 8;
      if (c < D) cx[i].load(static_cast<const TX*>(a.x) + base + c);
    }
    if (a.y) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * wpr * 32 + in_row) * 8;
        if (c < D) cy[i].load(static_cast<const TY*>(a.y) + base + c);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * wpr * 32 + in_row) * 8;
      if (c < D) {
        cx[i].get(v[i]);
        if (a.y) {
          float w[8];
          cy[i].get(w);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i][k] += w[k];
        }
        if (a.sum) Chunk<TX>::store(static_cast<TX*>(a.sum) + base + c, v[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
      }
    }
  }
  float mean = 0.f;
  if (!a.rms) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[i][k];
    mean = row_reduce<false>(s, red[0], warp, wpr) / D;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * wpr * 32 + in_row) * 8;
    if (c < D) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][k] -= mean;
        q += v[i][k] * v[i][k];
      }
    }
  }
  const float rstd = rsqrtf(row_reduce<false>(q, red[1], warp, wpr) / D + a.eps);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * wpr * 32 + in_row) * 8;
    if (c < D) {
      float g[8];
      if (a.gain) {
        load8f(a.gain + c, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = v[i][k] * rstd * g[k];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] *= rstd;
      }
      if (a.beta) {
        load8f(a.beta + c, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] += g[k];
      }
      if constexpr (Q) {
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(v[i][k]));
      } else {
        Chunk<TO>::store(static_cast<TO*>(a.out) + base + c, v[i]);
      }
    }
  }
  if constexpr (Q) {
    amax = row_reduce<true>(amax, red[2], warp, wpr);
    const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * wpr * 32 + in_row) * 8;
      if (c < D) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; k += 2)
          w[k >> 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                           make_float2(__fdiv_rn(v[i][k], sc), __fdiv_rn(v[i][k + 1], sc)), __NV_SATFINITE, __NV_E4M3))
                       << (8 * (k & 3));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + base + c) = make_uint2(w[0], w[1]);
      }
    }
    if (in_row == 0) a.scale[row] = sc;
  }
}

}  // namespace rows

// ------------------------------------------------------------------ host side
// How rows of D elements are laid out: nv chunks a lane and wpr warps that hold the row
// exactly, with the fewest warps, or else a power of two of warps that holds it.  Exact layouts
// of one or two chunks a lane are the slow ones (bf16, GB/s of add + norm / QK-norm + rotary, cold): one
// chunk, 1280 2905 / 2246 and 1792 3758 / 2891; two, 2560 4581 / 3734 and 3584 5329 / 4285; three and
// four, 1536 6280 / 4970, 2048 6522 / 5381, 4096 6443 / 5331, 5120 5798 / 5074, 7168 6355 / 4930.
struct RowShape {
  int wpr, nv;
  bool exact;
  int rows() const { return rows::WARPS / wpr; }           // of a block
  unsigned threads() const { return static_cast<unsigned>(rows() * wpr * 32); }
  unsigned blocks(int64_t n) const { return static_cast<unsigned>((n + rows() - 1) / rows()); }
};
static RowShape row_shape(int D) {
  for (int nv = rows::MAX_NV; nv > 0; --nv)
    if (D % (nv * 256) == 0 && D / (nv * 256) <= rows::WARPS) return {D / (nv * 256), nv, true};
  int w = 1;
  while (w * 256 * rows::MAX_NV < D) w *= 2;
  return {w, (D + w * 256 - 1) / (w * 256), false};
}

// f(integral constant nv)
template <typename F>
static void with_chunks(int nv, F&& f) {
  switch (nv) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 3: f(std::integral_constant<int, 3>()); break;
    default: f(std::integral_constant<int, 4>()); break;
  }
}

template <typename T>
static wd_status qknorm_rope_axes(const rows::RopeArgs& a, cudaStream_t st) {
  const RowShape r = row_shape(a.D[1] > a.D[0] ? a.D[1] : a.D[0]);
  const bool full = r.exact && (a.D[1] == 0 || a.D[1] == a.D[0]);
  const unsigned grid = r.blocks(a.rows), threads = r.threads();
  Trace tr(KC_ROPE, st);
  with_chunks(r.nv, [&](auto nv) {
    if (r.wpr * 256 % a.dh) rows::k_qknorm_rope_axes<T, nv(), false, false><<<grid, threads, 0, st>>>(a, r.wpr);
    else if (full) rows::k_qknorm_rope_axes<T, nv(), true, true><<<grid, threads, 0, st>>>(a, r.wpr);
    else rows::k_qknorm_rope_axes<T, nv(), true, false><<<grid, threads, 0, st>>>(a, r.wpr);
  });
  return launch_status("qknorm_rope_axes");
}

template <typename TX, typename TY, typename TO>
static wd_status add_norm_t(const rows::AddNormArgs& a, cudaStream_t st) {
  const RowShape r = row_shape(a.D);
  Trace tr(KC_NORM, st);
  with_chunks(r.nv, [&](auto nv) {
    rows::k_add_norm<TX, TY, TO, nv()><<<r.blocks(a.rows), r.threads(), 0, st>>>(a, r.wpr);
  });
  return launch_status("add_norm");
}

template <typename TX, typename TY>
static wd_status add_norm_o(const rows::AddNormArgs& a, int out_dtype, cudaStream_t st) {
  if (out_dtype == WD_F32) return add_norm_t<TX, TY, float>(a, st);
  if (out_dtype == WD_BF16) return add_norm_t<TX, TY, bf16>(a, st);
  return add_norm_t<TX, TY, uint8_t>(a, st);
}

static wd_status add_norm(const rows::AddNormArgs& a, int x_dtype, int y_dtype, int out_dtype, cudaStream_t st) {
  if (x_dtype == WD_F32)
    return y_dtype == WD_F32 ? add_norm_o<float, float>(a, out_dtype, st) : add_norm_o<float, bf16>(a, out_dtype, st);
  return y_dtype == WD_F32 ? add_norm_o<bf16, float>(a, out_dtype, st) : add_norm_o<bf16, bf16>(a, out_dtype, st);
}

}  // namespace wd
