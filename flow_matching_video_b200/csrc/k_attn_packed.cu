// k_attn_packed.cu — attention over packed sequences on the sm_100a tensor cores:
// sequence s owns query rows [cu_q[s], cu_q[s+1]) and keys [cu_k[s], cu_k[s+1]) of
// buffers that hold all sequences one behind the other, and
//   o_i = sum_j softmax_j(scale q_i k_j + b[h, clamp(j - i, -R, R)]) v_j
// over the keys of i's own sequence (i, j counted from its first row).  Query
// heads share kv_heads key/value heads in equal groups.
//
// The pipeline is that of k_attn_tc.cu: a block owns two query tiles of 128 rows of
// one sequence and head; warp 0 loads Q and then K_j, V_j by TMA through a ring,
// warp 1 issues S_t = Q_t K_j^T and O_t += P_t V_j (P from TMEM), and one softmax
// warp per 32 rows keeps the running maximum and sum, so the tiles' softmaxes and
// products alternate.  What packing adds:
//  - blocks find their (sequence, tile) by a scan over cu_q; the grid has the
//    largest number of tiles that q_rows rows in n_seq sequences can make, and
//    blocks without a tile leave at once;
//  - a sequence's last key block runs into the next sequence's rows (the TMA clips
//    at the end of the buffer only).  Its scores behind the end become -inf before
//    anything reads them, and its V rows are overwritten with zeros in shared
//    memory before the product, since 0 * NaN of a neighbour would not be 0;
//  - the second tile of a block may lie behind the sequence's end: it is left out
//    of every role.
// The bias table of the head sits in shared memory in log2 units, its ends
// repeated 160 times so that no index needs clamping; a block of keys that lies R
// or further from all of a warp's rows takes the one end value instead.  Where an
// end value is -inf, key blocks wholly behind it are neither loaded nor multiplied.
#include "wd_internal.cuh"

namespace wd {
namespace pka {

constexpr int BQ = 128, BK = 128, NQ = 2;
constexpr int MAX_RADIUS = 1024, PAD = 160;   // PAD >= 127 + 31 + 1: a tile's reach past +-R
constexpr float LOG2E = 1.4426950408889634f;

template <int DH, typename TI>
struct Cfg {
  static constexpr int Q_BYTES = BQ * DH * 2, KV_BYTES = BK * DH * 2;
  static constexpr int HALVES = DH / 64, HALF_BYTES = 128 * 128;   // 64 columns of 128 rows
  static constexpr int RING = 131072 / KV_BYTES;                   // K/V tiles in flight
  static constexpr int THREADS = 64 + 128 * NQ;
  static constexpr int BIAS_FLOATS = 2 * (MAX_RADIUS + PAD) + 4;
  static constexpr int Q_OFF = 0, RING_OFF = NQ * Q_BYTES, BIAS_OFF = RING_OFF + RING * KV_BYTES;
  static constexpr int BAR_OFF = BIAS_OFF + BIAS_FLOATS * 4;
  static constexpr int SMEM = 1024 + BAR_OFF + 512;
  static_assert(BAR_OFF % 8 == 0 && SMEM <= 232448, "shared memory of one block");
  __host__ __device__ static constexpr int s_col(int t) { return 256 * t; }
  __host__ __device__ static constexpr int o_col(int t) { return 256 * t + 128; }
  static constexpr bool HALF = std::is_same<TI, f16>::value;
  static constexpr uint32_t IDESC_S = HALF ? idesc_f16(128, BK, 0, 0) : idesc_bf16(128, BK, 0, 0);
  static constexpr uint32_t IDESC_O = HALF ? idesc_f16(128, DH, 0, 1) : idesc_bf16(128, DH, 0, 1);
};

enum : unsigned { SITE_Q = 0x501, SITE_KVF = 0x502, SITE_KVE = 0x503, SITE_S = 0x504, SITE_P = 0x505, SITE_O = 0x506,
                  SITE_TAIL = 0x507, SITE_DRAIN = 0x508 };

struct Params {
  const int *cu_q, *cu_k;
  int n_seq, q_rows, k_rows;
  int group;             // query heads per key/value head
  int heads;
  float scale_log2;      // scale * log2(e)
  const float* bias;     // [heads, 2 R + 1] or null
  int radius;
  bf16* o;
  int64_t o_rs;
};

// max that keeps a NaN (a row with a NaN score ends as NaN instead of skipping it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float o;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
  return o;
}

// Rows [lo, hi) of sequence s, inside the buffer whatever the offsets say.
__device__ __forceinline__ int2 extent(const int* cu, int s, int rows) {
  const int lo = min(max(cu[s], 0), rows);
  return make_int2(lo, max(min(cu[s + 1], rows), lo));
}

template <int DH, typename TI, bool BIAS>
__global__ void __launch_bounds__(Cfg<DH, TI>::THREADS, 1)
k_attn_packed(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using C = Cfg<DH, TI>;
  constexpr int RING = C::RING;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* tab = reinterpret_cast<float*>(smem + C::BIAS_OFF);   // tab[d + R + PAD] = bias at distance d
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* q_full = bars;
  uint64_t* tail = bars + 1;              // the last V tile has landed (before its rows are cleared)
  uint64_t* kv_full = bars + 2;           // RING
  uint64_t* kv_empty = kv_full + RING;    // RING
  uint64_t* s_full = kv_empty + RING;     // NQ
  uint64_t* p_part = s_full + NQ;         // NQ: the first 64 keys of P written
  uint64_t* p_full = p_part + NQ;         // NQ: all of P written
  uint64_t* o_done = p_full + NQ;         // NQ
  uint64_t* tdone = o_done + NQ;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tdone + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y;

  // ---------------------------------------------------------- which sequence and tile
  int seq = -1, l0 = 0;
  int2 eq = make_int2(0, 0);
  for (int s0 = 0, left = blockIdx.x; s0 < p.n_seq; s0 += 32) {
    const int s = s0 + lane;
    const int2 e = s < p.n_seq ? extent(p.cu_q, s, p.q_rows) : make_int2(0, 0);
    const int mine = (e.y - e.x + NQ * BQ - 1) / (NQ * BQ);
    int upto = mine;   // tiles of sequences s0 .. s
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, upto > left);
    if (hit) {
      const int src = __ffs(hit) - 1;
      seq = s0 + src;
      eq.x = __shfl_sync(0xffffffffu, e.x, src);
      eq.y = __shfl_sync(0xffffffffu, e.y, src);
      l0 = (left - __shfl_sync(0xffffffffu, upto - mine, src)) * NQ * BQ;
      break;
    }
    left -= __shfl_sync(0xffffffffu, upto, 31);
  }
  if (seq < 0) return;
  const int2 ek = extent(p.cu_k, seq, p.k_rows);
  const int lq = eq.y - eq.x, lk = ek.y - ek.x;
  const int nt = lq - l0 > BQ ? 2 : 1;                     // tiles with rows
  const int l1 = min(l0 + NQ * BQ, lq);
  // key blocks [n_lo, n_hi): all, or those that some row sees when an end of the table is -inf
  int n_lo = 0, n_hi = (lk + BK - 1) / BK;
  float far_lo = 0.f, far_hi = 0.f;                        // the ends of the table, log2 units
  const int R = p.radius;
  auto log2_units = [](float b) {   // finite values kept finite: they absorb any score either way
    return isinf(b) ? b : fminf(fmaxf(b * LOG2E, -1e30f), 1e30f);
  };
  if constexpr (BIAS) {
    const float* tb = p.bias + static_cast<int64_t>(h) * (2 * R + 1);
    far_lo = log2_units(tb[0]);
    far_hi = log2_units(tb[2 * R]);
    if (far_lo == -INFINITY) n_lo = max(0, l0 - R + 1) / BK;
    if (far_hi == -INFINITY) n_hi = min(n_hi, (l1 - 1 + R - 1) / BK + 1);
    for (int i = threadIdx.x; i < 2 * (R + PAD) + 1; i += C::THREADS)
      tab[i] = log2_units(tb[min(max(i - PAD, 0), 2 * R)]);
  }
  const int NB = n_hi - n_lo;
  if (NB <= 0) {   // no row of these tiles sees a key: zeros
    for (int i = threadIdx.x; i < (l1 - l0) * (DH / 8); i += C::THREADS) {
      const int64_t row = eq.x + l0 + i / (DH / 8);
      reinterpret_cast<uint4*>(p.o + row * p.o_rs + h * DH)[i % (DH / 8)] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(tail, 1);
    for (int s = 0; s < RING; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 1); }
    for (int t = 0; t < NQ; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_part[t], 4);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(tdone, 1);
    fence_mbar_init();
  }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA loader
    const int kvc = h / p.group * DH;
    const int rest = lk - (n_hi - 1) * BK;   // keys of the last block that are the sequence's
    uint32_t issued = 0, last_par = 0;
    bool ok = true;
    auto load = [&](int i, const CUtensorMap* tm, int row, uint64_t* bar) {   // ring position i
      uint8_t* dst = smem + C::RING_OFF + (i % RING) * C::KV_BYTES;
      mbar_arrive_expect_tx(bar, C::KV_BYTES);
      for (int hf = 0; hf < C::HALVES; ++hf) tma_load_3d(dst + hf * C::HALF_BYTES, tm, kvc + hf * 64, row, 0, bar);
    };
    auto ring = [&](int i, const CUtensorMap* tm, int row) -> bool {
      const int slot = i % RING;
      const uint32_t ph = (i / RING) & 1u;
      if (!mbar_wait(&kv_empty[slot], ph ^ 1u, SITE_KVE)) return false;
      load(i, tm, row, &kv_full[slot]);
      issued |= 1u << slot;
      last_par = (last_par & ~(1u << slot)) | (ph << slot);
      return true;
    };
    const bool clear = rest < BK;
    const int last = 2 * NB - 1;             // ring position of the last V tile
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, nt * C::Q_BYTES);
      for (int t = 0; t < nt; ++t)
        for (int hf = 0; hf < C::HALVES; ++hf)
          tma_load_3d(smem + C::Q_OFF + t * C::Q_BYTES + hf * C::HALF_BYTES, &tmQ, h * DH + hf * 64, eq.x + l0 + t * BQ,
                      0, q_full);
      for (int i = 0; i < (clear ? last : last + 1) && ok; ++i)
        ok = ring(i, (i & 1) ? &tmV : &tmK, ek.x + (n_lo + (i >> 1)) * BK);
      if (clear && ok) {   // the last V tile lands on its own barrier
        ok = mbar_wait(&kv_empty[last % RING], ((last / RING) & 1u) ^ 1u, SITE_KVE);
        if (ok) load(last, &tmV, ek.x + (n_hi - 1) * BK, tail);
        issued &= ~(1u << (last % RING));   // what that slot held before has been used; `tail` is waited for below
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (clear && ok) {
      // rows [rest, 128) of it to zero: a row is the same 128 bytes of each half in any swizzle
      ok = mbar_wait_warp(tail, 0, SITE_TAIL);
      uint8_t* dst = smem + C::RING_OFF + (last % RING) * C::KV_BYTES;
      for (int hf = 0; hf < C::HALVES; ++hf)
        for (int i = rest * 8 + lane; i < BK * 8; i += 32)
          reinterpret_cast<uint4*>(dst + hf * C::HALF_BYTES)[i] = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&kv_full[last % RING]);
    }
    if (lane == 0) {
      mbar_wait(q_full, 0, SITE_DRAIN);
      for (int s = 0; s < RING; ++s)
        if (issued & (1u << s)) mbar_wait(&kv_full[s], (last_par >> s) & 1u, SITE_DRAIN);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      bool ok = mbar_wait(q_full, 0, SITE_Q);
      tc_fence_after();
      // descriptors as fixed high halves and low halves that step by 16-byte units
      const uint32_t r0 = smem_u32(smem + C::RING_OFF);
      const uint64_t dq0 = sdesc_sw128(smem_u32(smem + C::Q_OFF), 16, 1024), dk0 = sdesc_sw128(r0, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(r0, C::HALF_BYTES, 1024);
      const uint32_t q_lo = static_cast<uint32_t>(dq0), k_lo = static_cast<uint32_t>(dk0), v_lo = static_cast<uint32_t>(dv0);
      const uint32_t s_hi = static_cast<uint32_t>(dq0 >> 32), v_hi = static_cast<uint32_t>(dv0 >> 32);
      auto issue_s = [&](int t, int n) {
        const uint32_t kb = k_lo + ((2 * n) % RING) * (C::KV_BYTES >> 4), qa = q_lo + t * (C::Q_BYTES >> 4);
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::HALF_BYTES + (kk & 3) * 32) >> 4;
          umma_ss_lh(tmem + C::s_col(t), qa + off, s_hi, kb + off, s_hi, C::IDESC_S, kk ? 1u : 0u);
        }
        umma_commit(&s_full[t]);
      };
      auto issue_pv = [&](int t, int n) -> bool {
        const int i = 2 * n + 1, slot = i % RING;
        const uint32_t vb = v_lo + slot * (C::KV_BYTES >> 4);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (!mbar_wait(part ? &p_full[t] : &p_part[t], n & 1u, SITE_P)) return false;
          if (part == 0 && t == 0 && !mbar_wait(&kv_full[slot], (i / RING) & 1u, SITE_KVF)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = part * 4; kk < part * 4 + 4; ++kk)
            umma_ts_lh(tmem + C::o_col(t), tmem + C::s_col(t) + kk * 8, vb + kk * (2048 >> 4), v_hi, C::IDESC_O,
                       (n | kk) ? 1u : 0u);
        }
        if (t == nt - 1) umma_commit(&kv_empty[slot]);
        return true;
      };
      for (int n = 0; n < NB && ok; ++n) {
        for (int t = 0; t < nt && ok; ++t) {
          if (n > 0 && !issue_pv(t, n - 1)) { ok = false; break; }
          if (t == 0) {
            ok = mbar_wait(&kv_full[(2 * n) % RING], ((2 * n) / RING) & 1u, SITE_KVF);
            tc_fence_after();
          }
          if (ok) issue_s(t, n);
        }
        if (ok) umma_commit(&kv_empty[(2 * n) % RING]);
      }
      for (int t = 0; t < nt && ok; ++t) {
        ok = issue_pv(t, NB - 1);
        if (ok) umma_commit(&o_done[t]);
      }
      umma_commit(tdone);
      mbar_wait(tdone, 0, SITE_DRAIN);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warps
    const int t = (warp - 2) >> 2, quarter = warp & 3;
    const int i_w = l0 + t * BQ + quarter * 32;            // the warp's first row
    const int i = i_w + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lanes + C::s_col(t), o_addr = tmem + lanes + C::o_col(t);
    float m = -INFINITY, l = 0.f;
    bool ok = t < nt;
    for (int n = 0; n < NB && ok; ++n) {
      const int j0 = (n_lo + n) * BK;
      if (!mbar_wait_warp(&s_full[t], n & 1u, SITE_S)) { ok = false; break; }
      tc_fence_after();
      uint32_t a[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, a[c]);
      tmem_wait_ld();
      if constexpr (BIAS) {   // a = scale * s + bias, log2 units
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        const bool past = j0 - i_w - 31 >= R, before = j0 + BK - 1 - i_w <= -R;   // warp-uniform
        const float* tj = tab + (j0 - i + R + PAD);
        const float cb = past ? far_hi : far_lo;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float2 b = make_float2(cb, cb);
            if (!past && !before) b = make_float2(tj[c * 32 + k], tj[c * 32 + k + 1]);
            const float2 x = ffma2(make_float2(__uint_as_float(a[c][k]), __uint_as_float(a[c][k + 1])), sc2, b);
            a[c][k] = __float_as_uint(x.x);
            a[c][k + 1] = __float_as_uint(x.y);
          }
      }
      const int valid = lk - j0;
      if (valid < BK) {   // keys behind the sequence's end
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (c * 32 + k >= valid) a[c][k] = __float_as_uint(-INFINITY);
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < 32; ++k) m4[k & 3] = max_nan(m4[k & 3], __uint_as_float(a[c][k]));
      float mx = max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3]));
      if constexpr (!BIAS) mx *= p.scale_log2;
      if (mx == INFINITY) mx = NAN;   // inf - inf below: the row is NaN, whichever pipe its exponentials take
      // the reference moves only when the maximum grew by more than the threshold (or is NaN);
      // P stays below 2^8 and the final 1 / l keeps the result exact
      const bool grow = !(mx <= m + tca::RESCALE_THRESHOLD);
      const float alpha = grow ? tca::ex2(m - mx) : 1.f;
      if (grow) m = mx;
      if (__any_sync(0xffffffffu, grow) && n > 0) {
        // P V of the block before has completed: its commit precedes the S waited for
#pragma unroll 1
        for (int c = 0; c < DH / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_addr + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tmem_st32(o_addr + c * 32, o);
        }
        tmem_wait_st();
      }
      // a row that has seen nothing yet has no reference: its exponentials are those of -inf - 0
      const float ref = m == -INFINITY ? 0.f : m;
      const float2 nm2 = make_float2(-ref, -ref), sc2 = make_float2(p.scale_log2, p.scale_log2);
      float2 rs[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 8; ++c) {   // 16 keys: two in eight exponentials on the FMA pipe (k_attn_tc.cu)
        uint32_t pk[8];
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const float2 s2 = make_float2(__uint_as_float(a[c >> 1][(c & 1) * 16 + k]),
                                        __uint_as_float(a[c >> 1][(c & 1) * 16 + k + 1]));
          const float2 arg = BIAS ? fadd2(s2, nm2) : ffma2(s2, sc2, nm2);
          const float2 e = (k & 7) == 6 ? tca::exp2_fma2(arg) : make_float2(tca::ex2(arg.x), tca::ex2(arg.y));
          rs[(k >> 1) & 3] = fadd2(rs[(k >> 1) & 3], e);
          pk[k >> 1] = C::HALF ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
        }
        tmem_st8(s_addr + c * 8, pk);
        if (c == 3) {   // the first 64 keys' product can start
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_part[t]);
        }
      }
      tmem_wait_st();
      const float2 r2 = fadd2(fadd2(rs[0], rs[1]), fadd2(rs[2], rs[3]));
      l = l * alpha + (r2.x + r2.y);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t]);
    }
    // ---------------------------------------------------------- output
    if (ok && mbar_wait_warp(&o_done[t], 0, SITE_O)) {
      tc_fence_after();
      const bool dead = m == -INFINITY;   // every score -inf: the row sees nothing
      const float inv = 1.f / l;
      bf16* dst = p.o + (static_cast<int64_t>(eq.x) + i) * p.o_rs + h * DH;
#pragma unroll 1
      for (int c = 0; c < DH / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o_addr + c * 32, o);
        tmem_wait_ld();
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = dead ? 0.f : __uint_as_float(o[k]) * inv;
        if (i < lq) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + c * 32);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            d4[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                               pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace pka

// ------------------------------------------------------------------ host side
// 2D tensor map over [rows, cols] two-byte elements (row stride rs elements), box 64 columns x 128 rows.
static wd_status make_tmap_rows(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t rows, int64_t cols,
                                int64_t rs) {
  return make_tmap_3d(m, type, base, cols, rows, 1, rs, 0);
}

template <int DH, typename TI, bool BIAS>
static wd_status launch_attn_packed(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                    const pka::Params& p, cudaStream_t st) {
  using C = pka::Cfg<DH, TI>;
  WD_TRY((allow_smem<pka::k_attn_packed<DH, TI, BIAS>>(C::SMEM)));
  const int64_t slots = p.q_rows / (pka::NQ * pka::BQ) + static_cast<int64_t>(p.n_seq);
  dim3 grid(static_cast<unsigned>(slots), p.heads);
  Trace tr(KC_ATTN_SELF, st);
  pka::k_attn_packed<DH, TI, BIAS><<<grid, C::THREADS, C::SMEM, st>>>(tq, tk, tv, p);
  return launch_status("attention_packed");
}

template <typename TI>
static wd_status attention_packed_t(int dh, int kv_heads, const void* q, int64_t q_rs, const void* k, const void* v,
                                    int64_t kv_rs, const pka::Params& p, cudaStream_t st) {
  const CUtensorMapDataType ty =
      std::is_same<TI, f16>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap tq, tk, tv;
  WD_TRY(make_tmap_rows(&tq, ty, q, p.q_rows, static_cast<int64_t>(p.heads) * dh, q_rs));
  WD_TRY(make_tmap_rows(&tk, ty, k, p.k_rows, static_cast<int64_t>(kv_heads) * dh, kv_rs));
  WD_TRY(make_tmap_rows(&tv, ty, v, p.k_rows, static_cast<int64_t>(kv_heads) * dh, kv_rs));
  if (dh == 128)
    return p.bias ? launch_attn_packed<128, TI, true>(tq, tk, tv, p, st) : launch_attn_packed<128, TI, false>(tq, tk, tv, p, st);
  return p.bias ? launch_attn_packed<64, TI, true>(tq, tk, tv, p, st) : launch_attn_packed<64, TI, false>(tq, tk, tv, p, st);
}

}  // namespace wd
