// k_gemm_lora.cu — the shared projection with each request's low-rank adapter:
// rows [seg[s], seg[s+1]) of A belong to request s, whose adapter a = ids[s] adds
//   scale[a] (A D_a^T) U_a^T,   D_a [r, K], U_a [N, r],
// to A W^T + bias before the epilogue.
//
// Two steps, the second launched so that it may start while the first one ends (it
// waits for T only where its own K loop is over).  k_lora_down makes T = scale[a] A D_a^T
// (fp32 sums, r columns wide), and k_gemm_lora or k_gemm_lora2 runs the dense GEMM of
// k_gemm_tc.cu whose K loop goes on, for each request that meets the row tile, over the r
// columns of T and U_a: the low-rank product lands in the same TMEM accumulator, so
// the output is written once and no epilogue knows of it.
//
// A row tile may hold the ends of several requests.  T is therefore stored in slabs, one
// per (row tile m, request s) that meet, with the rows of other requests zero: the
// extra K-blocks of a tile then add up to each row's own adapter.  A U that is not finite
// breaks that (0 x inf): the epilogue of a tile that holds more than one request's rows
// looks its accumulator through and sums what is not finite again (repair).  (Masking the
// rows in the MMA itself, by its vector of disabled lanes, gave wrong rows in some
// instantiations.)  Requests are in row order, so the meeting pairs (m, s) form a monotone
// chain and m + s numbers the slabs without a table.
//
// T enters the second product in bf16, rounded once when the output is bf16 (its own
// rounding is as large).  For half outputs T is split in two bf16 parts, for fp32 ones in
// three, each the remainder of those before, and all are multiplied: 2^-16 or 2^-24 of the
// middle is lost at most, instead of 2^-8.  For fp32 outputs the accumulators are also summed
// in fp32 every few stages of K, here across the cluster and in the dense part in registers
// (sum_every in k_gemm_tc.cu).
//
// Measured (B200, sustained loops on several boxes): 43745 x 4608 x 1536 with rank 32 to bf16
// 455 - 540 us, to half 500 - 555, where wd_gemm without adapters takes 505 - 545; 2500 x 1536 x 8960
// with rank 64 to fp32 77 - 91 us (wd_gemm 61 - 70); 891 x 1536 x 1536 with rank 16 14.4 - 16.6 us, 13.4
// in a graph (wd_gemm 13 - 15); 700 requests of one row over four adapters, 4608 x 1536 with rank 16,
// 210 us (wd_gemm 15): every request adds a K-block to its tile.  Bound by the power cap
// and an SM's 64 bytes a clock from L2 where there are many rows, by the latencies of two dependent
// launches where there are few.
#include "wd_internal.cuh"

namespace wd {
namespace lora {

constexpr int BM = tcg::BM, BK = tcg::BK;
constexpr int MAX_RANK = 256;

struct Args {
  const int* seg;       // [n_seg + 1], non-decreasing row offsets
  const int* ids;       // [n_seg]; outside [0, n_adapters): no adapter
  const float* scale;   // [n_adapters] or null (1)
  int n_seg, n_adapters, rank, parts;
  int M, N, K;
  int m_tiles, tile;    // row tiles and their height: 128 rows, or 256 for SM pairs
  bf16* slabs;          // [m_tiles + n_seg][parts][tile][rank]
  int4* tiles;          // [m_tiles]: where the tile's list begins, its length (negative: mixed), and its first entry
  int2* list;           // [m_tiles + n_seg]: (slab, adapter) of each tile's active requests
  const bf16 *A, *W, *up;
};

// Rows [x, y) of request s, kept inside the matrix whatever the offsets say.
__device__ __forceinline__ int2 seg_rows(const Args& a, int s) {
  const int lo = min(max(a.seg[s], 0), a.M);
  return make_int2(lo, max(min(a.seg[s + 1], a.M), lo));
}
// Whether a request has an adapter and rows in the tile at m0.
__device__ __forceinline__ bool active(const Args& a, int2 rows, int id, int m0) {
  return static_cast<unsigned>(id) < static_cast<unsigned>(a.n_adapters) && max(rows.x, m0) < min(rows.y, m0 + a.tile);
}

// The last s in [0, n) with ok(s), where ok holds up to some s and not behind it; -1 if
// nowhere.  A whole warp, 32 places at a time: one round of loads up to 32 requests,
// two up to 1024.
template <typename F>
__device__ __forceinline__ int last_where(int n, int lane, F&& ok) {
  int lo = 0, hi = n, best = -1;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5, s = lo + lane * step;
    const unsigned yes = __ballot_sync(0xffffffffu, s < hi && ok(s));
    if (!yes) break;
    best = lo + (31 - __clz(yes)) * step;
    if (step == 1) break;
    hi = min(hi, best + step);
    lo = best + 1;
  }
  return best;
}

// The list of row tile m (a whole warp): from the first request that ends behind its
// first row to the last that starts before its end, those that are active.  The tile is
// mixed unless it has none or all its rows are of one.
__device__ __forceinline__ void write_list(const Args& a, int m, int lane) {
  const int m0 = m * a.tile;
  const int first = last_where(a.n_seg, lane, [&](int s) { return a.seg[s] <= m0; });
  const int last = last_where(a.n_seg, lane, [&](int s) { return a.seg[s] < m0 + a.tile; });
  const int begin = max(first, 0);
  int count = 0;
  bool whole = false;
  int2 head = make_int2(0, 0);
  for (int s0 = begin; s0 <= last; s0 += 32) {
    const int s = s0 + lane;
    const int id = s <= last ? a.ids[s] : -1;
    const int2 rows = s <= last ? seg_rows(a, s) : make_int2(0, 0);
    const bool act = s <= last && active(a, rows, id, m0);
    const unsigned yes = __ballot_sync(0xffffffffu, act);
    whole |= __any_sync(0xffffffffu, act && rows.x <= m0 && rows.y >= min(m0 + a.tile, a.M));
    if (act) a.list[m + begin + count + __popc(yes & ((1u << lane) - 1))] = make_int2(m + s, id);
    if (!count && yes) {
      const int src = __ffs(yes) - 1;
      head = make_int2(m + s0 + src, __shfl_sync(0xffffffffu, id, src));
    }
    count += __popc(yes);
  }
  if (lane == 0) a.tiles[m] = make_int4(m + begin, whole ? count : -count, head.x, head.y);
}

// s[c] += sum over n (a multiple of 8) of x[i] y[c ld + i], in two fp32 sums, for eight rows c of y
__device__ __forceinline__ void dot8(float2 (&s)[8], const bf16* x, const bf16* y, int64_t ld, int n) {
#pragma unroll 1   // 2: 168 registers instead of 135, which all launches pay for (0.2 us)
  for (int k = 0; k < n; k += 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(x + k);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 w = *reinterpret_cast<const uint4*>(y + c * ld + k);
      s[c] = ffma2(unpack_bf16x2(u.x), unpack_bf16x2(w.x), s[c]);
      s[c] = ffma2(unpack_bf16x2(u.y), unpack_bf16x2(w.y), s[c]);
      s[c] = ffma2(unpack_bf16x2(u.z), unpack_bf16x2(w.z), s[c]);
      s[c] = ffma2(unpack_bf16x2(u.w), unpack_bf16x2(w.w), s[c]);
    }
  }
}

// Whether all of a lane's N values are finite: four chains of three-way maxima, which keep a NaN.
template <int N>
__device__ __forceinline__ bool all_finite(const float (&v)[N]) {
  float top[4] = {};
#pragma unroll
  for (int j = 0; j < N; j += 2)
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(top[j / 2 % 4]) : "f"(top[j / 2 % 4]), "f"(fabsf(v[j])), "f"(fabsf(v[j + 1])));
  return top[0] < INFINITY && top[1] < INFINITY && top[2] < INFINITY && top[3] < INFINITY;
}

// One warp's 32 rows (TMEM lanes of tbase; this lane's is row m) and `cols` columns from n on of a mixed
// tile's accumulator: each element that is not finite is summed again from the definition, over
// the row's own adapter only (0 x inf of another request's U is never finite; a row whose own
// numbers make it so stays so), eight columns at a time, since the lanes' rows of A come 16
// bytes a line.  Not inlined: it runs when an adapter is broken (one wholly NaN: 891 x 1536 x 1536 1.0 ms, 2500 x
// 1536 x 8960 in fp32 8 ms, 700 requests of one row at 4608 x 1536 2.1 ms).
__device__ __noinline__ void repair(const Args& a, int4 row, int tile, uint32_t tbase, int cols, int m, int n) {
  const bf16 *t = nullptr, *u = nullptr;   // the row's T and its adapter's U
  for (int i = 0; i < -row.y; ++i) {
    const int2 e = a.list[row.x + i];
    const int s = e.x - tile;   // offsets that decrease let tiles write into each other's lists
    if (static_cast<unsigned>(s) >= static_cast<unsigned>(a.n_seg)) continue;
    const int2 rows = seg_rows(a, s);
    if (m >= rows.x && m < rows.y) {
      t = a.slabs + (static_cast<int64_t>(e.x) * a.parts * a.tile + (m - tile * a.tile)) * a.rank;
      u = a.up + static_cast<int64_t>(e.y) * a.N * a.rank;
    }
  }
  for (int c = 0; c < cols; c += 8) {
    uint32_t r[8];
    tmem_ld8(tbase + c, r);
    tmem_wait_ld();
    uint32_t bad = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) bad |= (r[j] & 0x7f800000u) == 0x7f800000u ? 1u << j : 0u;
    if (m >= a.M) bad = 0;
    if (!__any_sync(0xffffffffu, bad)) continue;
    if (bad) {
      float2 s[8] = {};
      if (t)
        for (int p = 0; p < a.parts; ++p)
          dot8(s, t + static_cast<int64_t>(p) * a.tile * a.rank, u + static_cast<int64_t>(n + c) * a.rank, a.rank, a.rank);
      bool open = false;   // an element that its own adapter leaves finite
#pragma unroll
      for (int j = 0; j < 8; ++j) open |= (bad >> j & 1u) && isfinite(s[j].x + s[j].y);
      if (open) dot8(s, a.A + static_cast<int64_t>(m) * a.K, a.W + static_cast<int64_t>(n + c) * a.K, a.K, a.K);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (bad >> j & 1u) r[j] = __float_as_uint(s[j].x + s[j].y);
    }
    __syncwarp();
    tmem_st8(tbase + c, r);
  }
  tmem_wait_st();
}

// The extra K-blocks of gemm_body: request after request, part after part.
struct Extra {
  static constexpr bool ON = true;
  template <int MODE> __host__ __device__ static constexpr int sum_every() {
    return MODE == EPI_F32 || MODE == EPI_RESID ? 8 : 0;
  }
  template <int MODE> __host__ __device__ static constexpr int wg() { return sum_every<MODE>() ? 2 : tcg::epi_wg<MODE>(); }
  const Args& a;
  const CUtensorMap* tmT;   // slabs [rows, rank], box 64 x 128
  const CUtensorMap* tmU;   // U [n_adapters * N, rank], box 64 x BN
  using Row = int4;
  // k_lora_down's results from here on
  __device__ __forceinline__ void wait() const { asm volatile("griddepcontrol.wait;" ::: "memory"); }
  // (volatile: issued where it stands, a whole K loop before its first use)
  __device__ __forceinline__ Row row(int m) const {
    int4 t;
    asm volatile("ld.global.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(t.x), "=r"(t.y), "=r"(t.z), "=r"(t.w)
                 : "l"(a.tiles + m)
                 : "memory");
    return t;
  }
  __device__ __forceinline__ int per_part() const { return (a.rank + BK - 1) / BK; }
  __device__ __forceinline__ int count(const Row& r) const { return abs(r.y) * a.parts * per_part(); }
  // An epilogue warp's share of a tile (COLS columns of its lanes), taken out of TMEM by out().  In a mixed
  // tile, if anything of it is not finite, it is repaired and taken out again, over what the first time
  // stored.  Looking it through while those stores are under way takes 0.1 us in a graph (13.3 -> 13.4 at 891 x
  // 1536 x 1536 of three requests, rank 16; 14.5 -> 14.9 us a call on a stream), before them 0.3 us more; larger
  // batches take as long as without.  For epilogues that store; those that add to the output sum in
  // registers and use check().
  template <int COLS, typename F>
  __device__ __forceinline__ void take_out(const Row& r, int tile, uint32_t tbase, int m, int n, F&& out) const {
    for (bool last = r.y >= 0;; last = true) {
      out();
      if (last) return;
      bool ok = true;
#pragma unroll 1
      for (int c = 0; c < COLS; c += 32) {
        uint32_t u[32];
        tmem_ld32(tbase + c, u);
        tmem_wait_ld();
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
        ok &= all_finite(v);
      }
      if (__all_sync(0xffffffffu, ok)) return;
      bulk_wait_group<0>();   // of the lane that stores: performed, not only read
      __syncwarp();
      repair(a, r, tile, tbase, COLS, m, n);
    }
  }
  // The same for sums in registers, before they are taken out: they go back to TMEM for the repair.
  template <int COLS>
  __device__ __forceinline__ void check(const Row& r, int tile, uint32_t tbase, float (&v)[COLS], int m, int n) const {
    if (r.y >= 0 || __all_sync(0xffffffffu, all_finite(v))) return;
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      uint32_t u[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(v[c + j]);
      tmem_st32(tbase + c, u);
    }
    tmem_wait_st();
    repair(a, r, tile, tbase, COLS, m, n);
    tcg::add_columns(tbase, v, true);
  }
  // MMAs of the k-th extra block: 16 columns each, none for the zeros behind rank
  __device__ __forceinline__ int steps(int k) const {
    const int left = a.rank - k % per_part() * BK;
    return left >= BK ? BK / 16 : (left + 15) / 16;
  }
  template <typename F>
  __device__ __forceinline__ void each(const Row& r, int n0, F&& load) const {
    int2 e = make_int2(r.z, r.w);
    const int n = abs(r.y);
    for (int i = 0; i < n; ++i) {
      const int2 next = i + 1 < n ? a.list[r.x + i + 1] : e;   // fetched while this one's loads are issued
      for (int p = 0; p < a.parts; ++p)
        for (int k = 0; k < a.rank; k += BK)
          if (!load(tmT, k, (e.x * a.parts + p) * a.tile, tmU, k, e.y * a.N + n0)) return;
      e = next;
    }
  }
};

template <int MODE> __host__ __device__ constexpr int threads() { return 64 + 128 * Extra::wg<MODE>(); }
// staging: one 32 x 32 fp32 tile a warp, or as k_gemm_tc's
template <int BN, int MODE> __host__ __device__ constexpr int staging() {
  return Extra::sum_every<MODE>() ? 8 * 4096 : tcg::Cfg<BN>::stg(MODE);
}

template <int BN, int MODE>
__global__ void __launch_bounds__(threads<MODE>(), 1)
k_gemm_lora(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmT,
            const __grid_constant__ CUtensorMap tmU, const Epi ep, const __grid_constant__ Args a) {
  tcg::gemm_body<BN, MODE, false>(tmA, tmB, tmX, ep, a.M, a.N, a.K, Extra{a, &tmT, &tmU});
}

// ------------------------------------------------------------------ the product on SM pairs
// The same GEMM with tiles of 256 x 256 for a cluster of two blocks: one MMA of both SMs
// takes 128 rows of A and half of B's 256 rows from each, so a K stage brings 32 KB into
// an SM instead of the 48 KB of a 128 x 256 tile, which the SM's 64 bytes a clock from L2
// could not deliver in the MMAs' 512 clocks.  Each block loads its part (warp 0); the
// block of rank 0 issues for both (warp 1); each takes its 128 rows of the accumulator
// out (warps 2..).  Stages are counted on rank 0's barriers, freed on both.
constexpr int BN2 = 256, STAGES2 = 6, STAGE2_BYTES = 2 * BM * BK * 2;
constexpr uint32_t IDESC2 = idesc_bf16(256, BN2, 0, 0);
template <int MODE> constexpr int smem2() { return 1024 + STAGES2 * STAGE2_BYTES + staging<BN2, MODE>() + 256; }
static_assert(smem2<EPI_F32>() <= 232448 && smem2<EPI_GELU>() <= 232448, "shared memory of one block");
enum : unsigned { SITE2_EMPTY = 0x411, SITE2_FULL = 0x412, SITE2_TFULL = 0x413, SITE2_TEMPTY = 0x414, SITE2_DRAIN = 0x415 };

template <int MODE>
__global__ void __launch_bounds__(threads<MODE>(), 1)
k_gemm_lora2(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
             const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmT,
             const __grid_constant__ CUtensorMap tmU, const Epi ep, const __grid_constant__ Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES2 * BM * BK * 2;
  float* stg = reinterpret_cast<float*>(smem + STAGES2 * STAGE2_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES2 * STAGE2_BYTES + staging<BN2, MODE>());   // of rank 0
  uint64_t* empty = full + STAGES2;      // of each block
  uint64_t* tfull = empty + STAGES2;     // [2], of each block
  uint64_t* tempty = tfull + 2;          // [2], of rank 0
  uint64_t* tdone = tempty + 2;          // of each block
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tdone + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int n_tiles = a.N / BN2, tiles = a.m_tiles * n_tiles;
  const int k_iters = (a.K + BK - 1) / BK;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  constexpr int SUM = Extra::sum_every<MODE>();
  const Extra ex{a, &tmT, &tmU};

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES2; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 2 * 4 * Extra::wg<MODE>()); }
    mbar_init(tdone, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) { tmem_alloc2(tmem_slot, 512); tmem_relinquish2(); }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* ta, int ac, int ar, const CUtensorMap* tb, int bc, int br) -> bool {
        if (!mbar_wait_cluster(&empty[stage], phase ^ 1u, SITE2_EMPTY)) return ok = false;
        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * STAGE2_BYTES);   // both blocks' bytes
        const uint32_t bar = cluster_addr(&full[stage], 0);
        tma_load_2d_pair(sA + stage * (BM * BK * 2), ta, ac, ar + rank * BM, bar);
        tma_load_2d_pair(sB + stage * (BM * BK * 2), tb, bc, br + rank * BM, bar);
        if (++stage == STAGES2) { stage = 0; phase ^= 1u; }
        return true;
      };
      for (int t = first; t < tiles && ok; t += step) {
        const int m0 = t / n_tiles * 256, n0 = t % n_tiles * BN2;
        for (int k = 0; k < k_iters; ++k)
          if (!load(&tmA, k * BK, m0, &tmB, k * BK, n0)) break;
        ex.wait();
        if (ok) ex.each(ex.row(t / n_tiles), n0, load);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint64_t da0 = sdesc_sw128(smem_u32(sA), 16, 1024), db0 = sdesc_sw128(smem_u32(sB), 16, 1024);
      const uint32_t a_lo0 = static_cast<uint32_t>(da0), b_lo0 = static_cast<uint32_t>(db0);
      const uint32_t d_hi = static_cast<uint32_t>(da0 >> 32);
      for (int t = first; t < tiles && ok; t += step) {
        if (!mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, SITE2_TEMPTY)) { ok = false; break; }
        tc_fence_after();
        uint32_t d = tmem + acc * BN2;
        Extra::Row row{};
        if (t != first) row = ex.row(t / n_tiles);
        for (int k = 0; k < k_iters; ++k) {
          if constexpr (SUM > 0) {
            if (k && k % SUM == 0) {   // hand this part over and go on in the other accumulator
              umma2_commit(&tfull[acc]);
              if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
              if (!mbar_wait_cluster(&tempty[acc], acc_phase ^ 1u, SITE2_TEMPTY)) { ok = false; break; }
              tc_fence_after();
              d = tmem + acc * BN2;
            }
          }
          if (!mbar_wait_cluster(&full[stage], phase, SITE2_FULL)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_lo = a_lo0 + stage * (BM * BK * 2 >> 4), b_lo = b_lo0 + stage * (BM * BK * 2 >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            umma2_ss_lh(d, a_lo + kk * 2, d_hi, b_lo + kk * 2, d_hi, IDESC2, ((SUM ? k % (SUM ? SUM : 1) : k) | kk) != 0);
          umma2_commit(&empty[stage]);
          if (++stage == STAGES2) { stage = 0; phase ^= 1u; }
        }
        if (t == first) { ex.wait(); row = ex.row(t / n_tiles); }
        const int extra = ok ? ex.count(row) : 0;
        for (int k = 0; k < extra; ++k) {
          if (!mbar_wait_cluster(&full[stage], phase, SITE2_FULL)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_lo = a_lo0 + stage * (BM * BK * 2 >> 4), b_lo = b_lo0 + stage * (BM * BK * 2 >> 4);
          const int steps = ex.steps(k);
          for (int kk = 0; kk < steps; ++kk) umma2_ss_lh(d, a_lo + kk * 2, d_hi, b_lo + kk * 2, d_hi, IDESC2, 1u);
          umma2_commit(&empty[stage]);
          if (++stage == STAGES2) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma2_commit(&tfull[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      umma2_commit(tdone);   // arrives in both blocks once every MMA has read its operands
    }
    __syncwarp();
  } else {
    constexpr int COLS = BN2 / Extra::wg<MODE>();
    const int c_begin = ((warp - 2) >> 2) * COLS, q = warp & 3;
    int acc = 0;
    uint32_t acc_phase = 0;
    [[maybe_unused]] uint32_t chunk = 0;
    auto wait = [&]() -> bool {
      const bool ok = mbar_wait_cluster(&tfull[acc], acc_phase, SITE2_TFULL);
      tc_fence_after();
      return __all_sync(0xffffffffu, ok);
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&tempty[acc], 0));
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    };
    bool ok = true;
    ex.wait();
    for (int t = first; t < tiles && ok; t += step) {
      const int m0 = t / n_tiles * 256 + rank * BM, n0 = t % n_tiles * BN2;
      const Extra::Row row = ex.row(t / n_tiles);
      if constexpr (SUM > 0) {
        float v[COLS];
        for (int k = 0; k < k_iters && ok; k += SUM) {
          ok = wait();
          if (!ok) break;
          const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * BN2 + c_begin;
          tcg::add_columns(tbase, v, k == 0);
          if (k + SUM >= k_iters) ex.check(row, t / n_tiles, tbase, v, m0 + q * 32 + lane, n0 + c_begin);
          release();
        }
        if (ok) tcg::epi_sums<MODE>(ep, tmX, stg + (warp - 2) * 1024, lane, v, m0 + q * 32, n0 + c_begin, a.M);
      } else {
        ok = wait();
        if (!ok) break;
        ex.take_out<COLS>(row, t / n_tiles, tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * BN2 + c_begin,
                          m0 + q * 32 + lane, n0 + c_begin, [&]() {
          tcg::epi_tile<BN2, MODE>(ep, tmX, stg, warp, lane, c_begin, tmem + acc * BN2, m0, n0, a.M, chunk);
        });
        release();
      }
    }
    if (lane == 0) bulk_wait_group<0>();   // stores and reductions performed before exit
  }
  // Every copy has landed (its stage was multiplied) and every MMA has ended before a block leaves.
  if (warp == 1) {
    if (lane == 0) mbar_wait_cluster(tdone, 0, SITE2_DRAIN);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem, 512);
}

// ------------------------------------------------------------------ T = scale A D^T
// One cluster of `split` blocks per 128 rows of a slab, each with a share of K: 128 rows x rank, K in
// 64-wide TMA stages, tcgen05 MMAs of 128 x RN x 16 (RN = rank rounded up to 16; the
// rows of D behind rank belong to the next adapter and their columns are not stored).
// Warp 0 loads, warp 1 issues, warps 2-5 take the accumulator out.  The blocks'
// fp32 parts meet in shared memory across the cluster, summed in a fixed order, each
// block taking 128 / split of the rows.  A warp of the first block of each of the first
// m_tiles clusters also writes its row tile's list.
constexpr int STAGES = 3, THREADS = 192, MAX_SPLIT = 8;   // three stages: three blocks an SM up to rank 32
__host__ __device__ constexpr int stage_bytes(int rn) { return BM * BK * 2 + rn * BK * 2; }
constexpr int smem_bytes(int rn) { return 1024 + STAGES * stage_bytes(rn); }
// fp32 parts take the stages' place: rows of rn + 4 floats (no two of 8 neighbouring rows on one bank)
static_assert(BM * (MAX_RANK + 4) * 4 <= STAGES * stage_bytes(MAX_RANK) && BM * (16 + 4) * 4 <= STAGES * stage_bytes(16),
              "the parts fit into the stages");

enum : unsigned { SITE_EMPTY = 0x401, SITE_FULL = 0x402, SITE_DONE = 0x403, SITE_DRAIN = 0x404 };

// 16 bytes at shared address `addr` of block `rank` of the cluster
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr, uint32_t rank) {
  uint32_t peer;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer)
               : "memory");
  return v;
}

__global__ void __launch_bounds__(THREADS)
k_lora_down(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmD,
            const __grid_constant__ Args a, int rn, uint32_t tmem_cols, uint32_t idesc, int split) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[STAGES], empty[STAGES], done;
  __shared__ uint32_t tmem_slot;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int halves = a.tile / BM;   // of 128 rows a slab
  const int part = blockIdx.x % split, half = blockIdx.x / split % halves, slab = blockIdx.x / split / halves;

  if (threadIdx.x == 0) { tma_prefetch_desc(&tmA); tma_prefetch_desc(&tmD); }
  // the pair (m, s) of this slab: the last s whose request starts before the end of tile slab - s
  const int s = last_where(a.n_seg, lane, [&](int s) { return a.seg[s] < (slab - s + 1) * a.tile; });
  const int m = slab - s, m0 = m * a.tile + half * BM;
  const bool lists = slab < a.m_tiles && part == 0 && half == 0 && warp == 5;   // this warp writes a tile's list
  int2 rows_s = make_int2(0, 0);
  int ad = -1;
  if (s >= 0) { rows_s = seg_rows(a, s); ad = a.ids[s]; }
  if (s < 0 || m < 0 || m >= a.m_tiles || !active(a, rows_s, ad, m * a.tile)) {   // no such pair: all leave
    if (lists) write_list(a, slab, lane);
    return;
  }
  bf16* dst = a.slabs + (static_cast<int64_t>(slab) * a.parts * a.tile + half * BM) * a.rank;
  const int64_t next = static_cast<int64_t>(a.tile) * a.rank;   // from one part to the next
  if (max(rows_s.x, m0) >= min(rows_s.y, m0 + BM)) {           // the request lies in the tile's other half: zeros
    if (lists) write_list(a, slab, lane);
    for (int i = part * THREADS + threadIdx.x; i < BM * a.rank / 8; i += split * THREADS)
      for (int p = 0; p < a.parts; ++p) reinterpret_cast<uint4*>(dst + p * next)[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int k_iters = (a.K + BK - 1) / BK;
  const int k0 = k_iters * part / split, kn = k_iters * (part + 1) / split - k0;   // this block's K stages (>= 1)
  const int sb = stage_bytes(rn);

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    mbar_init(&done, 1);
    fence_mbar_init();
  }
  if (warp == 1) { tmem_alloc(&tmem_slot, tmem_cols); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  float* mine = reinterpret_cast<float*>(smem);
  const int ld = rn + 4;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t issued = 0, last_par = 0;
      for (int k = 0; k < kn; ++k) {
        const int st = k % STAGES;
        const uint32_t ph = (k / STAGES) & 1u;
        if (!mbar_wait(&empty[st], ph ^ 1u, SITE_EMPTY)) break;
        mbar_arrive_expect_tx(&full[st], sb);
        tma_load_2d(smem + st * sb, &tmA, (k0 + k) * BK, m0, &full[st]);
        tma_load_2d(smem + st * sb + BM * BK * 2, &tmD, (k0 + k) * BK, ad * a.rank, &full[st]);
        issued |= 1u << st;
        last_par = (last_par & ~(1u << st)) | (ph << st);
      }
      for (int i = 0; i < STAGES; ++i)
        if (issued & (1u << i)) mbar_wait(&full[i], (last_par >> i) & 1u, SITE_DRAIN);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t base = smem_u32(smem);
      for (int k = 0; k < kn; ++k) {
        const int st = k % STAGES;
        if (!mbar_wait(&full[st], (k / STAGES) & 1u, SITE_FULL)) break;
        tc_fence_after();
        const uint64_t da = sdesc_sw128(base + st * sb, 16, 1024);
        const uint64_t db = sdesc_sw128(base + st * sb + BM * BK * 2, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) umma_ss(tmem, da + kk * 2, db + kk * 2, idesc, (k | kk) != 0);
        umma_commit(&empty[st]);
      }
      umma_commit(&done);
      mbar_wait(&done, 0, SITE_DRAIN);
    }
    __syncwarp();
  } else {
    if (lists) write_list(a, slab, lane);
    if (mbar_wait_warp(&done, 0, SITE_DONE)) {   // every stage has been read: the parts may overwrite them
      tc_fence_after();
      const int q = warp & 3, r = q * 32 + lane;
      for (int c = 0; c < rn; c += 32) {
        uint32_t u[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, u);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          if (c + j < rn)
            *reinterpret_cast<float4*>(mine + r * ld + c + j) =
                make_float4(__uint_as_float(u[j]), __uint_as_float(u[j + 1]), __uint_as_float(u[j + 2]),
                            __uint_as_float(u[j + 3]));
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, tmem_cols);
  // rows [part * 128 / split, ...): all parts' sums, scaled, in bf16
  const float sc = a.scale ? a.scale[ad] : 1.f;
  const int rows = BM / split, chunks = a.rank / 8;
  for (int i = threadIdx.x; i < rows * chunks; i += THREADS) {
    const int r = part * rows + i / chunks, c = i % chunks * 8;
    float v[8] = {};
    if (m0 + r >= rows_s.x && m0 + r < rows_s.y) {   // rows of other requests stay zero
      const uint32_t addr = smem_u32(mine + r * ld + c);
      for (int p0 = 0; p0 < split; p0 += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int p = 0; p < 4; ++p)   // all on their way before the first is added
          if (p0 + p < split) { x[p] = cluster_ld4(addr, p0 + p); y[p] = cluster_ld4(addr + 16, p0 + p); }
#pragma unroll
        for (int p = 0; p < 4; ++p)
          if (p0 + p < split) {
            v[0] += x[p].x; v[1] += x[p].y; v[2] += x[p].z; v[3] += x[p].w;
            v[4] += y[p].x; v[5] += y[p].y; v[6] += y[p].z; v[7] += y[p].w;
          }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= sc;
    }
    for (int p = 0; p < a.parts; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // rounded, and the exact remainder kept for the next part
        w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        const float2 f = unpack_bf16x2(w[j]);
        v[2 * j] -= f.x;
        v[2 * j + 1] -= f.y;
      }
      *reinterpret_cast<uint4*>(dst + p * next + r * a.rank + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  cluster_sync();   // no block leaves while others read its part
}

}  // namespace lora

// ------------------------------------------------------------------ host side
static size_t lora_slab_bytes(int64_t slabs, int tile, int rank) {
  return static_cast<size_t>(slabs) * 3 * tile * rank * 2;   // up to three parts
}

size_t gemm_lora_bytes(int M, int n_seg, int rank) {
  size_t most = 0;
  for (int tile : {128, 256}) {
    const int64_t mt = (static_cast<int64_t>(M) + tile - 1) / tile;
    const size_t n = lora_slab_bytes(mt + n_seg, tile, rank) + static_cast<size_t>(mt) * sizeof(int4) +
                     static_cast<size_t>(mt + n_seg) * sizeof(int2);
    if (n > most) most = n;
  }
  return most;
}

constexpr int LORA_PAIR = 512;   // the "tile width" of k_gemm_lora2 in the dispatch

template <int BN, int MODE>
static wd_status launch_lora(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tt, const CUtensorMap& tu,
                             const Epi& ep, const lora::Args& a, cudaStream_t st) {
  constexpr bool PAIR = BN == LORA_PAIR;
  constexpr int W = PAIR ? 256 : BN;
  constexpr int SMEM =
      PAIR ? lora::smem2<MODE>() : tcg::Cfg<W>::smem(MODE) - tcg::Cfg<W>::stg(MODE) + lora::staging<W, MODE>();
  const int tiles = a.m_tiles * (a.N / W), at_once = PAIR ? sm_count() / 2 : sm_count();
  CUtensorMap tx = ta;
  if (lora::Extra::sum_every<MODE>()) WD_TRY(make_tmap_f32(&tx, ep.out, a.M, a.N, ep.ldo, 32, 32));
  if (tcg::staged2<MODE>() && (W / tcg::epi_wg<MODE>()) % 64 == 0)
    WD_TRY(make_tmap_2b(&tx, ep.out, a.M, a.N, ep.ldo, MODE == EPI_STORE_F16));
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // may start before k_lora_down has ended: Extra::wait
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((tiles < at_once ? tiles : at_once) * (PAIR ? 2 : 1));
  cfg.blockDim = dim3(lora::threads<MODE>());
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  Trace tr(KC_GEMM, st);
  if constexpr (PAIR) {
    WD_TRY((allow_smem<lora::k_gemm_lora2<MODE>>(SMEM)));
    cudaLaunchKernelEx(&cfg, lora::k_gemm_lora2<MODE>, ta, tb, tx, tt, tu, ep, a);
  } else {
    WD_TRY((allow_smem<lora::k_gemm_lora<W, MODE>>(SMEM)));
    cudaLaunchKernelEx(&cfg, lora::k_gemm_lora<W, MODE>, ta, tb, tx, tt, tu, ep, a);
  }
  return launch_status("gemm_lora");
}

template <int BN>
static wd_status dispatch_lora(int mode, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tt,
                               const CUtensorMap& tu, const Epi& ep, const lora::Args& a, cudaStream_t st) {
  switch (mode) {
    case EPI_STORE: return launch_lora<BN, EPI_STORE>(ta, tb, tt, tu, ep, a, st);
    case EPI_GELU: return launch_lora<BN, EPI_GELU>(ta, tb, tt, tu, ep, a, st);
    case EPI_F32: return launch_lora<BN, EPI_F32>(ta, tb, tt, tu, ep, a, st);
    case EPI_RESID: return launch_lora<BN, EPI_RESID>(ta, tb, tt, tu, ep, a, st);
    case EPI_STORE_F16: return launch_lora<BN, EPI_STORE_F16>(ta, tb, tt, tu, ep, a, st);
  }
  set_error("gemm_lora: bad epilogue %d", mode);
  return WD_ERR_ARG;
}

// Tile: the time of a round of tiles goes with the bytes of a K stage that an SM takes in, 128 + BN
// rows of A and B for a tile of 128 x BN and 128 + 128 for an SM pair's 256 x 256 (BN = 512
// here), so the tile with the least rounds * rows is taken; at equal cost the narrower one, whose
// row tiles are shorter.
static int lora_tile(int M, int N) {
  int best = 64;
  int64_t least = INT64_MAX;
  for (int bn : {64, 128, 256, LORA_PAIR}) {
    const bool pair = bn == LORA_PAIR;
    if (N % (pair ? 256 : bn)) continue;
    const int64_t tiles = pair ? (M + 255ll) / 256 * (N / 256) : (M + 127ll) / 128 * (N / bn);
    const int64_t at_once = pair ? sm_count() / 2 : sm_count();
    const int64_t cost = (tiles + at_once - 1) / at_once * (pair ? 256 : 128 + bn);
    if (cost < least) { least = cost; best = bn; }
  }
  return best;
}

static wd_status gemm_lora(int M, int N, int K, const void* A, const void* W, const wd_lora& l, int mode, const Epi& ep,
                           void* ws, cudaStream_t st) {
  lora::Args a{};
  a.seg = l.seg; a.ids = l.adapter; a.scale = l.scale;
  a.n_seg = l.n_seg; a.n_adapters = l.n_adapters; a.rank = l.rank;
  const bool fp32 = mode == EPI_F32 || mode == EPI_RESID;
  a.parts = fp32 ? 3 : mode == EPI_STORE_F16 ? 2 : 1;
  a.M = M; a.N = N; a.K = K;
  a.A = static_cast<const bf16*>(A); a.W = static_cast<const bf16*>(W); a.up = static_cast<const bf16*>(l.up);
  const int BN = lora_tile(M, N);
  const bool pair = BN == LORA_PAIR;
  a.tile = pair ? 256 : 128;
  a.m_tiles = static_cast<int>((static_cast<int64_t>(M) + a.tile - 1) / a.tile);
  const int64_t slabs = static_cast<int64_t>(a.m_tiles) + l.n_seg;
  a.slabs = static_cast<bf16*>(ws);
  a.tiles = reinterpret_cast<int4*>(static_cast<char*>(ws) + lora_slab_bytes(slabs, a.tile, l.rank));   // 16-byte aligned
  a.list = reinterpret_cast<int2*>(a.tiles + a.m_tiles);
  const int rn = (l.rank + 15) / 16 * 16;
  CUtensorMap ta, tb, td, tt, tu;
  WD_TRY(make_tmap_bf16(&ta, A, M, K, K, lora::BK, lora::BM));
  WD_TRY(make_tmap_bf16(&td, l.down, static_cast<int64_t>(l.n_adapters) * l.rank, K, K, lora::BK, rn));
  uint32_t cols = 32;
  while (cols < static_cast<uint32_t>(rn)) cols *= 2;
  WD_TRY((allow_smem<lora::k_lora_down>(lora::smem_bytes(lora::MAX_RANK))));
  {
    // a block for every SM, with 4 stages of K each at least (258 blocks of 24 stages: 25 us, 516 of 12: 31);
    // for fp32 outputs also no more than 24 stages each, since a block's accumulator truncates (see
    // sum_every)
    int split = 1;
    const int k_iters = (K + lora::BK - 1) / lora::BK;
    const int64_t blocks = slabs * (a.tile / lora::BM);
    while (split < lora::MAX_SPLIT && blocks * split < sm_count() && k_iters >= 8 * split) split *= 2;
    while (split < lora::MAX_SPLIT && fp32 && k_iters > 24 * split) split *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * split));
    cfg.blockDim = dim3(lora::THREADS);
    cfg.dynamicSmemBytes = lora::smem_bytes(rn);
    cfg.stream = st;
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = split;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    Trace tr(KC_GEMM, st);
    cudaLaunchKernelEx(&cfg, lora::k_lora_down, ta, td, a, rn, cols, idesc_bf16(lora::BM, rn, 0, 0), split);
  }
  WD_TRY(launch_status("lora_down"));
  const int rows_b = pair ? lora::BM : BN;   // of B a load brings: an SM of a pair loads half
  WD_TRY(make_tmap_bf16(&tb, W, N, K, K, lora::BK, rows_b));
  WD_TRY(make_tmap_bf16(&tt, a.slabs, slabs * a.parts * a.tile, l.rank, l.rank, lora::BK, lora::BM));
  WD_TRY(make_tmap_bf16(&tu, l.up, static_cast<int64_t>(l.n_adapters) * N, l.rank, l.rank, lora::BK, rows_b));
  switch (BN) {
    case LORA_PAIR: return dispatch_lora<LORA_PAIR>(mode, ta, tb, tt, tu, ep, a, st);
    case 256: return dispatch_lora<256>(mode, ta, tb, tt, tu, ep, a, st);
    case 128: return dispatch_lora<128>(mode, ta, tb, tt, tu, ep, a, st);
    default: return dispatch_lora<64>(mode, ta, tb, tt, tu, ep, a, st);
  }
}

}  // namespace wd
