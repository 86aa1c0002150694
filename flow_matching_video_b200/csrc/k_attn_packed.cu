// k_attn_packed.cu — attention over packed sequences on the sm_100a tensor cores:
// sequence s owns query rows [cu_q[s], cu_q[s+1]) and keys [cu_k[s], cu_k[s+1]) of
// buffers that hold all sequences one behind the other, and
//   o_i = sum_j softmax_j(scale q_i k_j + b[h, clamp(j - i, -R, R)]) v_j
// over the keys of i's own sequence (i, j counted from its first row).  Query
// heads share kv_heads key/value heads in equal groups.
//
// The products are those of k_attn_tc.cu: two query tiles of 128 rows of one sequence
// and head, S_t = Q_t K_j^T in TMEM, one softmax thread per row, O_t += P_t V_j with P
// from TMEM, the two tiles' softmaxes and products alternating.  Around them:
//  - Blocks are persistent and take their work one pair of tiles after the other from
//    the hardware's queue: the grid has one block per possible pair, and a running
//    block cancels the launch of the next pending one and does its work
//    (clusterlaunchcontrol).  While one pair ends, the next one's Q, K and V are
//    already loading, so short key sequences (prompts: four key blocks a pair) do not
//    wait for a block's start and end each time.
//  - Warp 0 finds each pair's sequence and tile by a scan over cu_q, with the
//    sequences of most key blocks first within each group of 32 (in a batch of up to 32 the
//    last pairs to run are short; further groups follow in their own order); it publishes the
//    pair to the other warps.
//  - A sequence's last key block runs into the next sequence's rows (the TMA clips
//    at the end of the buffer only).  Its scores behind the end become -inf before
//    anything reads them, and its V rows are overwritten with zeros in shared
//    memory before the product, since 0 * NaN of a neighbour would not be 0.
//  - The second tile of a pair may lie behind the sequence's end: it is left out.
// The bias table of the head sits in shared memory in log2 units, its ends
// repeated 160 times so that no index needs clamping; a block of keys that lies R
// or further from all of a warp's rows takes the one end value instead.  Where an
// end value is -inf, key blocks wholly behind it are neither loaded nor multiplied.
//
// Bound: per 128-key block of a pair the softmax's instructions (about 700 a warp, two warps a
// sub-partition) take as long as the MMAs of 128-wide heads, and longer than those of 64-wide ones;
// in a sustained loop the power cap holds both down.  Measured (B200, sustained loops): 7800 + 32760 tokens x
// 12 heads of 128 6.1 - 6.3 ms (1105 - 1140 TFLOP/s; cold 6.1; k_attn_tc on the two sequences one after the
// other 6.2 - 6.4 ms), 7800 + 3185 + 405 tokens 0.44 ms (cold 0.47), 43746 rows to 512 / 77 / 9 / 0 keys 0.15 ms.
// From some hundred sequences on find_work is the bound, whose scan begins at the first one for every pair:
// of 77 tokens, 24 x 64 heads of 64 take 68 us (6.6 us a pair and SM), 300 x 16 heads 0.29 ms (9), 1000 x 16 2.3
// ms (21), 3000 x 16 18 ms (56); 65536 of one token and head 0.36 s (820).
#include "wd_internal.cuh"

namespace wd {
namespace pka {

constexpr int BQ = 128, BK = 128, NQ = 2;
constexpr int MAX_RADIUS = 1024, PAD = 160;   // PAD >= 127 + 31 + 1: a tile's reach past +-R
constexpr float LOG2E = 1.4426950408889634f;
// Warps: 0 loads, 1 issues MMAs, 2 and 3 only fill their warpgroup, 4-7 and 8-11 are the
// softmax warps of the tiles.  The first warpgroup hands registers on to the softmax, whose thread
// holds a row of 128 scores: 120 and 192 a thread took 6.0 - 6.1 ms for 32760 tokens x 12 heads in a
// sustained loop (cold 5.2 - 5.3), 56 and 224 6.4 - 6.7 (the issuing thread then recomputes its
// descriptors), 136 and 184 6.4 - 6.6, 168 each 6.9.
constexpr int THREADS = 384, REGS_FEW = 120, REGS_MANY = 192;
static_assert(128 * (REGS_FEW + 2 * REGS_MANY) <= THREADS * 168, "registers of the block at launch");

template <int DH, typename TI, bool BIAS>
struct Cfg {
  static constexpr int Q_BYTES = BQ * DH * 2, KV_BYTES = BK * DH * 2;
  static constexpr int HALVES = DH / 64, HALF_BYTES = 128 * 128;   // 64 columns of 128 rows
  static constexpr int RING = 131072 / KV_BYTES;                   // K/V tiles in flight
  static constexpr int BIAS_BYTES = BIAS ? (2 * (MAX_RADIUS + PAD) + 4) * 4 : 0;
  // output staging of a softmax warp: 32 rows x OC columns (64, or 32 where the bias table leaves no room)
  static constexpr int OC = DH == 128 && BIAS ? 32 : 64, STG_BYTES = 32 * OC * 2;
  static constexpr int Q_OFF = 0, RING_OFF = NQ * Q_BYTES, STG_OFF = RING_OFF + RING * KV_BYTES;
  static constexpr int BIAS_OFF = STG_OFF + 4 * NQ * STG_BYTES, BAR_OFF = BIAS_OFF + BIAS_BYTES;
  static constexpr int SMEM = 1024 + BAR_OFF + 512;
  static_assert(BAR_OFF % 16 == 0 && SMEM <= 232448, "shared memory of one block");
  __host__ __device__ static constexpr int s_col(int t) { return 256 * t; }
  __host__ __device__ static constexpr int o_col(int t) { return 256 * t + 128; }
  static constexpr bool HALF = std::is_same<TI, f16>::value;
  static constexpr uint32_t IDESC_S = HALF ? idesc_f16(128, BK, 0, 0) : idesc_bf16(128, BK, 0, 0);
  static constexpr uint32_t IDESC_O = HALF ? idesc_f16(128, DH, 0, 1) : idesc_bf16(128, DH, 0, 1);
};

enum : unsigned { SITE_Q = 0x501, SITE_KVF = 0x502, SITE_KVE = 0x503, SITE_S = 0x504, SITE_P = 0x505, SITE_O = 0x506,
                  SITE_TAIL = 0x507, SITE_DRAIN = 0x508, SITE_WORK = 0x509, SITE_WORKE = 0x50a, SITE_QE = 0x50b,
                  SITE_NEXT = 0x50c, SITE_TAB = 0x50d };

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

// One pair of query tiles, as warp 0 publishes it.
struct Work {
  int h, seq_row, l0, lq;   // head; the sequence's first row; the pair's first row in it; its rows
  int key_row, lk;          // the sequence's first key row; its keys
  int n_lo, nb;             // key blocks n_lo .. n_lo + nb - 1 (nb = 0: zeros; -1: no more work)
};

// max that keeps a NaN (a row with a NaN score ends as NaN instead of skipping it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float o;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
  return o;
}
__device__ __forceinline__ float max_nan3(float a, float b, float c) {
  float o;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(o) : "f"(a), "f"(b), "f"(c));
  return o;
}

// Asks for the next pending block of this grid to be cancelled; 16 bytes of answer go to
// `slot`, signalled on `bar`.
__device__ __forceinline__ void next_block_ask(void* slot, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(slot)),
               "r"(smem_u32(bar))
               : "memory");
}
// The cancelled block's index along x, or -1 if none was left.
__device__ __forceinline__ int next_block_answer(const void* slot) {
  uint32_t x = 0, got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}\n"
      : "+r"(x), "=r"(got)
      : "r"(smem_u32(slot))
      : "memory");
  return got ? static_cast<int>(x) : -1;
}

// Rows [lo, hi) of sequence s, inside the buffer whatever the offsets say.
__device__ __forceinline__ int2 extent(const int* cu, int s, int rows) {
  const int lo = min(max(cu[s], 0), rows);
  return make_int2(lo, max(min(cu[s + 1], rows), lo));
}
// Bias in log2 units; finite values stay finite (they absorb any score either way), NaN stays
// NaN (fmaxf would drop it).
__device__ __forceinline__ float log2_units(float b) { return isfinite(b) ? fminf(fmaxf(b * LOG2E, -1e30f), 1e30f) : b; }

// Pair `index` of the grid (whole warp): the sequences with the most key blocks come
// first (within each group of 32), and the pairs of one sequence run head after head, so
// that the blocks at work share one head's keys and values in L2.  False: no such pair.
__device__ __forceinline__ bool find_work(const Params& p, int index, int lane, Work& w) {
  int left = index;
  for (int s0 = 0; s0 < p.n_seq; s0 += 32) {
    const int s = s0 + lane;
    const bool in = s < p.n_seq;
    const int2 eq = in ? extent(p.cu_q, s, p.q_rows) : make_int2(0, 0);
    const int2 ek = in ? extent(p.cu_k, s, p.k_rows) : make_int2(0, 0);
    const int pairs = (eq.y - eq.x + NQ * BQ - 1) / (NQ * BQ), cost = (ek.y - ek.x + BK - 1) / BK;
    const int mine = pairs * p.heads;
    int before = 0;   // pairs of the sequences that come before this lane's
#pragma unroll 4
    for (int j = 0; j < 32; ++j) {
      const int pj = __shfl_sync(0xffffffffu, mine, j), cj = __shfl_sync(0xffffffffu, cost, j);
      if (cj > cost || (cj == cost && j < lane)) before += pj;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, left >= before && left - before < mine);
    if (hit) {
      const int src = __ffs(hit) - 1;
      w.seq_row = __shfl_sync(0xffffffffu, eq.x, src);
      w.lq = __shfl_sync(0xffffffffu, eq.y, src) - w.seq_row;
      w.key_row = __shfl_sync(0xffffffffu, ek.x, src);
      w.lk = __shfl_sync(0xffffffffu, ek.y, src) - w.key_row;
      left -= __shfl_sync(0xffffffffu, before, src);
      const int per_head = __shfl_sync(0xffffffffu, pairs, src);
      w.h = left / per_head;
      w.l0 = (left - w.h * per_head) * NQ * BQ;
      return true;
    }
    left -= __reduce_add_sync(0xffffffffu, mine);
  }
  return false;
}

template <int DH, typename TI, bool BIAS>
__global__ void __launch_bounds__(THREADS, 1)
k_attn_packed(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using C = Cfg<DH, TI, BIAS>;
  constexpr int RING = C::RING;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* tab = reinterpret_cast<float*>(smem + C::BIAS_OFF);   // tab[d + R + PAD] = bias at distance d
  uint8_t* answer = smem + C::BAR_OFF;                          // 16 bytes: the queue's answer
  Work* work = reinterpret_cast<Work*>(answer + 16);            // [2]
  uint64_t* bars = reinterpret_cast<uint64_t*>(work + 2);
  uint64_t* asked = bars;
  uint64_t* tail = bars + 1;              // a last V tile has landed (before its rows are cleared)
  uint64_t* work_full = bars + 2;         // [2]
  uint64_t* work_empty = bars + 4;        // [2]
  uint64_t* q_full = bars + 6;            // NQ
  uint64_t* q_empty = q_full + NQ;        // NQ
  uint64_t* kv_full = q_empty + NQ;       // RING
  uint64_t* kv_empty = kv_full + RING;    // RING
  uint64_t* s_full = kv_empty + RING;     // NQ
  uint64_t* p_part = s_full + NQ;         // NQ: the first 64 keys of P written
  uint64_t* p_full = p_part + NQ;         // NQ: all of P written
  uint64_t* o_done = p_full + NQ;         // NQ
  uint64_t* tab_bar = o_done + NQ;        // the softmax warps around a change of the bias table
  uint64_t* tdone = tab_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tdone + 1);
  static_assert(16 + 2 * sizeof(Work) + (6 + 2 * NQ + 2 * RING + 4 * NQ + 3) * 8 <= 512, "barrier space");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(asked, 1);
    mbar_init(tail, 1);
    for (int i = 0; i < 2; ++i) { mbar_init(&work_full[i], 1); mbar_init(&work_empty[i], 1 + 4 * NQ); }
    for (int s = 0; s < RING; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 1); }
    for (int t = 0; t < NQ; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_part[t], 4);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(tab_bar, 4 * NQ);
    mbar_init(tdone, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int R = p.radius;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_FEW));
    if (warp == 0) {
      // ------------------------------------------------------------ scheduler and TMA loader
      uint32_t issued = 0, last_par = 0;      // ring slots: loads in flight
      uint32_t q_count[NQ] = {0, 0}, tails = 0, round = 0;
      int pos = 0;                            // ring position
      bool ok = true;
      for (int index = blockIdx.x, n = 0; ok && index >= 0; ++round) {
        Work w;
        const bool found = find_work(p, index, lane, w);
        if (found) {
          const int nt = w.lq - w.l0 > BQ ? 2 : 1, l1 = min(w.l0 + NQ * BQ, w.lq);
          int n_hi = (w.lk + BK - 1) / BK;
          w.n_lo = 0;
          if constexpr (BIAS) {   // key blocks that no row sees, behind an end of -inf
            const float* tb = p.bias + static_cast<int64_t>(w.h) * (2 * R + 1);
            if (tb[0] == -INFINITY) w.n_lo = max(0, w.l0 - R + 1) / BK;
            if (tb[2 * R] == -INFINITY) n_hi = min(n_hi, (l1 - 1 + R - 1) / BK + 1);
          }
          w.nb = max(0, n_hi - w.n_lo);
          ok = mbar_wait_warp(&work_empty[n & 1], ((n >> 1) & 1) ^ 1u, SITE_WORKE);
          if (!ok) break;
          if (lane == 0) {
            work[n & 1] = w;
            mbar_arrive(&work_full[n & 1]);
          }
          ++n;
          const int kvc = w.h / p.group * DH;
          const int rest = w.lk - (n_hi - 1) * BK;   // keys of the last block that are the sequence's
          const bool clear = rest < BK;
          const int tiles = 2 * w.nb;                // K and V tiles in turn
          auto load = [&](const CUtensorMap* tm, int row, uint64_t* bar) {
            uint8_t* dst = smem + C::RING_OFF + (pos % RING) * C::KV_BYTES;
            mbar_arrive_expect_tx(bar, C::KV_BYTES);
            for (int hf = 0; hf < C::HALVES; ++hf)
              tma_load_3d(dst + hf * C::HALF_BYTES, tm, kvc + hf * 64, row, 0, bar);
          };
          if (w.nb && lane == 0) {
            for (int t = 0; t < nt && ok; ++t) {
              ok = mbar_wait(&q_empty[t], (q_count[t] & 1u) ^ 1u, SITE_QE);
              if (!ok) break;
              ++q_count[t];
              mbar_arrive_expect_tx(&q_full[t], C::Q_BYTES);
              for (int hf = 0; hf < C::HALVES; ++hf)
                tma_load_3d(smem + C::Q_OFF + t * C::Q_BYTES + hf * C::HALF_BYTES, &tmQ, w.h * DH + hf * 64,
                            w.seq_row + w.l0 + t * BQ, 0, &q_full[t]);
            }
            for (int i = 0; i < tiles && ok; ++i, ++pos) {
              const int slot = pos % RING;
              const uint32_t ph = (pos / RING) & 1u;
              ok = mbar_wait(&kv_empty[slot], ph ^ 1u, SITE_KVE);
              if (!ok) break;
              const int row = w.key_row + (w.n_lo + (i >> 1)) * BK;
              if (clear && i == tiles - 1) {   // the last V tile lands on its own barrier
                load(&tmV, row, tail);
                issued &= ~(1u << slot);       // what the slot held before has been used
                break;
              }
              load((i & 1) ? &tmV : &tmK, row, &kv_full[slot]);
              issued |= 1u << slot;
              last_par = (last_par & ~(1u << slot)) | (ph << slot);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          pos = __shfl_sync(0xffffffffu, pos, 0);
          if (w.nb && clear && ok) {
            // rows [rest, 128) of it to zero: a row is the same 128 bytes of each half in any swizzle
            ok = mbar_wait_warp(tail, tails & 1u, SITE_TAIL);
            ++tails;
            uint8_t* dst = smem + C::RING_OFF + (pos % RING) * C::KV_BYTES;
            for (int hf = 0; hf < C::HALVES; ++hf)
              for (int i = rest * 8 + lane; i < BK * 8; i += 32)
                reinterpret_cast<uint4*>(dst + hf * C::HALF_BYTES)[i] = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(&kv_full[pos % RING]);
            ++pos;
          }
          if (!ok) break;
        }
        // The next pending block's work: early enough to have the next pair's loads under way when
        // this one ends, and late enough to leave the work to blocks that are free sooner.  With a
        // ring of two key blocks (128-wide heads) the loads end two blocks before the pair; with four
        // (64-wide heads) a short sequence's would end at its start, so the K tile of the last block
        // but one has to be used first (prompts of 512 and 77 tokens x 64 heads: 20.2 -> 18.5 us;
        // 128-wide heads lost 2 % by the same).  A block without a pair asks no more (there are
        // such blocks behind the last pair, many of them where most of q lies outside the
        // sequences): those still pending start and end by themselves.
        index = -1;
        if (found) {
          if (RING > 4 && w.nb >= 2) {
            ok = mbar_wait_warp(&kv_empty[(pos - 4) % RING], ((pos - 4) / RING) & 1u, SITE_NEXT);
            if (!ok) break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(asked, 16);
            next_block_ask(answer, asked);
          }
          ok = mbar_wait_warp(asked, round & 1u, SITE_NEXT);
          if (ok) index = next_block_answer(answer);
          fence_proxy_async_smem();   // read before the next answer is written
          __syncwarp();
        }
        if (index < 0 && ok) {      // the end, published like a pair
          ok = mbar_wait_warp(&work_empty[n & 1], ((n >> 1) & 1) ^ 1u, SITE_WORKE);
          if (lane == 0 && ok) {
            work[n & 1].nb = -1;
            mbar_arrive(&work_full[n & 1]);
          }
        }
      }
      if (lane == 0) {
        for (int t = 0; t < NQ; ++t)
          if (q_count[t]) mbar_wait(&q_full[t], (q_count[t] - 1) & 1u, SITE_DRAIN);
        for (int s = 0; s < RING; ++s)
          if (issued & (1u << s)) mbar_wait(&kv_full[s], (last_par >> s) & 1u, SITE_DRAIN);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        bool ok = true;
        // descriptors as fixed high halves and low halves that step by 16-byte units
        const uint32_t r0 = smem_u32(smem + C::RING_OFF);
        const uint64_t dq0 = sdesc_sw128(smem_u32(smem + C::Q_OFF), 16, 1024), dk0 = sdesc_sw128(r0, 16, 1024);
        const uint64_t dv0 = sdesc_sw128(r0, C::HALF_BYTES, 1024);
        const uint32_t q_lo = static_cast<uint32_t>(dq0), k_lo = static_cast<uint32_t>(dk0);
        const uint32_t v_lo = static_cast<uint32_t>(dv0);
        const uint32_t s_hi = static_cast<uint32_t>(dq0 >> 32), v_hi = static_cast<uint32_t>(dv0 >> 32);
        uint32_t u = 0;                   // key blocks so far: K of block u is ring position 2u, V 2u + 1
        uint32_t blocks[NQ] = {0, 0};     // key blocks of each tile before this pair
        uint32_t q_count[NQ] = {0, 0};
        // one pair with NT live tiles (a compile-time number: the issuing thread runs in step
        // with the tensor pipe, and what it does between two MMAs is what the pipe waits for)
        auto pair = [&](auto nt_c, int nb) -> bool {
          constexpr int NT = decltype(nt_c)::value;
          auto issue_s = [&](int t, uint32_t kslot) {
            const uint32_t kb = k_lo + kslot * (C::KV_BYTES >> 4), qa = q_lo + t * (C::Q_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * C::HALF_BYTES + (kk & 3) * 32) >> 4;
              umma_ss_lh(tmem + C::s_col(t), qa + off, s_hi, kb + off, s_hi, C::IDESC_S, kk ? 1u : 0u);
            }
            umma_commit(&s_full[t]);
          };
          auto issue_pv = [&](int t, uint32_t v, int j) -> bool {   // block v, the pair's j-th
            const uint32_t slot = (2 * v + 1) % RING, vb = v_lo + slot * (C::KV_BYTES >> 4);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (!mbar_wait(part ? &p_full[t] : &p_part[t], (blocks[t] + j) & 1u, SITE_P)) return false;
              if (part == 0 && t == 0 && !mbar_wait(&kv_full[slot], ((2 * v + 1) / RING) & 1u, SITE_KVF)) return false;
              tc_fence_after();
#pragma unroll
              for (int kk = part * 4; kk < part * 4 + 4; ++kk)
                umma_ts_lh(tmem + C::o_col(t), tmem + C::s_col(t) + kk * 8, vb + kk * (2048 >> 4), v_hi, C::IDESC_O,
                           (j || kk) ? 1u : 0u);
            }
            if (t == NT - 1) umma_commit(&kv_empty[slot]);
            return true;
          };
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (!mbar_wait(&q_full[t], q_count[t]++ & 1u, SITE_Q)) return false;
          for (int j = 0; j < nb; ++j, ++u) {
            const uint32_t kslot = (2 * u) % RING;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if (j > 0 && !issue_pv(t, u - 1, j - 1)) return false;
              if (t == 0) {
                if (!mbar_wait(&kv_full[kslot], ((2 * u) / RING) & 1u, SITE_KVF)) return false;
                tc_fence_after();
              }
              issue_s(t, kslot);
            }
            umma_commit(&kv_empty[kslot]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) umma_commit(&q_empty[t]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (!issue_pv(t, u - 1, nb - 1)) return false;
            umma_commit(&o_done[t]);
            blocks[t] += nb;
          }
          return true;
        };
        for (uint32_t n = 0; ok; ++n) {
          if (!mbar_wait(&work_full[n & 1], (n >> 1) & 1u, SITE_WORK)) break;
          const int nb = work[n & 1].nb;
          const bool two = work[n & 1].lq - work[n & 1].l0 > BQ;
          mbar_arrive(&work_empty[n & 1]);
          if (nb < 0) break;
          if (nb == 0) continue;
          ok = two ? pair(std::integral_constant<int, 2>(), nb) : pair(std::integral_constant<int, 1>(), nb);
        }
        umma_commit(tdone);
        mbar_wait(tdone, 0, SITE_DRAIN);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_MANY));
    // ------------------------------------------------------------ softmax warps
    const int t = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lanes + C::s_col(t), o_addr = tmem + lanes + C::o_col(t);
    uint32_t blocks = 0, pairs = 0;   // of this tile so far
    [[maybe_unused]] int tab_h = -1;
    [[maybe_unused]] uint32_t tabs = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      // The pair stays published until its output is written: the loop over key blocks keeps
      // only what it needs of it in registers (the row of scores takes 128 of them).
      const Work& w = work[n & 1];
      if (!mbar_wait_warp(&work_full[n & 1], (n >> 1) & 1u, SITE_WORK)) break;
      const int nb = w.nb;
      if (nb < 0) break;
      if (nb == 0) {   // no row of the pair sees a key: zeros
        const int rows = min(w.lq - w.l0, NQ * BQ);
        for (int i = threadIdx.x - 128; i < rows * (DH / 8); i += 256) {
          const int64_t row = static_cast<int64_t>(w.seq_row) + w.l0 + i / (DH / 8);
          reinterpret_cast<uint4*>(p.o + row * p.o_rs + w.h * DH)[i % (DH / 8)] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if constexpr (BIAS) {
        if (nb && w.h != tab_h) {   // all softmax warps take the same pairs, so they change heads together
          const float* tb = p.bias + static_cast<int64_t>(w.h) * (2 * R + 1);
          auto all_softmax_warps = [&]() -> bool {   // an mbarrier: a warp that gave up must not leave the others waiting
            __syncwarp();
            if (lane == 0) mbar_arrive(tab_bar);
            return mbar_wait_warp(tab_bar, tabs++ & 1u, SITE_TAB);
          };
          if (!all_softmax_warps()) break;           // the old table has been used
          for (int i = threadIdx.x - 128; i < 2 * (R + PAD) + 1; i += 256)
            tab[i] = log2_units(tb[min(max(i - PAD, 0), 2 * R)]);
          if (!all_softmax_warps()) break;
          tab_h = w.h;
        }
      }
      if (nb == 0 || (t == 1 && w.lq - w.l0 <= BQ)) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&work_empty[n & 1]);
        continue;
      }
      const int keys = w.lk - w.n_lo * BK;                               // from the first key block on
      // that block's first key, counted from the warp's first row
      [[maybe_unused]] const int far = w.n_lo * BK - (w.l0 + t * BQ + quarter * 32);
      float m = -INFINITY, l = 0.f;
      for (int kb = 0; kb < nb; ++kb) {
        if (!mbar_wait_warp(&s_full[t], blocks & 1u, SITE_S)) { ok = false; break; }
        ++blocks;
        tc_fence_after();
        uint32_t a[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, a[c]);
        tmem_wait_ld();
        if constexpr (BIAS) {   // a = scale * s + bias, log2 units
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
          const int d = far + kb * BK;
          const bool past = d - 31 >= R, before = d + BK - 1 <= -R;   // warp-uniform
          if (past || before) {
            const float cb = tab[past ? 2 * (R + PAD) : 0];
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 x = ffma2(make_float2(__uint_as_float(a[c][k]), __uint_as_float(a[c][k + 1])), sc2,
                                       make_float2(cb, cb));
                a[c][k] = __float_as_uint(x.x);
                a[c][k + 1] = __float_as_uint(x.y);
              }
          } else {
            const float* tj = tab + (d - lane + R + PAD);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 x = ffma2(make_float2(__uint_as_float(a[c][k]), __uint_as_float(a[c][k + 1])), sc2,
                                       make_float2(tj[c * 32 + k], tj[c * 32 + k + 1]));
                a[c][k] = __float_as_uint(x.x);
                a[c][k + 1] = __float_as_uint(x.y);
              }
          }
        }
        const int valid = keys - kb * BK;
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
          for (int k = 0; k < 32; k += 2)
            m4[(k >> 1) & 3] = max_nan3(m4[(k >> 1) & 3], __uint_as_float(a[c][k]), __uint_as_float(a[c][k + 1]));
        float mx = max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3]));
        if constexpr (!BIAS) mx *= p.scale_log2;
        if (mx == INFINITY) mx = NAN;   // inf - inf below: the row is NaN, whichever pipe its exponentials take
        // the reference moves only when the maximum grew by more than the threshold (or is NaN);
        // P stays below 2^8 and the final 1 / l keeps the result exact
        const bool grow = !(mx <= m + tca::RESCALE_THRESHOLD);
        const float alpha = grow ? tca::ex2(m - mx) : 1.f;
        if (grow) m = mx;
        if (__any_sync(0xffffffffu, grow) && kb > 0) {
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
        // 16 keys: two in eight exponentials on the FMA pipe (k_attn_tc.cu).  A key that is left out has
        // P = 0 on either pipe: its value row may hold anything finite, and 2^-125 of 3e38 is 7.
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t pk[8];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float2 s2 = make_float2(__uint_as_float(a[c >> 1][(c & 1) * 16 + k]),
                                          __uint_as_float(a[c >> 1][(c & 1) * 16 + k + 1]));
            const float2 arg = BIAS ? fadd2(s2, nm2) : ffma2(s2, sc2, nm2);
            const float2 e = (k & 7) == 6 ? tca::exp2_fma2<true>(arg) : make_float2(tca::ex2(arg.x), tca::ex2(arg.y));
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
      // -------------------------------------------------------- output
      // (the next pair's S may already be computed meanwhile; its P V waits for this warp's P)
      if (!ok || !mbar_wait_warp(&o_done[t], pairs & 1u, SITE_O)) { ok = false; break; }
      ++pairs;
      tc_fence_after();
      const bool dead = m == -INFINITY;   // every score -inf: the row sees nothing
      const float inv = 1.f / l;
      // Through shared memory, so that a store writes whole row pieces: a thread holds one row,
      // and 16 bytes of 32 rows a store would occupy L1 for 32 lines each.  Row r's 16-byte chunk
      // j lies at chunk j ^ (r mod 8) (or j ^ (r / 2 mod 4) of 64-byte rows): no bank conflicts.
      const int row0 = w.l0 + t * BQ + quarter * 32, rows = w.lq - row0;   // the warp's first row, rows left
      bf16* dst = p.o + (static_cast<int64_t>(w.seq_row) + row0) * p.o_rs + w.h * DH;
      __syncwarp();
      if (lane == 0) mbar_arrive(&work_empty[n & 1]);
      constexpr int CPR = C::OC / 8, RPS = 32 / CPR;   // chunks per row, rows per store
      uint8_t* stg = smem + C::STG_OFF + (warp - 4) * C::STG_BYTES;
      auto chunk = [&](int r, int j) -> uint4* {
        return reinterpret_cast<uint4*>(stg) + r * CPR + (CPR == 8 ? j ^ (r & 7) : j ^ ((r >> 1) & 3));
      };
#pragma unroll 1
      for (int c = 0; c < DH; c += C::OC) {
#pragma unroll
        for (int c2 = 0; c2 < C::OC; c2 += 32) {
          uint32_t o[32];
          tmem_ld32(o_addr + c + c2, o);
          tmem_wait_ld();
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = dead ? 0.f : __uint_as_float(o[k]) * inv;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *chunk(lane, c2 / 8 + j) =
                make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                           pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < CPR; ++k) {
          const int r = k * RPS + lane / CPR, j = lane % CPR;
          if (r < rows) *reinterpret_cast<uint4*>(dst + r * p.o_rs + c + 8 * j) = *chunk(r, j);
        }
        __syncwarp();
      }
      tc_fence_before();
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
  using C = pka::Cfg<DH, TI, BIAS>;
  WD_TRY((allow_smem<pka::k_attn_packed<DH, TI, BIAS>>(C::SMEM)));
  // as many pairs of tiles as q_rows rows in n_seq sequences can make, times heads
  const int64_t pairs = (p.q_rows / (pka::NQ * pka::BQ) + static_cast<int64_t>(p.n_seq)) * p.heads;
  if (pairs > 0x7fffffff) { set_error("attention_packed: %lld tiles", (long long)pairs); return WD_ERR_SHAPE; }
  Trace tr(KC_ATTN_SELF, st);
  pka::k_attn_packed<DH, TI, BIAS><<<static_cast<unsigned>(pairs), pka::THREADS, C::SMEM, st>>>(tq, tk, tv, p);
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
  if (dh == 128 && p.bias) return launch_attn_packed<128, TI, true>(tq, tk, tv, p, st);
  if (dh == 128) return launch_attn_packed<128, TI, false>(tq, tk, tv, p, st);
  if (p.bias) return launch_attn_packed<64, TI, true>(tq, tk, tv, p, st);
  return launch_attn_packed<64, TI, false>(tq, tk, tv, p, st);
}

}  // namespace wd
