// attention_tc.cuh -- attention of chunks and prompts on the sm_100a tensor
// cores (tcgen05.mma kind::f16, accumulators in tensor memory).
//
// The mathematics, the items and the splits are those of attention.cuh; an
// item here is two row tiles of 128 (row t * G + g of a sequence is token t,
// head g of the group) over blocks of 128 keys.  Per block and tile T
//   S_T = Q_T K^T      A, B from shared memory, 128 x 128 fp32 into tensor memory
//   P_T = 2^(S_T - m)  one thread per row, bf16, over S_T's columns
//   O_T += P_T V       A from tensor memory, B = V as it lies (key rows, MN-major)
// The two tiles alternate: while one is in the softmax the tensor core works on
// the other.
//
// Running maximum: O_T is only rescaled when a row's maximum grows by more
// than 2^8 (log2 units); until then the old reference stays, probabilities are
// at most 2^8 and every sum is unchanged in exact arithmetic.
//
// Bound by the alternation of softmax and tensor core: a 4096-token prompt of
// the 2B heads takes 103 us (837 TFLOP/s, tensor pipe active 42 % of the time).
// A tile's turn is ~1930 cycles for 1024 of products; what it waits for most
// is the end of the product with V (~410), before the scores may overwrite the
// probabilities that product reads (the architecture orders the two only by
// completion).
//
// Warp roles (384 threads, one CTA per SM):
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row (TMEM lane)
//   warp 8          TMA producer: a ring of 128-key slots, K and V in turn,
//                   one load per page piece and 64 columns
//   warps 9, 11     MMA issuers of tile 0, 1 (11 also holds the tensor memory)
//   warp 10         zeroes the value rows past the last key (whatever those
//                   slots hold, 0 x NaN must not reach the sums)
#pragma once

#include "attention.cuh"
#include "common.cuh"
#include "gemv_tc.cuh"

namespace bitnet {

// D[tmem] (+)= A[smem] x B[smem]^T, kind::f16.
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D[tmem] (+)= A[tmem] x B[smem], kind::f16.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// kind::f16: D fp32, A and B bf16, A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t make_idesc_bf16(int M, int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// MN-major operand in the 128-byte swizzled layout: atoms of 64 elements (128
// bytes) x 8 k; `mn_stride` bytes to the next 64 elements, 1024 to the next 8 k.
__device__ __forceinline__ uint64_t make_sdesc_mn_sw128(uint32_t smem_addr, uint32_t mn_stride) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(mn_stride >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 32 lanes x 8 columns of 32-bit TMEM -> registers.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

// registers -> 32 lanes x 16 columns of 32-bit TMEM.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// Two fp32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

constexpr int kAttnTcThreads = 384;
constexpr int kAttnTcTarget = 148;     // most shares of a call: one per SM
constexpr int kAttnTcKeys = 128;       // keys per block
constexpr float kAttnTcLazy = 8.0f;    // growth of a row's maximum that rescales O

constexpr int kAttnTcList = 8;         // items laid out at a time

struct AttnTcItem {
  AttnPiece q;
  int count, tail, fix;                // blocks; count < 0: no item
  int cnt[2];                          // blocks of each tile
};

template <int DP>
struct AttnTcConfig {
  static constexpr int RT = 256;
  static constexpr int HALVES = DP / 64;                     // 64-column sub-tiles
  static constexpr int SUB = 128 * 128;                      // bytes of one
  static constexpr int TILE = HALVES * SUB;                  // Q tile, K or V block
  static constexpr int SLOTS = DP == 128 ? 4 : 8;            // five were no faster than four
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_BAR = OFF_KV + SLOTS * TILE;
  static constexpr int NUM_BARS = 2 * SLOTS + 16;
  static constexpr int OFF_PLAN = OFF_BAR + NUM_BARS * 8 + 16;
  static constexpr int OFF_ITEMS = OFF_PLAN + (int)((sizeof(PlanShared) + 15) & ~15u);
  static constexpr int SMEM =
      OFF_ITEMS + kAttnTcList * (int)sizeof(AttnTcItem) + 16 + 1024;            // + alignment slack
  static constexpr uint32_t S_COL = 0, O_COL = 256;          // + 128 T
  static_assert(OFF_PLAN % 16 == 0 && SMEM <= 227 * 1024, "shared memory");

  // Byte offset in a row tile of 16-byte chunk c of row r.  A softmax warp's 32
  // rows hold its queries, then its outputs or its fp32 sums: the four warps of a
  // tile go from item to item without a common barrier, so whatever a warp
  // puts there has to lie in its own rows.
  __host__ __device__ static constexpr int row_chunk(int r, int c) {
    return (c >> 3) * SUB + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }
};

// Every chunk of a row lies in the 128 bytes that each half of the tile has for
// that row, and no two coincide.
template <class C>
constexpr bool attn_tc_rows_apart() {
  for (int r = 0; r < 128; ++r) {
    unsigned seen = 0;
    for (int c = 0; c < 8 * C::HALVES; ++c) {
      const int at = C::row_chunk(r, c), half = at / C::SUB, in = at % C::SUB;
      if (half >= C::HALVES || in / 128 != r || in % 16 != 0) return false;
      seen |= 1u << (8 * half + in % 128 / 16);
    }
    if (seen != (1u << (8 * C::HALVES)) - 1u) return false;
  }
  return true;
}

template <int DP>
__global__ void __launch_bounds__(kAttnTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, AttnParams p, int box_rows) {
  using C = AttnTcConfig<DP>;
  static_assert(attn_tc_rows_apart<C>(), "a row's chunks lie in its own bytes");
  extern __shared__ uint8_t attn_tc_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(attn_tc_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;                         // slot filled (TMA bytes)
  uint64_t* empty = full + C::SLOTS;             // slot read (tcgen05.commit)
  uint64_t* qfull = empty + C::SLOTS;            // [T] Q tile written (4 warps)
  uint64_t* turn = qfull + 2;                    // [T] tile T may use the tensor core (issuer)
  uint64_t* sfull = turn + 2;                    // [T] scores ready (commit)
  uint64_t* pfull = sfull + 2;                   // [T][half] probabilities written (4 warps)
  uint64_t* odone = pfull + 4;                   // [T] product with V done (commit)
  uint64_t* vlast = odone + 2;                   // both issuers are at the last key's block
  uint64_t* vfix = vlast + 1;                    // its rows past that key are zeroed (warp 10)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  PlanShared& plan = *reinterpret_cast<PlanShared*>(smem + C::OFF_PLAN);
  AttnTcItem* items = reinterpret_cast<AttnTcItem*>(smem + C::OFF_ITEMS);
  int* listed = reinterpret_cast<int*>(items + kAttnTcList);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = p.D;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&qfull[t], 4);
      mbar_init(&turn[t], 1);
      mbar_init(&sfull[t], 1);
      mbar_init(&pfull[2 * t], 4);
      mbar_init(&pfull[2 * t + 1], 4);
      mbar_init(&odone[t], 1);
    }
    mbar_init(vlast, 2);
    mbar_init(vfix, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 11) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();                        // in this order: see rope_append_kernel
  grid_launch_dependents();
  const uint32_t tbase = *tmem_slot;
  make_plan(p, plan);

  uint32_t slot_it = 0;                          // ring position (producer, issuers, warp 10)
  uint32_t issued = 0;                           // slots whose loads are in flight or done
  uint32_t fixes = 0, both_done = 0;
  uint32_t tiles_done[2] = {0, 0};               // items in which tile T has blocks
  uint32_t blocks_done[2] = {0, 0};              // blocks of tile T so far

  // Every role walks the same items, each at its own pace: the barriers above
  // are all that ties them, so the producer fetches the next item's keys while
  // the softmax still writes the last one's rows.  Only the list of items is
  // common, laid out kAttnTcList at a time.
  auto lay_out = [&](int k, const AttnPiece& q) {
    AttnTcItem& job = items[k];
    job.q = q;
    // tile 0 ends with the keys its last row sees
    const int last0 = q.row0 + min(q.nrows, 128) - 1;
    const int end0 = (max(0, q.past + last0 / p.G + 1) + kAttnTcKeys - 1) / kAttnTcKeys;
    job.cnt[0] = max(0, min(q.blk1, end0) - q.blk0);
    job.cnt[1] = q.nrows > 128 ? q.blk1 - q.blk0 : 0;
    job.count = max(job.cnt[0], job.cnt[1]);
    // the block that holds the last key needs its value rows past it zeroed
    job.tail = q.kv_end - (q.blk0 + job.count - 1) * kAttnTcKeys;
    job.fix = job.count > 0 && job.tail < kAttnTcKeys;
  };
  auto walk = [&](auto&& role) {
    for (long long wave = 0;; wave += kAttnTcList) {
      __syncthreads();                           // the last list is done with
      if (threadIdx.x < kAttnTcList) items[threadIdx.x].count = -1;
      if (threadIdx.x == 0) *listed = 0;
      __syncthreads();
      if (plan.align != kWhole) {
        next_pieces(p, plan, kAttnTcList, *listed, lay_out);
      } else {
        for (int k = 0; k < kAttnTcList; ++k) {
          // items come longest first: every other wave runs the other way
          // round, so that a CTA's share evens out
          const int at = ((wave + k) & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
          const long long c = (wave + k) * gridDim.x + at;
          if (c < plan.total) find_item(p, plan, c, [&](const AttnPiece& q) { lay_out(k, q); });
        }
        if (threadIdx.x == 0) *listed = wave * gridDim.x < plan.total ? kAttnTcList : 0;
      }
      __syncthreads();
      const int n = *listed;
      if (n == 0) break;
      for (int k = 0; k < n; ++k) {
        const AttnTcItem job = items[k];
        if (job.count < 0) continue;
        role(job);
        slot_it += 2 * job.count;
        blocks_done[0] += job.cnt[0];
        blocks_done[1] += job.cnt[1];
        both_done += min(job.cnt[0], job.cnt[1]);
        if (job.cnt[0] > 0) ++tiles_done[0];
        if (job.cnt[1] > 0) ++tiles_done[1];
        if (job.fix) ++fixes;
        // another warp may set the flag at any time: the whole warp leaves or stays
        if (__any_sync(0xffffffffu, *abort_flag)) break;
      }
      if (__syncthreads_or(*abort_flag)) break;
    }
  };

  // 256 x 224 + 128 x 56 registers: the 384 x 168 of the launch
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    walk([&](const AttnTcItem& job) {
      // --------------------------------------------------------- softmax
      const int t = warp >> 2, r = threadIdx.x & 127;        // tile and row in it
      const int row = 128 * t + r;                           // of the item
      const bool live = row < job.q.nrows;
      // Rows move 16 bytes a lane, so that a warp takes whole rows at a time:
      // LR lanes per row, rows sub, sub + 32 / LR, ... of the warp's 32.
      constexpr int LR = DP / 8, STEP = 32 / LR;
      const int ch = lane % LR, sub = lane / LR, wrow = 32 * (warp & 3);
      uint8_t* qtile = smem + t * C::TILE;
      // element offset of the first such row, and the way to the next
      const int gr0 = job.q.row0 + 128 * t + wrow + sub;
      const int tok0 = gr0 / p.G, g0 = gr0 - tok0 * p.G;
      const int tok_step = STEP / p.G, g_step = STEP - tok_step * p.G;
      auto each_row = [&](auto&& f) {
        int tok = tok0, g = g0;
#pragma unroll
        for (int k = 0; k < LR; ++k) {
          f(k, ((long long)(job.q.c0 + tok) * p.qh + (long long)job.q.head * p.G + g) * D + 8 * ch);
          tok += tok_step;
          g += g_step;
          if (g >= p.G) {
            g -= p.G;
            ++tok;
          }
        }
      };
      // (without blocks there is nothing to wait for on either side: the softmax
      // would run ahead of its issuer by more than one phase of the barrier)
      if (job.cnt[t] > 0) {
        uint4 u[LR];
        each_row([&](int k, long long off) {
          u[k] = make_uint4(0, 0, 0, 0);
          if (128 * t + wrow + sub + STEP * k < job.q.nrows && 8 * ch < D)
            u[k] = *reinterpret_cast<const uint4*>(
                reinterpret_cast<const __nv_bfloat16*>(p.Q) + off);
        });
#pragma unroll
        for (int k = 0; k < LR; ++k) {
          const int rr = wrow + sub + STEP * k;
          *reinterpret_cast<uint4*>(qtile + C::row_chunk(rr, ch)) = u[k];
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[t]);
      }
      const uint32_t lanes = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
      const uint32_t scol = lanes + C::S_COL + 128u * t, ocol = lanes + C::O_COL + 128u * t;
      // keys this row sees
      const int lim = live ? job.q.past + (job.q.row0 + row) / p.G + 1 : 0;
      // keys that the warp's rows all see
      const int lim_warp = __reduce_min_sync(0xffffffffu, lim);
      float m = -INFINITY;                                   // reference, log2 units
      uint64_t l2 = 0;                                       // two partial sums
      bool ok = true;
#pragma unroll 1
      for (int i = 0; i < job.cnt[t]; ++i) {
        // (all lanes agree: what follows is executed by whole warps)
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&sfull[t], (blocks_done[t] + i) & 1u, abort_flag));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(scol + 32u * q, s[q]);
        tmem_ld_wait();
        const int key0 = (job.q.blk0 + i) * kAttnTcKeys;
        if (key0 + kAttnTcKeys > lim_warp) {
          const int n = lim - key0;
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * q + k >= n) s[q][k] = 0xff800000u;    // -inf
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mx[q] = max3(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]),
                       __uint_as_float(s[q][2]));
#pragma unroll
          for (int k = 3; k < 31; k += 2)
            mx[q] = max3(mx[q], __uint_as_float(s[q][k]), __uint_as_float(s[q][k + 1]));
          mx[q] = fmaxf(mx[q], __uint_as_float(s[q][31]));
        }
        const float mnew =
            fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        if (i == 0) m = mnew;
        // The first half's powers are taken relative to the reference of the
        // blocks before, beside the search for this block's maximum; only if
        // that turns out to have outgrown the reference are they taken again.
        const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2);
        uint64_t lh = 0;
        uint32_t ph[32];
        auto powers = [&](int half, float base) {
          const uint64_t base2 = pack_f32x2(base, base);
          lh = 0;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int q = 2 * half + (k >> 4), e = 2 * (k & 15);
            const uint64_t z = fma_f32x2(
                pack_f32x2(__uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1])), scale2, base2);
            float u, v;
            unpack_f32x2(z, u, v);
            u = ex2(u);
            v = ex2(v);
            lh = add_f32x2(lh, pack_f32x2(u, v));
            ph[k] = pack_bf16x2(u, v);
          }
        };
        auto hand_over = [&](int half) {
          tmem_st_32x32b_x32(scol + 32u * half, ph);
          l2 = add_f32x2(l2, lh);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[2 * t + half]);
        };
        float base = m == -INFINITY ? 0.0f : -m;
        powers(0, base);
        const bool grow = mnew > m + kAttnTcLazy || (m == -INFINITY && mnew != -INFINITY);
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(m - mnew) : 1.0f;
          l2 = fma_f32x2(l2, pack_f32x2(f, f), 0);
          if (grow) m = mnew;
          base = m == -INFINITY ? 0.0f : -m;
          // the product of the last block is done: its completion precedes
          // that of the scores just read
#pragma unroll 1
          for (int d = 0; d < DP; d += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(ocol + d, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st_32x32b_x16(ocol + d, o);
          }
          tmem_st_wait();
          powers(0, base);
        }
        hand_over(0);
        powers(1, base);
        hand_over(1);
      }
      // ---- the rows' sums
      float l, lb;
      unpack_f32x2(l2, l, lb);
      l += lb;
      if (ok && job.cnt[t] > 0)
        ok = __all_sync(0xffffffffu, mbar_wait(&odone[t], (blocks_done[t] + job.cnt[t] - 1) & 1u,
                                               abort_flag));
      tc_fence_after();
      if (ok && 128 * t < job.q.nrows) {
        float* part = job.q.slot >= 0 ? p.part + (long long)job.q.slot * C::RT * (D + 2) : nullptr;
        const float inv = job.q.slot >= 0 ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
        if (job.q.slot >= 0 && live) {
          part[row] = m;
          part[C::RT + row] = l;
        }
        // The rows leave through the warp's own rows of the Q tile, which the
        // products are done with, so that a warp stores whole rows: bf16, or fp32
        // sums, as many columns at a time as fit a row's bytes.
        auto columns = [&](int d, float (&x)[8]) {
          uint32_t o[8];
          if (job.cnt[t] > 0) {
            tmem_ld_32x32b_x8(ocol + d, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(o[k]) * inv;
        };
        if (job.q.slot < 0) {
#pragma unroll 4
          for (int d = 0; d < DP; d += 8) {
            float x[8];
            columns(d, x);
            store_bf16<8>(reinterpret_cast<__nv_bfloat16*>(qtile + C::row_chunk(r, d / 8)), x);
          }
          __syncwarp();
          each_row([&](int k, long long off) {
            const int rr = wrow + sub + STEP * k;
            if (128 * t + rr < job.q.nrows && 8 * ch < D)
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.O) + off) =
                  *reinterpret_cast<const uint4*>(qtile + C::row_chunk(rr, ch));
          });
          __syncwarp();
        } else {
          // lanes per row: its chunks of four columns; rows at a time
          constexpr int WL = 8 * C::HALVES, W = 4 * WL, WSTEP = 32 / WL;
#pragma unroll 1
          for (int d0 = 0; d0 < DP; d0 += W) {
#pragma unroll 4
            for (int d = 0; d < W; d += 8) {
              float x[8];
              columns(d0 + d, x);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4*>(qtile + C::row_chunk(r, d / 4 + e)) =
                    make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
            __syncwarp();
            const int wch = lane % WL, d = d0 + 4 * wch;
#pragma unroll 4
            for (int rr = wrow + lane / WL; rr < wrow + 32; rr += WSTEP) {
              if (128 * t + rr < job.q.nrows && d < D)
                *reinterpret_cast<float4*>(part + 2 * C::RT + (long long)(128 * t + rr) * D + d) =
                    *reinterpret_cast<const float4*>(qtile + C::row_chunk(rr, wch));
            }
            __syncwarp();
          }
        }
      }
      tc_fence_before();
    });
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 8) {
      walk([&](const AttnTcItem& job) {
      // -------------------------------------------------------- producer
      const int pieces = kAttnTcKeys / box_rows;             // loads per block and 64 columns
      bool ok = true;
      for (int i = 0; i < 2 * job.count; ++i) {
        const uint32_t it = slot_it + i;
        const int key0 = (job.q.blk0 + (i >> 1)) * kAttnTcKeys;
        // lane x < pieces: place of piece x (out of range: the load fills zeros)
        const int key = key0 + lane * box_rows;
        const bool live = lane < pieces && key < job.q.kv_end;
        int page = -1;
        if (live) {
          page = __ldg(p.pb.table + (long long)job.q.b * p.pb.stride + key / p.pb.page_size);
          if (page < 0 || page >= p.pb.num_pages) {
            record_device_error(DEV_ERR_INDEX);
            page = p.pb.num_pages;
          }
        }
        const uint32_t st = it % C::SLOTS, ph = (it / C::SLOTS) & 1u;
        if (!mbar_wait(&empty[st], ph ^ 1u, abort_flag)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t n_live = __popc(__ballot_sync(0xffffffffu, live));
        if (lane == 0)
          mbar_arrive_expect_tx(&full[st], n_live * (uint32_t)box_rows * 128u * C::HALVES);
        __syncwarp();
        if (live) {
          uint8_t* dst = smem + C::OFF_KV + st * C::TILE + lane * box_rows * 128;
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(dst + h * C::SUB, (i & 1) ? &tm_v : &tm_k, &full[st], 64 * h,
                        key % p.pb.page_size, page * p.kvh + job.q.head);
        }
        issued = it + 1;
      }
      });
    } else if (warp == 9 || warp == 11) {
      const int t = warp == 9 ? 0 : 1;
      walk([&](const AttnTcItem& job) {
      // -------------------------------------------------- MMA issuer, tile t
      // One issuer per tile: each waits for its own probabilities while the
      // tensor core works for the other (one issuer for both in turn left it
      // idle half of the time).  The whole warp follows the loop and one
      // elected lane issues, so that descriptors live in uniform registers.
      // A parity wait takes the phase two before for its own if the one between
      // is still open, and misses its own if the barrier gets two ahead.  So no
      // barrier can complete a phase before all its waiters have seen the last:
      // slots need both issuers' release, vlast both their arrivals, the others
      // go to and fro between two sides.  Of odone the issuer waits for every
      // phase but an item's last and the softmax for that one only; each knows
      // the phase before complete by other means: scores are issued after the
      // product before them is done, so the softmax that read an item's last
      // scores waits in the open phase, and queries are handed over after the
      // softmax saw the last item's end, so the issuer that got them does.
      const int cnt = t == 0 ? job.cnt[0] : job.cnt[1];
      const uint32_t q_phase = t == 0 ? tiles_done[0] : tiles_done[1];
      bool ok = true;
      if (cnt > 0) ok = __all_sync(0xffffffffu, mbar_wait(&qfull[t], q_phase & 1u, abort_flag));
      if (job.count > 0) {
        constexpr uint32_t idesc_s = make_idesc_bf16(128, 128, false);
        constexpr uint32_t idesc_o = make_idesc_bf16(128, DP, true);
        const bool leader = elect_one();
        const uint32_t kva = smem_u32(smem) + C::OFF_KV;
        const uint64_t qd = make_sdesc_sw128(smem_u32(smem) + t * C::TILE);
        const uint32_t dcol = tbase + C::O_COL + 128u * t, scol = tbase + C::S_COL + 128u * t;
        const uint32_t done0 = t == 0 ? blocks_done[0] : blocks_done[1];
        const int both = min(job.cnt[0], job.cnt[1]);
        // pass: hand the turn over half way, since it takes the other issuer
        // about as long as the second half to notice
        auto scores = [&](uint32_t st, bool pass) {
          const uint64_t kd = make_sdesc_sw128(kva + st * C::TILE);
          if (leader) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
              const uint64_t o = (uint64_t)((k >> 2) * (C::SUB >> 4) + 2 * (k & 3));
              mma_f16_ss(scol, qd + o, kd + o, idesc_s, k != 0);
              if (k == DP / 32 - 1 && pass) mbar_arrive(&turn[1 - t]);
            }
            tc_commit(&sfull[t]);
            tc_commit(&empty[st]);
          }
          __syncwarp();
        };
        uint32_t it = slot_it;
        // a slot is free once both issuers have let go of it
        ok = ok && mbar_wait(&full[it % C::SLOTS], (it / C::SLOTS) & 1u, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && cnt > 0) {
          tc_fence_after();
          scores(it % C::SLOTS, false);
        } else if (ok && lane == 0) {
          mbar_arrive(&empty[it % C::SLOTS]);
        }
        ++it;
        for (int i = 0; ok && i < job.count; ++i, it += 2) {
          const uint32_t sv = it % C::SLOTS, sk = (it + 1) % C::SLOTS;
          const bool more = i + 1 < job.count;
          if (i >= cnt) {                        // the other tile sees more keys
            ok = mbar_wait(&full[sv], (it / C::SLOTS) & 1u, abort_flag);
            if (job.fix && !more) {
              if (ok && leader) mbar_arrive(vlast);
              ok = ok && mbar_wait(vfix, fixes & 1u, abort_flag);
            }
            ok = __all_sync(0xffffffffu, ok);    // every lane has seen the phase
            if (ok && lane == 0) mbar_arrive(&empty[sv]);
            if (ok && more) {
              ok = __all_sync(0xffffffffu,
                              mbar_wait(&full[sk], ((it + 1) / C::SLOTS) & 1u, abort_flag));
              if (ok && lane == 0) mbar_arrive(&empty[sk]);
            }
            continue;
          }
          ok = mbar_wait(&full[sv], (it / C::SLOTS) & 1u, abort_flag);
          if (job.fix && !more) {
            if (ok && leader) mbar_arrive(vlast);
            ok = ok && mbar_wait(vfix, fixes & 1u, abort_flag);
          }
          const uint64_t vd = make_sdesc_mn_sw128(kva + sv * C::TILE, C::SUB);
          // While both tiles have blocks they take turns of one product with V
          // and the next scores: one tile's runs while the other is in the
          // softmax.  The first half of the keys goes ahead of the second.
          const uint32_t nth = both_done + i;
          const bool turns = i < both;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && mbar_wait(&pfull[2 * t + h], (done0 + i) & 1u, abort_flag);
            if (h == 0 && turns && (t == 1 || nth > 0))
              ok = ok && mbar_wait(&turn[t], (t == 0 ? nth - 1 : nth) & 1u, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              tc_fence_after();
              if (leader) {
#pragma unroll
                for (int k = 4 * h; k < 4 * h + 4; ++k)
                  mma_f16_ts(dcol, scol + 8u * k, vd + (uint64_t)(128 * k), idesc_o,
                             k == 0 ? i != 0 : 1);
                if (h == 1) {
                  tc_commit(&odone[t]);
                  tc_commit(&empty[sv]);
                }
              }
              __syncwarp();
            }
          }
          if (more && i + 1 < cnt) {
            ok = ok && mbar_wait(&full[sk], ((it + 1) / C::SLOTS) & 1u, abort_flag);
            // the scores overwrite the probabilities the product reads
            ok = ok && mbar_wait(&odone[t], (done0 + i) & 1u, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              tc_fence_after();
              scores(sk, turns);
            }
          } else if (more) {
            ok = ok && mbar_wait(&full[sk], ((it + 1) / C::SLOTS) & 1u, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && lane == 0) mbar_arrive(&empty[sk]);
          }
          if (ok && turns && leader && !(more && i + 1 < cnt)) mbar_arrive(&turn[1 - t]);
        }
      }
      __syncwarp();
      });
    } else if (warp == 10) {
      walk([&](const AttnTcItem& job) {
      // ------------------------------------------ value rows past the end
      if (job.fix) {
        const uint32_t it = slot_it + 2 * job.count - 1;
        mbar_wait(vlast, fixes & 1u, abort_flag);
        uint8_t* v = smem + C::OFF_KV + (it % C::SLOTS) * C::TILE;
        constexpr int LR = 8 * C::HALVES;          // lanes per row
        v += ((lane >> 3) % C::HALVES) * C::SUB + (lane & 7) * 16;
        for (int r = job.tail + lane / LR; r < kAttnTcKeys; r += 32 / LR)
          *reinterpret_cast<uint4*>(v + r * 128) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(vfix);
      }
      });
    }
  }

  // Never leave tensor-core work or bulk copies in flight (an abort can).
  if (__any_sync(0xffffffffu, *abort_flag)) {
    if ((warp == 9 || warp == 11) && elect_one()) {
      uint64_t* bar = &odone[warp == 9 ? 0 : 1];
      tc_commit(bar);
      mbar_wait(bar, 0, nullptr, 100000000ull);
      mbar_wait(bar, 1, nullptr, 100000000ull);
    }
    if (warp == 8 && lane == 0) {
      const uint32_t last = issued < (uint32_t)C::SLOTS ? issued : (uint32_t)C::SLOTS;
      for (uint32_t i = 0; i < last; ++i) {
        const uint32_t j = issued - 1 - i;
        mbar_wait(&full[j % C::SLOTS], (j / C::SLOTS) & 1u, nullptr, 100000000ull);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 11) tmem_dealloc(tbase, 512);
}

}  // namespace bitnet
