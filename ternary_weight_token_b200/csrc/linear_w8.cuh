// linear_w8.cuh -- int8 activations x int8 weights with a scale per token and
// per output channel, on the sm_100a tensor cores (tcgen05.mma kind::i8).
//
// For the layers of a W1.58A8 model that are not ternary (the output head,
// first and last blocks): the activation codes are those of the BitLinear
// quantiser (q = rint(x s), s = 127 / max|x| per token) and a weight row is
// quantised the same way, so
//   y[m][n] = (sum_k qx[m][k] qw[n][k]) / (sx[m] sw[n]),
// the sum exact in int32 (K <= 16384: below 2^28).
//
// D^T[n][m]: the A operand is 128 weight rows, the B operand a tile of BN
// tokens, both int8 rows in shared memory (128 bytes of K per stage, TMA,
// 128-byte swizzle); int32 accumulators in tensor memory, two buffers so that
// the epilogue of one tile overlaps the products of the next.  An epilogue
// thread holds one weight row, so its channel factor stays in a register and
// a warp stores 32 consecutive outputs of one token.
//
// Few tokens: the weights are read once from HBM, which is what bounds it
// (one token, 128256 x 2560: 54.7 us, 6.0 TB/s); many tokens: the tensor cores
// (4096 tokens, 6912 x 2560: 58 us, 2.5 POPS).  The token tile (16 .. 256) is
// the host's choice.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "gemv.cuh"
#include "gemv_tc.cuh"

namespace bitnet {

// D[tmem] (+)= A[smem] x B[smem]^T, kind::i8 (int32 accumulate).
__device__ __forceinline__ void mma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// kind::i8, both operands signed 8-bit, K-major.
__host__ __device__ constexpr uint32_t make_idesc_s8(int M, int N) {
  return make_idesc_i8(M, N) | (1u << 7);
}

template <int BN_, int STAGES_>
struct W8Config {
  static constexpr int BN = BN_;
  static constexpr int BM = 128;
  static constexpr int BK = 128;
  static constexpr int STAGES = STAGES_;
  static constexpr int W_STAGE = BM * BK, X_STAGE = BN * BK;
  // two groups of four epilogue warps share a tile's tokens where they have
  // 64 or more: one group alone is slower than the products it follows
  static constexpr int GROUPS = BN >= 64 ? 2 : 1;
  static constexpr int THREADS = 128 + 128 * GROUPS;
  static constexpr int TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
  static constexpr int OFF_X = STAGES * W_STAGE;
  static constexpr int OFF_BAR = OFF_X + STAGES * X_STAGE;
  static constexpr int NUM_BARS = 2 * STAGES + 7;
  static constexpr int OFF_TOK = OFF_BAR + ((NUM_BARS * 8 + 16 + 127) & ~127);  // [2][BN] fp32
  static constexpr int SMEM_ALLOC = OFF_TOK + 2 * BN * 4 + 1024;
  static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS <= 512, "tensor memory");
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory");
};

struct W8Params {
  const float* xs;            // [M]
  const float* ws;            // [N]
  void* Y;                    // [M][N]
  const void* resid;
  int M, N, num_kb;
  int tiles_n, num_tiles;
  int out_type, flags;
};

// One thread's CW outputs (one weight row, consecutive tokens) of a tile: at =
// first element, stride = elements between tokens, the first `live` tokens
// stored.  One instance per output type and epilogue, so that the unrolled
// code stays small.
template <int CW, int TYPE, bool SILU, bool RESID>
__device__ __forceinline__ void w8_store(const uint32_t (&v)[CW], float wf, const float* tok,
                                         void* Y, const void* resid, size_t at, size_t stride,
                                         int live) {
  if constexpr (TYPE == OUT_I32) {
    int32_t* y = reinterpret_cast<int32_t*>(Y) + at;
#pragma unroll
    for (int j = 0; j < CW; ++j, y += stride)
      if (j < live) *y = (int)v[j];
  } else {
    using T = typename std::conditional<TYPE == OUT_BF16, __nv_bfloat16, float>::type;
    float r[CW];
    if constexpr (RESID) {                       // independent loads first
      const T* q = reinterpret_cast<const T*>(resid) + at;
#pragma unroll
      for (int j = 0; j < CW; ++j, q += stride) r[j] = j < live ? static_cast<float>(*q) : 0.0f;
    }
    T* y = reinterpret_cast<T*>(Y) + at;
    // the sum, two reciprocals, their product and the last product: 2^-24 each
    // (the quotient itself, three roundings, costs 69 us for 55 at 4096 tokens,
    // 6912 x 2560; a reciprocal with one correction 59)
    auto value = [&](int j) {
      float x = __fmul_rn(__int2float_rn((int)v[j]), __fmul_rn(wf, tok[j]));
      if constexpr (SILU) x = silu_f32(x);
      if constexpr (RESID) x = __fadd_rn(r[j], x);
      return static_cast<T>(x);
    };
    if (live == CW) {                            // a full step: no test per token
#pragma unroll
      for (int j = 0; j < CW; ++j, y += stride) *y = value(j);
    } else {
#pragma unroll
      for (int j = 0; j < CW; ++j, y += stride)
        if (j < live) *y = value(j);
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    linear_w8_kernel(const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_w, W8Params p) {
  extern __shared__ uint8_t w8_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(w8_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;
  uint64_t* empty = bars + C::STAGES;
  uint64_t* accfull = bars + 2 * C::STAGES;
  uint64_t* accempty = accfull + 2;
  uint64_t* drain = accempty + 2;
  uint64_t* tokbar = drain + 1;                  // a tile's token factors are written
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_tok = reinterpret_cast<float*>(smem + C::OFF_TOK);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 4 * C::GROUPS);
      mbar_init(&tokbar[b], 4 * C::GROUPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();                        // in this order: see rope_append_kernel
  grid_launch_dependents();
  const uint32_t tbase = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      for (int tile = blockIdx.x; tile < p.num_tiles; tile += gridDim.x) {
        const int tn = tile % p.tiles_n, tm = tile / p.tiles_n;
        for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
          const uint32_t st = it % C::STAGES, ph = (it / C::STAGES) & 1u;
          if (!mbar_wait(&empty[st], ph ^ 1u, abort_flag)) goto producer_done;
          mbar_arrive_expect_tx(&full[st], C::W_STAGE + C::X_STAGE);
          tma_load_2d(smem + st * C::W_STAGE, &tm_w, &full[st], kb * C::BK, tn * C::BM);
          tma_load_2d(smem + C::OFF_X + st * C::X_STAGE, &tm_x, &full[st], kb * C::BK, tm * C::BN);
        }
      }
    producer_done:
      // never leave bulk copies in flight
      const uint32_t last = it < (uint32_t)C::STAGES ? it : (uint32_t)C::STAGES;
      for (uint32_t i = 0; i < last; ++i) {
        const uint32_t j = it - 1 - i;
        mbar_wait(&full[j % C::STAGES], (j / C::STAGES) & 1u, nullptr, 100000000ull);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc_s8(C::BM, C::BN);
      uint32_t it = 0, tcount = 0;
      for (int tile = blockIdx.x; tile < p.num_tiles; tile += gridDim.x, ++tcount) {
        const uint32_t ab = tcount & 1u, use = tcount >> 1;
        if (!mbar_wait(&accempty[ab], (use & 1u) ^ 1u, abort_flag)) break;
        tc_fence_after();
        const uint32_t d_col = tbase + ab * C::BN;
        for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
          const uint32_t st = it % C::STAGES, ph = (it / C::STAGES) & 1u;
          if (!mbar_wait(&full[st], ph, abort_flag)) goto mma_done;
          tc_fence_after();
          const uint32_t wa = smem_u32(smem + st * C::W_STAGE);
          const uint32_t xa = smem_u32(smem + C::OFF_X + st * C::X_STAGE);
#pragma unroll
          for (int j = 0; j < C::BK / 32; ++j)
            mma_i8_ss(d_col, make_sdesc_sw128(wa + 32u * j), make_sdesc_sw128(xa + 32u * j),
                      idesc, (kb | j) != 0);
          tc_commit(&empty[st]);
        }
        tc_commit(&accfull[ab]);
      }
    mma_done:
      tc_commit(drain);
      mbar_wait(drain, 0, nullptr, 100000000ull);
    }
  } else if (warp >= 4) {
    const int q = warp & 3, group = (warp - 4) >> 2, et = threadIdx.x - 128;
    const uint32_t lane_base = tbase + ((uint32_t)(32 * q) << 16);
    uint32_t tcount = 0;
    for (int tile = blockIdx.x; tile < p.num_tiles; tile += gridDim.x, ++tcount) {
      const int tn = tile % p.tiles_n, tm = tile / p.tiles_n;
      const uint32_t ab = tcount & 1u, aph = (tcount >> 1) & 1u;
      const int m0 = tm * C::BN;
      const int n = tn * C::BM + 32 * q + lane;
      const bool n_ok = n < p.N;
      // this buffer was last read two tiles ago, before its readers arrived for
      // the tile between
      float* tok = s_tok + ab * C::BN;
      for (int j = et; j < C::BN; j += 128 * C::GROUPS)
        tok[j] = m0 + j < p.M ? __fdiv_rn(1.0f, p.xs[m0 + j]) : 0.0f;
      const float wf = n_ok ? __fdiv_rn(1.0f, p.ws[n]) : 0.0f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&tokbar[ab]);
      const bool ok = mbar_wait(&tokbar[ab], aph, abort_flag) &&
                      mbar_wait(&accfull[ab], aph, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      constexpr int CW = 16;                      // tokens per step
#pragma unroll 1
      for (int c = CW * group; c < C::BN; c += CW * C::GROUPS) {
        if (m0 + c >= p.M) break;
        uint32_t v[CW];
        tmem_ld_32x32b_x16(lane_base + ab * C::BN + c, v);
        tmem_ld_wait();
        if (n_ok) {
          const size_t at = (size_t)(m0 + c) * p.N + n;
          const int live = min(CW, p.M - (m0 + c));
          const bool silu = (p.flags & EPI_SILU) != 0, res = (p.flags & EPI_RESIDUAL) != 0;
          auto store = [&](auto type, auto si, auto re) {
            w8_store<CW, decltype(type)::value, decltype(si)::value, decltype(re)::value>(
                v, wf, tok + c, p.Y, p.resid, at, (size_t)p.N, live);
          };
          auto pick = [&](auto type) {
            if (silu && res)
              store(type, std::true_type{}, std::true_type{});
            else if (silu)
              store(type, std::true_type{}, std::false_type{});
            else if (res)
              store(type, std::false_type{}, std::true_type{});
            else
              store(type, std::false_type{}, std::false_type{});
          };
          if (p.out_type == OUT_BF16)
            pick(std::integral_constant<int, OUT_BF16>{});
          else if (p.out_type == OUT_F32)
            pick(std::integral_constant<int, OUT_F32>{});
          else
            store(std::integral_constant<int, OUT_I32>{}, std::false_type{}, std::false_type{});
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&accempty[ab]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tbase, C::TMEM_COLS);
}

}  // namespace bitnet
