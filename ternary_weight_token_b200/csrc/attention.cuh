// attention.cuh -- causal attention of the new tokens of a batch over their
// paged key/value cache: work plan, the mma.sync kernel, and the join of
// split sequences.
//
// nnterp encyclopedia "bitnet", "Printout": 20 query heads over 5 key/value
// heads of 128.
//
// Row r of sequence b at position p sees keys 0 .. p of its own sequence:
//   o = sum_j softmax_j(scale q . k_j) v_j,
// computed in one pass with a running maximum m and sum l (fp32):
//   m' = max(m, z_j), l' = l 2^(m - m') + sum 2^(z_j - m'), o' likewise,
// with z in units of log2 (scale * log2 e folded into one factor).  A row
// that sees no key gives zeros.
//
// The query heads that share a key/value head are rows of one tile: row
// t * G + g of a sequence is token t, head g of the group, so a tile reads
// its keys and values once for all of them.
//
// Work: a tile of rows (RT) times one key/value head is an item.  Its length is
// its keys (a linear count, so that items before it add up in closed form) and
// one block more for its start and end.  Where the items are too few to deal
// out evenly, all lengths of the call are laid end to end and cut into one
// equal share per CTA, on the device, from what it finds there (so a captured
// graph keeps fitting as the cache grows).  A CTA whose share starts or ends
// inside an item writes unnormalised sums and statistics to the workspace and
// the join kernel adds them; an item inside one share is written directly.  A
// call too small to fill the GPU with shares of the smallest size takes those,
// each item rounded up to whole shares so that no CTA has parts of two.  Where
// the longest item is little longer than an equal share (`slack`: what cutting
// and joining cost), items are dealt out whole: sequences in the batch's order,
// the late tiles of each, which are its longest, first.
#pragma once

#include "common.cuh"
#include "rope_append.cuh"

namespace bitnet {

constexpr int kAttnThreads = 128;
constexpr int kAttnTile = 64;          // keys per block of the mma.sync kernel
constexpr int kAttnPlanHead = 3;       // words of the plan before the sequences'
constexpr int kAttnTarget = 592;       // most shares of a call (mma.sync kernel)

struct AttnParams {
  PagedBatch pb;
  const void* Q;
  void* O;
  const __nv_bfloat16 *Kc, *Vc;
  int qh, kvh, G, D;
  float scale_log2;                    // softmax scale * log2(e)
  int rt_shift, unit_shift;            // log2 of the rows per tile and the keys per block
  int min_keys;                        // smallest share, whole blocks
  int target;                          // shares wanted, 0: whole items, dealt out in turn
  int slack;                           // keys that a whole item may exceed a share by, or -1
  long long* plan;                     // length of a share, alignment, length of the call;
                                       // then the lengths before each sequence
  float* part;                         // slots: m[RT], l[RT], o[RT][D]
};

// --------------------------------------------------------------- the plan
// Items of a sequence come late tiles first, all heads of a tile together: the
// items of turn j (tile tiles - 1 - j) are base + slope * (tiles - j) long.
struct SeqWork {
  int c0, n, len;                      // first row, new tokens, cached tokens
  int tiles, base, slope;
};

__device__ __forceinline__ int item_length(const SeqWork& w, int j) {
  return w.base + w.slope * (w.tiles - j);
}

// Length of the sequence's items before turn j.
__device__ __forceinline__ long long turn_start(const AttnParams& p, const SeqWork& w, int j) {
  const long long n = j;
  return p.kvh * (n * w.base + w.slope * (n * w.tiles - n * (n - 1) / 2));
}

// align > 0: items are rounded up to whole shares of that length; kWhole: every
// item counts one.
constexpr int kWhole = -1;
__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, int b, bool report, int align) {
  SeqWork w;
  w.c0 = __ldg(p.pb.cu_q + b);
  const int c1 = __ldg(p.pb.cu_q + b + 1);
  w.len = __ldg(p.pb.kv_len + b);
  const int cap = p.pb.stride * p.pb.page_size;      // at most 2^30
  if (w.c0 < 0 || c1 < w.c0 || c1 > p.pb.M) {
    if (report) record_device_error(DEV_ERR_INDEX);
    w.c0 = 0;
    w.n = 0;
  } else {
    w.n = c1 - w.c0;
  }
  if (w.len < 0 || w.len > cap) {
    if (report) record_device_error(DEV_ERR_INDEX);
    w.len = w.len < 0 ? 0 : cap;
  }
  w.tiles = (w.n * p.G + (1 << p.rt_shift) - 1) >> p.rt_shift;
  w.slope = 0;
  if (align == kWhole) {
    w.base = 1;
  } else if (align > 0) {
    w.base = max((w.len + align - 1) / align, 1) * align;
  } else if (w.tiles <= 1) {                         // whole blocks, as shares are
    w.base = (((w.len - 1) >> p.unit_shift) + 2) << p.unit_shift;
  } else {
    w.base = max(w.len - w.n, 0) + (1 << p.unit_shift);
    w.slope = (1 << p.rt_shift) / p.G;               // tokens of a tile
  }
  return w;
}

// Thread t of the CTA holds sequences [t per, (t + 1) per) of the batch.
struct PlanShared {
  long long share, total;              // length of a share, of the call
  int align;                           // items are whole shares of that length, 0, or kWhole
  long long cursor;                    // where this CTA's share goes on
  long long first[kAttnThreads + 1];   // lengths before each thread's sequences
  long long red[kAttnThreads / 32], sums[kAttnThreads / 32][4];
};

// All threads of the CTA, kAttnThreads at least (sequences of later threads
// would start past the batch: they hold none).
__device__ __forceinline__ void make_plan(const AttnParams& p, PlanShared& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.pb.batch;
  const int per = (B + kAttnThreads - 1) / kAttnThreads;
  const int b0 = tid * per, b1 = min(B, b0 + per);
  const bool first = blockIdx.x == 0;
  bool cut = p.target > 0;
  if (cut && p.slack >= 0) {
    // length and items of the call, the longest and the shortest item (negated)
    long long v[4] = {0, 0, 0, -(1ll << 40)};
    for (int b = b0; b < b1; ++b) {
      const SeqWork w = seq_work(p, b, false, 0);
      v[0] += turn_start(p, w, w.tiles);
      v[1] += (long long)w.tiles * p.kvh;
      if (w.tiles > 0) {
        v[2] = max(v[2], (long long)item_length(w, 0));
        v[3] = max(v[3], -(long long)item_length(w, w.tiles - 1));
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      for (int o = 16; o > 0; o /= 2) {
        const long long x = __shfl_xor_sync(0xffffffffu, v[k], o);
        v[k] = k >= 2 ? max(v[k], x) : v[k] + x;
      }
      if (lane == 0 && warp < kAttnThreads / 32) s.sums[warp][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = s.sums[0][k];
      for (int i = 1; i < kAttnThreads / 32; ++i)
        v[k] = k >= 2 ? max(v[k], s.sums[i][k]) : v[k] + s.sums[i][k];
    }
    // Dealt out whole, as many items as CTAs take the longest one's time; up to
    // twice as many, CTA i takes items i and 2 CTAs - 1 - i, the worst of them
    // the first that has two; more, half an item over the average.  (An estimate:
    // lengths are taken to fall evenly over the call, and a long sequence behind
    // short ones takes longer: ten prompts of 500 tokens and one of 3000 121 us
    // with the long one first, 133 with it last.)
    const long long items = v[1], ctas = p.target, shortest = -v[3];
    const long long equal = (v[0] + ctas - 1) / ctas;
    long long whole = max(v[2], equal);
    if (items > 2 * ctas)
      whole = max(whole, equal + v[0] / items / 2);
    else if (items > ctas)
      whole = max(whole, v[2] - (v[2] - shortest) * (2 * ctas - items) / items + shortest);
    cut = whole > equal + p.slack;
  }
  // smallest shares first; if those are too many, equal ones
  int align = cut ? p.min_keys : kWhole;
  long long share = cut ? align : 1, mine, sum, total;
  for (;;) {
    mine = 0;
    for (int b = b0; b < b1; ++b) {
      const SeqWork w = seq_work(p, b, first, align);
      mine += turn_start(p, w, w.tiles);
    }
    sum = mine;                        // inclusive scan
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    if (lane == 31 && warp < kAttnThreads / 32) s.red[warp] = sum;
    __syncthreads();
    for (int i = 0; i < warp && i < kAttnThreads / 32; ++i) sum += s.red[i];
    total = 0;
    for (int i = 0; i < kAttnThreads / 32; ++i) total += s.red[i];
    if (align <= 0 || total <= share * p.target) break;
    align = 0;
    __syncthreads();
  }
  if (align == 0 && p.slack >= 0)
    share = max((total + p.target - 1) / p.target, 1ll);
  else if (align == 0)                 // decode: whole blocks, as its items are
    share = ((((total + p.target - 1) / p.target - 1) >> p.unit_shift) + 1) << p.unit_shift;
  if (tid < kAttnThreads) s.first[tid] = sum - mine;
  if (tid == 0) {
    s.first[kAttnThreads] = total;
    s.total = total;
    s.share = share;
    s.align = align;
    s.cursor = share * blockIdx.x;
  }
  if (first && p.target > 0) {         // for the join kernel
    if (tid == 0) {
      p.plan[0] = share;
      p.plan[1] = align;
      p.plan[2] = total;
    }
    long long at = sum - mine;
    for (int b = b0; b < b1; ++b) {
      const SeqWork w = seq_work(p, b, false, align);
      p.plan[kAttnPlanHead + b] = at;
      at += turn_start(p, w, w.tiles);
    }
  }
  __syncthreads();
}

// One CTA's part of one item: rows of a tile, one key/value head, blocks of keys.
struct AttnPiece {
  int b, c0, head;
  int slot;                            // where the sums go, or -1: the item is whole
  int row0, nrows;                     // rows of the sequence
  int past;                            // tokens before the new ones (may be negative)
  int kv_end;                          // keys that the last row sees
  int blk0, blk1;
};

// The part x0 .. x1 of an item of turn j.
__device__ __forceinline__ AttnPiece piece_of(const AttnParams& p, int b, const SeqWork& w, int j,
                                              int head, int x0, int x1, int slot) {
  AttnPiece q;
  q.b = b;
  q.c0 = w.c0;
  q.head = head;
  q.slot = slot;
  q.row0 = (w.tiles - 1 - j) << p.rt_shift;
  q.nrows = min(1 << p.rt_shift, w.n * p.G - q.row0);
  q.past = w.len - w.n;
  q.kv_end = max(0, q.past + (q.row0 + q.nrows - 1) / p.G + 1);
  const int blocks = (q.kv_end + (1 << p.unit_shift) - 1) >> p.unit_shift;
  const int length = item_length(w, j);
  q.blk0 = x0 == 0 ? 0 : (int)((long long)blocks * x0 / length);
  q.blk1 = x1 == length ? blocks : (int)((long long)blocks * x1 / length);
  return q;
}

// Turn and head of the item at `rel` in a sequence, and where it starts there.
__device__ __forceinline__ long long item_at(const AttnParams& p, const SeqWork& w, long long rel,
                                             int& j, int& head) {
  int lo = 0, hi = w.tiles - 1;        // the last turn that starts at rel or before
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (turn_start(p, w, mid) <= rel)
      lo = mid;
    else
      hi = mid - 1;
  }
  j = lo;
  const long long start = turn_start(p, w, j);
  const int length = item_length(w, j);
  head = (int)((rel - start) / length);
  return start + (long long)head * length;
}

// Whole item c: calls take(piece) on the one thread whose sequences hold it
// (on none if the lengths changed under the call).
template <class F>
__device__ __forceinline__ void find_item(const AttnParams& p, const PlanShared& s, long long c,
                                          F&& take) {
  const int tid = threadIdx.x;
  if (tid >= kAttnThreads || c < s.first[tid] || c >= s.first[tid + 1]) return;
  const int per = (p.pb.batch + kAttnThreads - 1) / kAttnThreads;
  long long at = s.first[tid];
  for (int b = tid * per; b < p.pb.batch; ++b) {
    const SeqWork w = seq_work(p, b, false, s.align);
    const long long k = (long long)w.tiles * p.kvh;
    if (c < at + k) {
      const int local = (int)(c - at), j = local / p.kvh;
      take(piece_of(p, b, w, j, local - j * p.kvh, 0, item_length(w, j), -1));
      return;
    }
    at += k;
  }
}

// The next pieces of this CTA's share, `most` at most: take(k, piece) for each
// and put their number in `count` (shared), on one thread; the cursor moves
// on.  All threads call it, and a barrier follows.
template <class F>
__device__ __forceinline__ void next_pieces(const AttnParams& p, PlanShared& s, int most,
                                            int& count, F&& take) {
  const int tid = threadIdx.x;
  const long long begin = s.share * blockIdx.x;
  const long long end = min(begin + s.share, s.total);
  long long pos = s.cursor;
  __syncthreads();                     // every thread has it before one moves it on
  if (pos >= end) {
    if (tid == 0) count = 0;
    return;
  }
  if (tid >= kAttnThreads || pos < s.first[tid] || pos >= s.first[tid + 1]) return;
  const int per = (p.pb.batch + kAttnThreads - 1) / kAttnThreads;
  long long at = s.first[tid];
  int k = 0;
  for (int b = tid * per; b < p.pb.batch && k < most && pos < end; ++b) {
    const SeqWork w = seq_work(p, b, false, s.align);
    const long long all = turn_start(p, w, w.tiles);
    if (pos < at + all) {
      int j, head;
      long long item = at + item_at(p, w, pos - at, j, head);
      for (;;) {
        const int length = item_length(w, j);
        const int x0 = (int)(pos - item);
        const int x1 = (int)min((long long)length, end - item);
        const int slot = x0 == 0 && x1 == length ? -1 : 2 * (int)blockIdx.x + (x0 == 0 ? 1 : 0);
        take(k++, piece_of(p, b, w, j, head, x0, x1, slot));
        pos = item + x1;
        item += length;
        if (++head == p.kvh) {
          head = 0;
          ++j;
        }
        if (j == w.tiles || k == most || pos >= end) break;
      }
    }
    at += all;
  }
  count = k;
  s.cursor = k > 0 ? pos : end;
}

// ------------------------------------------------------------ instructions
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool take) {
  const int n = take ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, one row per four lanes, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------- mma.sync kernel
// Bound by HBM once sequences are long: 50 us for 32 sequences of 95144 cached
// tokens (244 MB, 4.9 TB/s with plan and join), 65 us for two of 129198; by
// latency when short: 11 us for one token over 715.
//
// Four warps: WR of them along the rows (16 each), 4 / WR along the keys of a
// block.  WR = 1 takes up to 16 rows, each warp its own quarter of every block
// with its own statistics, joined in shared memory at the end.  WR = 4 takes
// 64 rows of a chunk.  WR = 0 is the decode form: 8 rows, the four warps along
// the keys, and both products transposed (keys and head elements are the 16
// rows of the matrix instruction, the query rows its 8 columns), which halves
// the instructions and registers where most of 16 rows would be padding.
//
// fp32 queries (F32): q and the probabilities are held as three bf16 terms (24
// bits, exact), so their products with the bf16 cache are those of fp32, for
// three matrix products in place of one.  (Two terms of the probabilities left
// a relative error of 1.6e-6, three 2e-7.)
// bf16 queries round the probabilities to bf16 (at most 2^-8 of each, of either
// sign; l sums the unrounded ones): over a call that is about as much as the
// output's own rounding (relative error 2.0e-3 to 2.3e-3, with fp32
// probabilities 1.6e-3).
template <int DP, int WR, bool F32>
struct AttnConfig {
  static constexpr int RT = WR == 0 ? 8 : 16 * WR;
  static constexpr int WK = WR == 4 ? 1 : 4;
  static constexpr int KW = kAttnTile / WK;          // keys of a warp per block
  static constexpr int STAGES = DP == 64 ? 4 : DP == 128 ? 3 : 2;
  static constexpr int TERMS = F32 ? 3 : 1;
  static constexpr int ROW = DP * 2;                 // bytes of a staged row
  static constexpr int Q_BYTES = RT * ROW * TERMS;
  static constexpr int KV_BYTES = kAttnTile * ROW;
  static constexpr int PAGE_TILES = 128;             // blocks whose page offsets are staged
  static constexpr int OFF_KV = Q_BYTES;
  static constexpr int OFF_PAGES = OFF_KV + STAGES * 2 * KV_BYTES;
  static constexpr int SMEM = OFF_PAGES + PAGE_TILES * (kAttnTile / 16) * 8;
  static constexpr bool Q_REGS = WR > 0 && !F32 && DP <= 128;
  static_assert(WK * RT * DP * 4 <= STAGES * 2 * KV_BYTES || WR == 4, "join buffer");
};

// 16-byte chunk c of staged row r.
template <int ROW>
__device__ __forceinline__ uint32_t attn_at(uint32_t base, int r, int c) {
  return base + (uint32_t)(r * ROW + ((c ^ (r & 7)) << 4));
}

template <int DP, int WR, bool F32>
__global__ void __launch_bounds__(kAttnThreads) attn_rows_kernel(AttnParams p) {
  using C = AttnConfig<DP, WR, F32>;
  extern __shared__ __align__(1024) uint8_t attn_smem[];
  __shared__ PlanShared plan;
  __shared__ AttnPiece s_piece;
  __shared__ int s_count;
  __shared__ float s_m[4][16], s_l[4][16];
  const uint32_t sq = smem_u32(attn_smem), skv = sq + C::OFF_KV;
  long long* s_off = reinterpret_cast<long long*>(attn_smem + C::OFF_PAGES);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wr = WR == 4 ? warp : 0, wk = WR == 4 ? 0 : warp;
  const int D = p.D, chunks = D / 8;

  grid_dependency_wait();                        // in this order: see rope_append_kernel
  grid_launch_dependents();
  make_plan(p, plan);

  for (long long c = blockIdx.x;; c += gridDim.x) {
    if (tid == 0) s_count = 0;
    __syncthreads();
    if (plan.align != kWhole)
      next_pieces(p, plan, 1, s_count, [&](int, const AttnPiece& q) { s_piece = q; });
    else if (c < plan.total)
      find_item(p, plan, c, [&](const AttnPiece& q) {
        s_piece = q;
        s_count = 1;
      });
    __syncthreads();
    if (s_count == 0) {
      if (plan.align != kWhole || c + gridDim.x >= plan.total) break;
      __syncthreads();
      continue;
    }
    const int b = s_piece.b, c0 = s_piece.c0, head = s_piece.head, slot = s_piece.slot;
    const int row0 = s_piece.row0, nrows = s_piece.nrows, past = s_piece.past;
    const int kv_end = s_piece.kv_end, blk0 = s_piece.blk0, blk1 = s_piece.blk1;
    const int lim_first = past + row0 / p.G + 1;     // keys that the first row sees

    // ---- queries to shared memory (zeros past the rows and past D)
    for (int i = tid; i < C::RT * (DP / 8); i += kAttnThreads) {
      const int r = i / (DP / 8), ch = i % (DP / 8);
      const bool ok = r < nrows && ch < chunks;
      const int rr = row0 + (ok ? r : 0);
      const long long off =
          ((long long)(c0 + rr / p.G) * p.qh + (long long)head * p.G + rr % p.G) * D + 8 * ch;
      uint4 u[C::TERMS];
#pragma unroll
      for (int t = 0; t < C::TERMS; ++t) u[t] = make_uint4(0, 0, 0, 0);
      if (ok) {
        if constexpr (F32) {
          const float* src = reinterpret_cast<const float*>(p.Q) + off;
          float x[8];
          *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
          *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(src + 4);
#pragma unroll
          for (int t = 0; t < 3; ++t) {
            uint32_t wds[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              wds[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
              x[2 * k] -= __uint_as_float(wds[k] << 16);
              x[2 * k + 1] -= __uint_as_float(wds[k] & 0xffff0000u);
            }
            u[t] = make_uint4(wds[0], wds[1], wds[2], wds[3]);
          }
        } else {
          u[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.Q) + off);
        }
      }
#pragma unroll
      for (int t = 0; t < C::TERMS; ++t)
        *reinterpret_cast<uint4*>(attn_smem + (attn_at<C::ROW>(sq, r, ch) - sq) +
                                  t * C::RT * C::ROW) = u[t];
    }

    // ---- keys and values: a ring of blocks filled by cp.async
    auto load = [&](int i) {
      const int blk = blk0 + i;
      if (i % C::PAGE_TILES == 0) {                  // page offsets of the next blocks
        __syncthreads();
        const int need = 4 * min(C::PAGE_TILES, blk1 - blk);
        for (int k = tid; k < need; k += kAttnThreads) {
          const int key = blk * kAttnTile + 16 * k;  // capacities stay below 2^30
          long long off = -1;
          if (key < kv_end) {
            const int page = __ldg(p.pb.table + (long long)b * p.pb.stride + key / p.pb.page_size);
            if (page < 0 || page >= p.pb.num_pages)
              record_device_error(DEV_ERR_INDEX);
            else
              off = (((long long)page * p.kvh + head) * p.pb.page_size + key % p.pb.page_size) * D;
          }
          s_off[k] = off;
        }
        __syncthreads();
      }
      if (blk < blk1) {
        const uint32_t dst = skv + (uint32_t)((i % C::STAGES) * 2 * C::KV_BYTES);
        const int g0 = (i % C::PAGE_TILES) * 4;
#pragma unroll
        for (int k = 0; k < kAttnTile * (DP / 8) / kAttnThreads; ++k) {
          const int idx = tid + k * kAttnThreads;
          const int r = idx / (DP / 8), ch = idx % (DP / 8);
          const long long base = s_off[g0 + (r >> 4)];
          // keys past the end may be anything, NaN too: zeros take their place
          const bool ok = base >= 0 && blk * kAttnTile + r < kv_end && ch < chunks;
          const long long off = ok ? base + (long long)(r & 15) * D + 8 * ch : 0;
          cp_async_16(attn_at<C::ROW>(dst, r, ch), p.Kc + off, ok);
          cp_async_16(attn_at<C::ROW>(dst + C::KV_BYTES, r, ch), p.Vc + off, ok);
        }
      }
      cp_async_commit();
    };

    const int count = blk1 - blk0;
#pragma unroll 1
    for (int i = 0; i < C::STAGES - 1; ++i) load(i);

    constexpr int OT = WR == 0 ? DP / 16 : DP / 8;   // accumulator tiles
    float o[OT][4];
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int lim[2];                                      // keys that this thread's rows see
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = WR == 0 ? 2 * (lane & 3) + k : 16 * wr + (lane >> 2) + 8 * k;
      lim[k] = r < nrows ? past + (row0 + r) / p.G + 1 : 0;
    }
    uint32_t qf[C::Q_REGS ? DP / 16 : 1][4];
    uint32_t qt[WR == 0 ? C::TERMS : 1][WR == 0 ? DP / 32 : 1][4];   // transposed: two steps each

#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      cp_async_wait<C::STAGES - 2>();
      __syncthreads();
      if constexpr (C::Q_REGS) {
        if (i == 0) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            ldmatrix_x4(attn_at<C::ROW>(sq, 16 * wr + (lane & 15), 2 * k + (lane >> 4)), qf[k]);
        }
      }
      if constexpr (WR == 0) {
        if (i == 0) {
#pragma unroll
          for (int t = 0; t < C::TERMS; ++t)
#pragma unroll
            for (int k = 0; k < DP / 32; ++k)
              ldmatrix_x4(attn_at<C::ROW>(sq + t * C::RT * C::ROW, lane & 7, 4 * k + (lane >> 3)),
                          qt[t][k]);
        }
      }
      load(i + C::STAGES - 1);
      const uint32_t sk = skv + (uint32_t)((i % C::STAGES) * 2 * C::KV_BYTES);
      const uint32_t sv = sk + C::KV_BYTES;
      if constexpr (WR == 0) {
        // scores: rows are this warp's 16 keys, columns the query rows; two
        // chains of products, so that one's latency hides the other's
        float z0[4] = {0, 0, 0, 0}, z1[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          uint32_t a[4];
          ldmatrix_x4(attn_at<C::ROW>(sk, 16 * wk + (lane & 15), 2 * k + (lane >> 4)), a);
#pragma unroll
          for (int t = C::TERMS - 1; t >= 0; --t)    // smallest terms first
            mma_bf16((k & 1) ? z1 : z0, a, qt[t][k / 2][2 * (k & 1)],
                     qt[t][k / 2][2 * (k & 1) + 1]);
        }
        const int key = (blk0 + i) * kAttnTile + 16 * wk + (lane >> 2);
        const bool masked = (blk0 + i + 1) * kAttnTile > lim_first || nrows < C::RT;
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z0[k] = (z0[k] + z1[k]) * p.scale_log2;
          if (masked && key + 8 * (k >> 1) >= lim[k & 1]) z0[k] = -INFINITY;
          mx[k & 1] = fmaxf(mx[k & 1], z0[k]);
        }
#pragma unroll
        for (int x = 4; x < 32; x *= 2)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], x));
        float alpha[2], base[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          base[k] = mx[k] == -INFINITY ? 0.0f : mx[k];   // nothing seen yet: all terms are 0
          alpha[k] = ex2(m[k] - base[k]);
          m[k] = mx[k];
          l[k] *= alpha[k];
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
          for (int n = 0; n < OT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[n][k] *= alpha[k & 1];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z0[k] = ex2(z0[k] - base[k & 1]);
          l[k & 1] += z0[k];
        }
        uint32_t pb[C::TERMS][2];                    // probabilities, keys along the pairs
#pragma unroll
        for (int t = 0; t < C::TERMS; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w2 = pack_bf16x2(z0[2 * k], z0[2 * k + 1]);
            if constexpr (F32) {
              z0[2 * k] -= __uint_as_float(w2 << 16);
              z0[2 * k + 1] -= __uint_as_float(w2 & 0xffff0000u);
            }
            pb[t][k] = movmatrix_trans(w2);
          }
#pragma unroll
        for (int d = 0; d < OT; ++d) {
          uint32_t a[4];
          ldmatrix_x4_trans(attn_at<C::ROW>(sv, 16 * wk + (lane & 7) + ((lane >> 4) << 3),
                                            2 * d + ((lane >> 3) & 1)), a[0], a[1], a[2], a[3]);
          if constexpr (F32) {                       // a block's sum is added rounded, see below
            float t0[4] = {0, 0, 0, 0};
#pragma unroll
            for (int t = C::TERMS - 1; t >= 0; --t) mma_bf16(t0, a, pb[t][0], pb[t][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[d][k] += t0[k];
          } else {
            mma_bf16(o[d], a, pb[0][0], pb[0][1]);
          }
        }
      } else {
        float z[C::KW / 8][4];
#pragma unroll
        for (int n = 0; n < C::KW / 8; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[n][k] = 0.0f;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          uint32_t a[C::TERMS][4];
          if constexpr (C::Q_REGS) {
#pragma unroll
            for (int x = 0; x < 4; ++x) a[0][x] = qf[k][x];
          } else {
#pragma unroll
            for (int t = 0; t < C::TERMS; ++t)
              ldmatrix_x4(attn_at<C::ROW>(sq + t * C::RT * C::ROW, 16 * wr + (lane & 15),
                                          2 * k + (lane >> 4)), a[t]);
          }
#pragma unroll
          for (int n = 0; n < C::KW / 16; ++n) {
            uint32_t kb[4];
            ldmatrix_x4(attn_at<C::ROW>(sk, C::KW * wk + 16 * n + (lane & 7) + ((lane >> 4) << 3),
                                        2 * k + ((lane >> 3) & 1)), kb);
#pragma unroll
            for (int t = C::TERMS - 1; t >= 0; --t) {  // smallest terms first
              mma_bf16(z[2 * n], a[t], kb[0], kb[1]);
              mma_bf16(z[2 * n + 1], a[t], kb[2], kb[3]);
            }
          }
        }
        const int key0 = (blk0 + i) * kAttnTile + C::KW * wk + 2 * (lane & 3);
        const bool masked = (blk0 + i + 1) * kAttnTile > lim_first || nrows < C::RT;
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < C::KW / 8; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float v = z[n][k] * p.scale_log2;
            if (masked && key0 + 8 * n + (k & 1) >= lim[k >> 1]) v = -INFINITY;
            z[n][k] = v;
            mx[k >> 1] = fmaxf(mx[k >> 1], v);
          }
        float alpha[2], base[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
          mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
          base[k] = mx[k] == -INFINITY ? 0.0f : mx[k];  // nothing seen yet: all terms are 0
          alpha[k] = ex2(m[k] - base[k]);
          m[k] = mx[k];
          l[k] *= alpha[k];
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            o[n][0] *= alpha[0];
            o[n][1] *= alpha[0];
            o[n][2] *= alpha[1];
            o[n][3] *= alpha[1];
          }
        }
        uint32_t pf[C::KW / 16][C::TERMS][4];          // the probabilities' terms
#pragma unroll
        for (int n = 0; n < C::KW / 16; ++n) {
          float e[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            e[k] = ex2(z[2 * n + (k >> 2)][k & 3] - base[(k >> 1) & 1]);
            l[(k >> 1) & 1] += e[k];
          }
#pragma unroll
          for (int t = 0; t < C::TERMS; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              pf[n][t][k] = pack_bf16x2(e[2 * k], e[2 * k + 1]);
              if constexpr (F32) {
                e[2 * k] -= __uint_as_float(pf[n][t][k] << 16);
                e[2 * k + 1] -= __uint_as_float(pf[n][t][k] & 0xffff0000u);
              }
            }
        }
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          // fp32: a block's sum starts at zero and is added rounded, since a
          // matrix instruction truncates its running sum (over thousands of
          // keys that came to 1.6e-6)
          float t0[4], t1[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            t0[k] = F32 ? 0.0f : o[2 * d][k];
            t1[k] = F32 ? 0.0f : o[2 * d + 1][k];
          }
#pragma unroll
          for (int n = 0; n < C::KW / 16; ++n) {
            uint32_t v0, v1, v2, v3;
            ldmatrix_x4_trans(attn_at<C::ROW>(sv, C::KW * wk + 16 * n + (lane & 15),
                                              2 * d + (lane >> 4)), v0, v1, v2, v3);
#pragma unroll
            for (int t = C::TERMS - 1; t >= 0; --t) {
              mma_bf16(t0, pf[n][t], v0, v1);
              mma_bf16(t1, pf[n][t], v2, v3);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            o[2 * d][k] = F32 ? o[2 * d][k] + t0[k] : t0[k];
            o[2 * d + 1][k] = F32 ? o[2 * d + 1][k] + t1[k] : t1[k];
          }
        }
      }
    }
    cp_async_wait<0>();
#pragma unroll
    for (int x = WR == 0 ? 4 : 1; x < (WR == 0 ? 32 : 4); x *= 2)
#pragma unroll
      for (int k = 0; k < 2; ++k) l[k] += __shfl_xor_sync(0xffffffffu, l[k], x);

    float* part = slot >= 0 ? p.part + (long long)slot * C::RT * (D + 2) : nullptr;
    auto store2 = [&](int r, int d, float x, float y) {
      if (slot >= 0) {
        *reinterpret_cast<float2*>(part + 2 * C::RT + r * D + d) = make_float2(x, y);
        return;
      }
      const int rr = row0 + r;
      const long long off =
          ((long long)(c0 + rr / p.G) * p.qh + (long long)head * p.G + rr % p.G) * D + d;
      if constexpr (F32)
        *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.O) + off) = make_float2(x, y);
      else
        *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.O) + off) =
            pack_bf16x2(x, y);
    };
    if constexpr (WR <= 1) {
      // the four warps' sums, each relative to the rows' common maximum
      __syncthreads();                               // the ring is free
      if (WR == 0 ? lane < 4 : (lane & 3) == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = WR == 0 ? 2 * lane + k : (lane >> 2) + 8 * k;
          s_m[warp][r] = m[k];
          s_l[warp][r] = l[k];
        }
      }
      __syncthreads();
      float* so = reinterpret_cast<float*>(attn_smem + C::OFF_KV);   // [4][RT][DP]
      float f[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = WR == 0 ? 2 * (lane & 3) + k : (lane >> 2) + 8 * k;
        const float mm = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
        f[k] = mm == -INFINITY ? 0.0f : ex2(m[k] - mm);
      }
#pragma unroll
      for (int n = 0; n < OT; ++n) {
        if constexpr (WR == 0) {
          float* x = so + (warp * C::RT + 2 * (lane & 3)) * DP + 16 * n + (lane >> 2);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[(k & 1) * DP + 8 * (k >> 1)] = o[n][k] * f[k & 1];
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float2*>(so + (warp * C::RT + (lane >> 2) + 8 * k) * DP + 8 * n +
                                       2 * (lane & 3)) =
                make_float2(o[n][2 * k] * f[k], o[n][2 * k + 1] * f[k]);
        }
      }
      __syncthreads();
      for (int i = tid; i < C::RT * (D / 2); i += kAttnThreads) {
        const int r = i / (D / 2), d = 2 * (i % (D / 2));
        if (r >= nrows) break;
        const float mm = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
        float sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sum += mm == -INFINITY ? 0.0f : s_l[q][r] * ex2(s_m[q][r] - mm);
          const float2 v = *reinterpret_cast<const float2*>(so + (q * C::RT + r) * DP + d);
          x += v.x;
          y += v.y;
        }
        if (slot >= 0) {
          if (d == 0) {
            part[r] = mm;
            part[C::RT + r] = sum;
          }
          store2(r, d, x, y);
        } else {
          const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
          store2(r, d, x * inv, y * inv);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 16 * wr + (lane >> 2) + 8 * k;
        if (r < nrows) {
          float inv = l[k] > 0.0f ? 1.0f / l[k] : 0.0f;
          if (slot >= 0) {
            inv = 1.0f;
            if ((lane & 3) == 0) {
              part[r] = m[k];
              part[C::RT + r] = l[k];
            }
          }
#pragma unroll
          for (int n = 0; n < DP / 8; ++n)
            if (8 * n < D)
              store2(r, 8 * n + 2 * (lane & 3), o[n][2 * k] * inv, o[n][2 * k + 1] * inv);
        }
      }
    }
    __syncthreads();                                 // plan, ring and statistics are free
  }
}

// --------------------------------------------------------------- the join
// CTA (c, y) joins the item that starts in share c and goes on past its end, if
// there is one.  Its rows are dealt out to the CTAs of c: WIDE, to their warps,
// as many at a time as fit a warp's lanes; else a row to a CTA, whose warps
// take the row's parts in turn.  The first part is in slot 2 c + 1, those of
// the shares after it in slots 2 (c + 1), 2 (c + 2), ...  Lanes hold 8 values
// each.
template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kAttnThreads) attn_join_kernel(AttnParams p) {
  __shared__ float s_o[4][kRopeMaxDim];
  __shared__ float s_ml[4][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_wait();                        // in this order: see rope_append_kernel
  grid_launch_dependents();
  const long long share = p.plan[0], total = p.plan[2];
  const int align = (int)p.plan[1];
  const int c = blockIdx.x;
  const long long end = share * (c + 1);
  if (align == kWhole || end >= total) return;
  // the sequence that holds place end - 1: the last one that starts before it
  int b = -1;
  for (int base = 0; base < p.pb.batch; base += 128) {
    int in = 0;
    bool starts[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = base + 32 * k + lane;
      starts[k] = i < p.pb.batch && p.plan[kAttnPlanHead + i] < end;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) in += __popc(__ballot_sync(0xffffffffu, starts[k]));
    b += in;
    if (in < 128) break;
  }
  const SeqWork w = seq_work(p, b, false, align);
  const long long at = p.plan[kAttnPlanHead + b];
  if (w.tiles == 0) return;                          // the lengths changed under the call
  int j, head;
  const long long item = at + item_at(p, w, end - 1 - at, j, head);
  const int length = item_length(w, j);
  if (item + length <= end || item < end - share) return;    // does not go on, or began before
  const int splits = (int)((item + length - 1) / share) - c + 1;
  const AttnPiece q = piece_of(p, b, w, j, head, 0, length, -1);

  const int RT = 1 << p.rt_shift, per = p.D / 8;
  const long long size = (long long)RT * (p.D + 2);
  const float* part0 = p.part + (2ll * c + 1) * size;
  const float* part1 = p.part + (2ll * c + 2) * size;        // further parts: 2 size apart
  const int sub = WIDE ? lane / per : 0, at_once = WIDE ? 32 / per : 1;   // rows of a warp
  const int ln = WIDE ? lane - sub * per : lane;     // place in the row
  const int step = WIDE ? gridDim.y * 4 * at_once : gridDim.y;
  for (int r0 = WIDE ? (blockIdx.y * 4 + warp) * at_once : blockIdx.y; r0 < q.nrows; r0 += step) {
    const int rt = min(r0 + sub, q.nrows - 1);
    const bool mine = WIDE ? sub < at_once && r0 + sub < q.nrows : lane < per;
    // one pass with a running maximum: a part's statistics and sums are loaded
    // together, several parts in flight
    float m = -INFINITY, l = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int s = WIDE ? 0 : warp; s < splits; s += WIDE ? 1 : 4) {
      const float* f = s == 0 ? part0 : part1 + 2 * (s - 1) * size;
      const float ms = f[rt], ls = f[RT + rt];
      float4 x = make_float4(0, 0, 0, 0), y = x;
      if (mine) {
        const float4* v = reinterpret_cast<const float4*>(f + 2 * RT + rt * p.D + 8 * ln);
        x = v[0];
        y = v[1];
      }
      const float mm = fmaxf(m, ms), base = mm == -INFINITY ? 0.0f : mm;
      const float e = ex2(m - base), g = ex2(ms - base);
      m = mm;
      l = l * e + ls * g;
      o[0] = o[0] * e + x.x * g; o[1] = o[1] * e + x.y * g;
      o[2] = o[2] * e + x.z * g; o[3] = o[3] * e + x.w * g;
      o[4] = o[4] * e + y.x * g; o[5] = o[5] * e + y.y * g;
      o[6] = o[6] * e + y.z * g; o[7] = o[7] * e + y.w * g;
    }
    const int rr = q.row0 + rt;
    const long long off =
        ((long long)(q.c0 + rr / p.G) * p.qh + (long long)q.head * p.G + rr % p.G) * p.D;
    if constexpr (WIDE) {
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] *= inv;
      if (mine) {
        if constexpr (F32)
          store_f32<8>(reinterpret_cast<float*>(p.O) + off + 8 * ln, o);
        else
          store_bf16<8>(reinterpret_cast<__nv_bfloat16*>(p.O) + off + 8 * ln, o);
      }
    } else {
      if (lane == 0) {
        s_ml[warp][0] = m;
        s_ml[warp][1] = l;
      }
      if (lane < per) {
#pragma unroll
        for (int k = 0; k < 8; ++k) s_o[warp][8 * lane + k] = o[k];
      }
      __syncthreads();
      float mm = -INFINITY, sum = 0.0f, f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) mm = fmaxf(mm, s_ml[k][0]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[k] = mm == -INFINITY ? 0.0f : ex2(s_ml[k][0] - mm);
        sum += f[k] * s_ml[k][1];
      }
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
      for (int d = tid; d < p.D; d += kAttnThreads) {
        const float x = inv * (f[0] * s_o[0][d] + f[1] * s_o[1][d] + f[2] * s_o[2][d] +
                               f[3] * s_o[3][d]);
        if (F32)
          reinterpret_cast<float*>(p.O)[off + d] = x;
        else
          reinterpret_cast<__nv_bfloat16*>(p.O)[off + d] = __float2bfloat16_rn(x);
      }
      __syncthreads();
    }
  }
}

}  // namespace bitnet
