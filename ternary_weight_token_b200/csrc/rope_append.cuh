// rope_append.cuh -- rotary position embedding of the new tokens' queries and
// keys, and the append of their keys and values to a paged cache.
//
// nnterp encyclopedia "bitnet", "Config" and "Printout": 20 query and 5
// key/value heads of 128, rotary embedding with theta 500000.
//
// For token row r of sequence b at position p, pair i of a head
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a),  a = p * inv_freq[i],
// optionally after an RMSNorm of the head (x * g / sqrt(mean(x^2) + eps)).
// The angle is formed in fp64 (p * inv_freq is exact there: 31 + 24 bits, two
// of them rounded), reduced to a fraction of a turn, and only the reduced
// angle is rounded to fp32; norms, rotation and products are fp32, and each
// output is rounded once.
//
// Bound by memory: a token of the 2B model reads 7.5 KB and writes 7.5 KB.  A
// group of lanes owns one head and moves it in 16-byte loads and stores (eight
// bf16 or four fp32 pairs per lane).  A warp serves one token, or a part of
// its heads where tokens are few: it looks the token up and forms its cosines
// and sines by itself, so warps never wait for one another, and a lane keeps
// the few angles of its place in the head in registers for all heads.  The
// first head is loaded before the token is looked up.  Measured: 14.8 us for
// 3909 tokens (60 MB, 4.1 TB/s), 2.8 us for one.
#pragma once

#include "common.cuh"

namespace bitnet {

// Device error word: a page index, row or length in device memory is out of
// range; the kernel skipped the access.
constexpr unsigned DEV_ERR_INDEX = 2u;

// Where the new tokens of a batch of sequences stand, and the pages that hold
// their past: shared by the append and by the attention that reads the cache.
struct PagedBatch {
  const int32_t* cu_q;     // [batch + 1] first token row of each sequence
  const int32_t* kv_len;   // [batch] tokens in the cache once the new ones are appended
  const int32_t* table;    // [batch][stride] pages of each sequence
  int batch, stride;
  int num_pages, page_size;
  int M;                   // token rows the caller's tensors have
};

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 256;
// Heads a lane group has in flight: with two or four the registers cost more
// warps than the loads gain (14.7 -> 17.4 / 19 us for 3909 tokens).
constexpr int kRopeDepth = 1;

struct RopeParams {
  PagedBatch pb;
  const void *Q, *K, *V;
  long long ldq, ldk, ldv;          // elements between token rows
  void* Qo;
  __nv_bfloat16 *Kc, *Vc;
  const float* inv_freq;            // [rot / 2]
  const float *qg, *kg;             // [D] or null
  float eps;
  int qh, kvh, D, rot;
  int interleaved;
  int warps_per_token;              // a power of two up to the CTA's warps
};

// Sequence of token row r: the first one that ends behind it, or the batch
// (every lane of the warp gets it).
__device__ __forceinline__ int sequence_of(const PagedBatch& pb, int r, int lane) {
  for (int base = 0; base < pb.batch; base += 128) {
    bool behind[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = base + 32 * k + lane;
      behind[k] = i >= pb.batch || __ldg(pb.cu_q + i + 1) > r;
    }
    int first = 128;
#pragma unroll
    for (int k = 3; k >= 0; --k) {
      const uint32_t any = __ballot_sync(0xffffffffu, behind[k]);
      if (any != 0) first = 32 * k + __ffs((int)any) - 1;
    }
    if (first < 128) return min(base + first, pb.batch);
  }
  return pb.batch;
}

// The tables' entries of sequence s; false where they are out of range (its
// rows do not rise within the M there are, or its length has no room in the
// block table).
__device__ __forceinline__ bool sequence_entries(const PagedBatch& pb, int s, int& c0, int& c1,
                                                 int& len) {
  c0 = __ldg(pb.cu_q + s);
  c1 = __ldg(pb.cu_q + s + 1);
  len = __ldg(pb.kv_len + s);
  return c0 >= 0 && c1 >= c0 && c1 <= pb.M && len >= 0 &&
         len <= pb.stride * pb.page_size;            // at most 2^30
}

template <bool BF16>
struct RopeVec;                     // 16 bytes of one head
template <>
struct RopeVec<true> {
  static constexpr int N = 8;
  __device__ static void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct RopeVec<false> {
  static constexpr int N = 4;
  __device__ static void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// N consecutive elements from fp32 values.
template <int N>
__device__ __forceinline__ void store_f32(float* p, const float* x) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
template <int N>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* p, const float* x) {
  if constexpr (N == 8) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  }
}

// First element of the two runs of N that lane slot j of a head holds: runs of
// pairs (first[i], second[i]) when the pairs are split in halves, one run of
// 2 N elements when they are interleaved.  Past the rotated part the rest of
// the head is paired the same way, and is not turned; rot / 2 is a multiple of
// 8, so a slot lies on one side.
__device__ __forceinline__ void rope_runs(int j, int n, const RopeParams& p, int& e0, int& e1) {
  if (p.interleaved) {
    e0 = 2 * n * j;
    e1 = e0 + n;
    return;
  }
  const int half = p.rot / 2;
  int i = n * j;
  if (i < half) {
    e0 = i;
    e1 = i + half;
  } else {
    e0 = p.rot + (i - half);
    e1 = e0 + (p.D - p.rot) / 2;
  }
}

template <bool BF16, bool NORM>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(RopeParams p) {
  extern __shared__ float2 s_cs[];               // [warps][D / 2] cosine, sine
  constexpr int N = RopeVec<BF16>::N, ESZ = BF16 ? 2 : 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = p.D, half_d = D / 2;
  const int lanes = half_d / N;                  // lane slots of a head
  int width = 1;                                 // lanes of a group: a power of two
  while (width < lanes) width *= 2;
  const int j = lane & (width - 1);
  const bool active = j < lanes;
  const bool turned = N * j < p.rot / 2;         // the slot's pairs are rotated
  const int slots = 32 / width;                  // heads of a warp at a time
  const int heads = p.qh + 2 * p.kvh;
  const int gw = blockIdx.x * (kRopeThreads / 32) + warp;
  const int r = gw / p.warps_per_token, part = gw - r * p.warps_per_token;
  const int h0 = part * slots + lane / width, step = slots * p.warps_per_token;
  int e0, e1;
  rope_runs(active ? j : 0, N, p, e0, e1);

  // the next launch may start only once the work before this one has completed:
  // one that reads inputs early then never looks past the launch before it
  grid_dependency_wait();
  grid_launch_dependents();

  const char* qrow = reinterpret_cast<const char*>(p.Q) + (long long)r * p.ldq * ESZ;
  const char* krow = reinterpret_cast<const char*>(p.K) + (long long)r * p.ldk * ESZ;
  const char* vrow = reinterpret_cast<const char*>(p.V) + (long long)r * p.ldv * ESZ;
  auto load = [&](int h, uint4& x, uint4& y) {
    x = y = make_uint4(0, 0, 0, 0);
    if (h >= heads || !active || r >= p.pb.M) return;
    const char* base = h < p.qh           ? qrow + h * D * ESZ
                       : h < p.qh + p.kvh ? krow + (h - p.qh) * D * ESZ
                                          : vrow + (h - p.qh - p.kvh) * D * ESZ;
    x = *reinterpret_cast<const uint4*>(base + e0 * ESZ);
    y = *reinterpret_cast<const uint4*>(base + e1 * ESZ);
  };
  uint4 a[kRopeDepth], b[kRopeDepth];
#pragma unroll
  for (int k = 0; k < kRopeDepth; ++k) load(h0 + k * step, a[k], b[k]);

  // ---- the tables: each sequence is looked at once, whether or not a row is
  // found to be its own (beside the loads above and the look-up below)
  for (long long s = (long long)blockIdx.x * kRopeThreads + threadIdx.x; s < p.pb.batch;
       s += (long long)gridDim.x * kRopeThreads) {
    int c0, c1, len;
    if (!sequence_entries(p.pb, (int)s, c0, c1, len)) record_device_error(DEV_ERR_INDEX);
  }
  if (r >= p.pb.M) return;

  // ---- the token's place
  int pos;
  long long dst = -1;                            // first element of its head 0 in the cache
  {
    const int s = sequence_of(p.pb, r, lane);
    if (s >= p.pb.batch) return;                 // behind the last sequence
    int c0, c1, len;
    // r < c0 or r >= c1 only in a table of rows that does not rise
    if (!sequence_entries(p.pb, s, c0, c1, len) || r < c0 || r >= c1) return;
    pos = len - (c1 - r);
    if (pos < 0) return;
    const int at = pos / p.pb.page_size;
    int page = -1;
    if (at < p.pb.stride) page = __ldg(p.pb.table + (long long)s * p.pb.stride + at);
    if (page < 0 || page >= p.pb.num_pages) {
      if (lane == 0) record_device_error(DEV_ERR_INDEX);
    } else {
      dst = ((long long)page * p.kvh * p.pb.page_size + (pos - at * p.pb.page_size)) * D;
    }
  }
  float2* cs_row = s_cs + warp * half_d;
  for (int f = lane; f < half_d; f += 32) {
    float2 cs = make_float2(1.0f, 0.0f);
    if (f < p.rot / 2) {
      // turns = p * inv_freq / (2 pi); the nearest whole turn is dropped in fp64
      double turns = (double)pos * (double)__ldg(p.inv_freq + f) * 0.15915494309189533577;
      turns -= rint(turns);
      sincospif((float)(2.0 * turns), &cs.y, &cs.x);
    }
    cs_row[f] = cs;
  }
  __syncwarp();
  float2 cs[N];
#pragma unroll
  for (int i = 0; i < N; ++i) cs[i] = cs_row[N * (active ? j : 0) + i];

  // every lane of a warp makes the same number of trips: the norm's sums go
  // through warp shuffles
  for (int h = h0, first = part * slots; first < heads; h += step, first += step) {
    const uint4 ua = a[0], ub = b[0];
#pragma unroll
    for (int k = 0; k + 1 < kRopeDepth; ++k) {
      a[k] = a[k + 1];
      b[k] = b[k + 1];
    }
    load(h + kRopeDepth * step, a[kRopeDepth - 1], b[kRopeDepth - 1]);
    const bool isq = h < p.qh, isv = h >= p.qh + p.kvh;
    const bool live = h < heads && active;
    float x[2 * N];
    RopeVec<BF16>::unpack(ua, x);
    RopeVec<BF16>::unpack(ub, x + N);
    float rr = 1.0f;
    if (NORM) {
      float sum = 0.0f;                          // idle lanes hold zeros
#pragma unroll
      for (int i = 0; i < 2 * N; ++i) sum = __fmaf_rn(x[i], x[i], sum);
      for (int o = width / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      rr = 1.0f / sqrtf(sum / (float)D + p.eps);
    }
    if (!isv) {
      if (NORM) {
        const float* g = isq ? p.qg : p.kg;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          x[i] = x[i] * rr * (g ? __ldg(g + e0 + i) : 1.0f);
          x[N + i] = x[N + i] * rr * (g ? __ldg(g + e1 + i) : 1.0f);
        }
      }
      if (!turned) {
        // passes as it is: 0 times an infinity is not 0
      } else if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float u = x[2 * i], v = x[2 * i + 1];
          x[2 * i] = __fmaf_rn(u, cs[i].x, -__fmul_rn(v, cs[i].y));
          x[2 * i + 1] = __fmaf_rn(v, cs[i].x, __fmul_rn(u, cs[i].y));
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float u = x[i], v = x[N + i];
          x[i] = __fmaf_rn(u, cs[i].x, -__fmul_rn(v, cs[i].y));
          x[N + i] = __fmaf_rn(v, cs[i].x, __fmul_rn(u, cs[i].y));
        }
      }
    }
    if (live) {
      if (isq) {
        const long long o = ((long long)r * p.qh + h) * D;
        if (BF16) {
          __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.Qo) + o;
          store_bf16<N>(out + e0, x);
          store_bf16<N>(out + e1, x + N);
        } else {
          float* out = reinterpret_cast<float*>(p.Qo) + o;
          store_f32<N>(out + e0, x);
          store_f32<N>(out + e1, x + N);
        }
      } else if (dst >= 0) {
        const int kh = isv ? h - p.qh - p.kvh : h - p.qh;
        __nv_bfloat16* out = (isv ? p.Vc : p.Kc) + dst + (long long)kh * p.pb.page_size * D;
        store_bf16<N>(out + e0, x);
        store_bf16<N>(out + e1, x + N);
      }
    }
  }
}

}  // namespace bitnet
