// kv4.cu — key/value cache held in 4 bits: rows written, read back, and the
// gated sparse decode over it.
//
// A group of 32 channels of one token and head is stored as fp16 (scale s,
// minimum m) and codes n in 0..15; a code stands for m + s n. Channel c has
// nibble c % 4 of the row's 16-bit word (c % 32) / 4 * (d / 32) + c / 32.
#include <atomic>
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gbs {
namespace {

constexpr int kBS = 64;
constexpr float kMaxValue = 60000.f;  // below fp16's largest, so that m + 15 s cannot overflow it

struct RowArgs {
  int B, Hkv, T, N;
  Kv4 c;
  Heads t[2];  // keys, values [B, Hkv, T, d]
  const int32_t *start, *count;
};

// Index of token t of sequence b, head h among the cache's rows, or -1.
__device__ __forceinline__ long long cache_row(const RowArgs& a, int b, int h, int t) {
  const int s = __ldg(a.start + b);
  const long long pos = (long long)s + t;
  if (pos < 0 || pos >= a.N) {
    set_error(a.c.err, GBS_ERR_INVALID_ARG);
    return -1;
  }
  if (!a.c.btab) return ((long long)b * a.Hkv + h) * a.c.cap + pos;
  const int page = __ldg(a.c.btab + (size_t)b * a.c.max_blocks + pos / kBS);
  if (page < 0 || page >= a.c.num_pages) {
    set_error(a.c.err, GBS_ERR_INVALID_ARG);
    return -1;
  }
  return ((long long)page * a.Hkv + h) * kBS + pos % kBS;
}

__device__ __forceinline__ int token_count(const RowArgs& a, int b) {
  if (!a.count) return a.T;
  const int n = __ldg(a.count + b);
  if (n < 0 || n > a.T) {
    set_error(a.c.err, GBS_ERR_INVALID_ARG);
    return n < 0 ? 0 : a.T;
  }
  return n;
}

__device__ __forceinline__ float low_half(uint32_t w) {
  return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
}
__device__ __forceinline__ float high_half(uint32_t w) {
  return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}

// Append and read give a row to d / 32 lanes, 16 code bytes to each: halfwords 8 p ..
// 8 p + 7 of lane p, which hold kSpan consecutive channels of every group, from channel
// 32 k + kSpan p of group k on (append). So a lane moves 16 bytes at a time on both sides,
// and a group's extremes take one or two shuffles for all rows of a warp at once. Append
// of 32768 tokens x 8 heads, d = 128, bf16 (176 MB, 27 us): 55 us, bound by issue (0.68 an
// SM quarter's clock); with scalar fp32 70 us, with all 32 quotients of a lane decided in 64
// bits where one has to be 149. Without that slow path it would take 8 us less.
template <int D>
struct RowLanes {
  static constexpr int NG = D / 32, kSpan = 32 / NG;
};

// kSpan channels from or to p.
template <int N>
__device__ __forceinline__ void load_span(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(p + i));
    v[i] = u.x; v[i + 1] = u.y; v[i + 2] = u.z; v[i + 3] = u.w;
  }
}
template <int N>
__device__ __forceinline__ void load_span(const __nv_bfloat16* p, float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + i));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i + j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
}
template <int N>
__device__ __forceinline__ void store_span(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int N>
__device__ __forceinline__ void store_span(__nv_bfloat16* p, const float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// min and max of three that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// fp16((hi - m) / 15) as through 64 bits: the fp32 product is within 2^-22 of the
// quotient, so it decides unless the fp16 on both sides of it differ.
__device__ __forceinline__ __half group_scale(float hi, float m) {
  const float q = (hi - m) * (1.f / 15.f);
  const __half a = __float2half_rn(q * (1.f - 0x1p-20f)), b = __float2half_rn(q * (1.f + 0x1p-20f));
  if (__half_as_ushort(a) == __half_as_ushort(b)) return a;
  return __float2half_rn((float)(((double)hi - (double)m) / 15.0));
}

// Parameter word of a group with extremes lo and hi.
__device__ __forceinline__ uint32_t group_params(float lo, float hi) {
  if (isnan(lo)) return 0x7fff7fffu;
  const __half m = __float2half_rn(fminf(fmaxf(lo, -kMaxValue), kMaxValue));
  const __half s = group_scale(fminf(fmaxf(hi, -kMaxValue), kMaxValue), __half2float(m));
  return (uint32_t)__half_as_ushort(s) | (uint32_t)__half_as_ushort(m) << 16;
}

constexpr float kUnsure = 0.5f - 0x1p-17f;
// The codes of four channels as 16 bits, from i15 = 1 / (15 s). In fp32 (x - m) / s is
// within 2^-18 of the quotient in 0..15, so it decides unless it is within 2^-17 of a
// half: *unsure tells that one is. Saturation to 0..1 limits the codes and makes a NaN 0.
__device__ __forceinline__ uint32_t codes_of(const float* x, float m, float i15, bool* unsure) {
  using namespace sm100;
  constexpr float kRound = 12582912.f;  // 1.5 2^23: adding it rounds to whole numbers, ties to even
  const f32x2 m2 = f2_make(m, m), fifteen = f2_make(15.f, 15.f), up = f2_make(kRound, kRound);
  f32x2 n[2];
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // channels i and i + 2, so that both halves take the same step below
    float d0, d1, e0, e1;
    f2_split(f2_sub(f2_make(x[i], x[i + 2]), m2), d0, d1);
    const f32x2 t = f2_make(__saturatef(d0 * i15), __saturatef(d1 * i15));
    n[i] = f2_sub(f2_fma(t, fifteen, up), up);
    f2_split(f2_sub(f2_mul(t, fifteen), n[i]), e0, e1);
    far = fmaxf(far, fmaxf(fabsf(e0), fabsf(e1)));
  }
  *unsure = far > kUnsure;
  float lo, hi;
  f2_split(f2_fma(n[1], f2_make(16.f, 16.f), n[0]), lo, hi);
  return (uint32_t)fmaf(hi, 256.f, lo);
}
// Row of a lane: sequence, head and token; token -1 behind the last.
struct RowPlace {
  int b, h, t;
};
template <int D>
__device__ __forceinline__ RowPlace row_place(const RowArgs& a) {
  constexpr unsigned NG = RowLanes<D>::NG;
  const unsigned row = blockIdx.x * (256u / NG) + threadIdx.x / NG;
  if (row >= (unsigned)a.B * a.Hkv * a.T) return {0, 0, -1};
  const unsigned bh = row / (unsigned)a.T;
  return {(int)(bh / (unsigned)a.Hkv), (int)(bh % (unsigned)a.Hkv), (int)(row - bh * (unsigned)a.T)};
}

template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const __grid_constant__ RowArgs a) {
  using R = RowLanes<D>;
  constexpr int NG = R::NG, kSpan = R::kSpan;
  const int p = threadIdx.x % NG;
  const RowPlace r = row_place<D>(a);
  const Heads& src = blockIdx.y ? a.t[1] : a.t[0];
  long long at = -1;
  if (r.t >= 0 && r.t < token_count(a, r.b)) at = cache_row(a, r.b, r.h, r.t);
  float x[NG][kSpan];
  if (at >= 0) {
    const T* row = reinterpret_cast<const T*>(src.ptr) + r.b * src.sb + r.h * src.sh + r.t * src.sn;
#pragma unroll
    for (int k = 0; k < NG; ++k) load_span<kSpan>(row + 32 * k + kSpan * p, x[k]);
  } else {
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
      for (int i = 0; i < kSpan; ++i) x[k][i] = 0.f;
  }
  float lo[NG], hi[NG];
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    lo[k] = hi[k] = x[k][0];
#pragma unroll
    for (int i = 1; i < kSpan; i += 2) {
      lo[k] = min_nan(lo[k], x[k][i], x[k][i + 1 < kSpan ? i + 1 : i]);
      hi[k] = max_nan(hi[k], x[k][i], x[k][i + 1 < kSpan ? i + 1 : i]);
    }
#pragma unroll
    for (int o = NG / 2; o > 0; o >>= 1) {
      const float l = __shfl_xor_sync(0xffffffffu, lo[k], o), h = __shfl_xor_sync(0xffffffffu, hi[k], o);
      lo[k] = min_nan(lo[k], l, l);
      hi[k] = max_nan(hi[k], h, h);
    }
  }
  // a lane makes the parameters of group p and gets the others' from its row's lanes
  float my_lo = lo[0], my_hi = hi[0];
#pragma unroll
  for (int k = 1; k < NG; ++k) {
    my_lo = k == p ? lo[k] : my_lo;
    my_hi = k == p ? hi[k] : my_hi;
  }
  const uint32_t mine = group_params(my_lo, my_hi);
  const float my_scale = low_half(mine), my_i15 = my_scale > 0.f ? __frcp_rn(my_scale * 15.f) : 0.f;
  uint32_t half[NG][kSpan / 4], params[NG], unsure = 0u;
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    params[k] = __shfl_sync(0xffffffffu, mine, k, NG);
    const float m = high_half(params[k]), i15 = __shfl_sync(0xffffffffu, my_i15, k, NG);
#pragma unroll
    for (int i = 0; i < kSpan / 4; ++i) {
      bool u;
      half[k][i] = codes_of(x[k] + 4 * i, m, i15, &u);
      unsure |= u ? 1u << (i * NG + k) : 0u;
    }
  }
  if (at < 0) return;
  // halfword j of the lane's eight: group j % NG, four channels j / NG
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = half[2 * j % NG][2 * j / NG] | half[(2 * j + 1) % NG][(2 * j + 1) / NG] << 16;
  // Halfwords with a quotient next to a half, which 64 bits decide: one value in 65,000,
  // but one in about 8,000 where bf16 values meet a border exactly. Channels are loaded
  // again, so that x stays in registers above.
  while (unsure) {
    const int j = __ffs(unsure) - 1, k = j % NG;
    unsure &= unsure - 1;
    uint32_t param = params[0], bits = 0u;
#pragma unroll
    for (int q = 1; q < NG; ++q) param = q == k ? params[q] : param;
    const float m = high_half(param), s = low_half(param), i15 = __frcp_rn(s * 15.f);
    const T* at4 = reinterpret_cast<const T*>(src.ptr) + r.b * src.sb + r.h * src.sh + r.t * src.sn + 32 * k + kSpan * p + j / NG * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = to_f32<T>(at4[i]), t = __saturatef((v - m) * i15) * 15.f;
      float n = rintf(t);
      if (fabsf(t - n) > kUnsure - 0x1p-19f) {  // on which side of the half that t is next to?
        const float below = floorf(t);
        const double over = ((double)v - (double)m) - ((double)below + 0.5) * (double)s;
        n = over > 0. || (over == 0. && ((int)below & 1)) ? below + 1.f : below;
      }
      bits |= (uint32_t)n << (4 * i);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q == j / 2) w[q] = j & 1 ? (w[q] & 0xffffu) | bits << 16 : (w[q] & 0xffff0000u) | bits;
  }
  reinterpret_cast<uint4*>((blockIdx.y ? a.c.vc : a.c.kc) + at * (D / 2))[p] = make_uint4(w[0], w[1], w[2], w[3]);
  (blockIdx.y ? a.c.vp : a.c.kp)[at * NG + p] = mine;
}

// A lane writes 16 bytes at a time, next to its neighbours' (whole sectors): unit p, p + NG,
// ... of a group's. Bound by memory: 32768 tokens x 8 heads, d = 128, as fp32 (310 MB) 53 us,
// 5.8 TB/s (68 us when a lane wrote its 32 bytes in two halves), as bf16 33 us.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ RowArgs a) {
  constexpr int NG = RowLanes<D>::NG, kChunks = 4 / (int)sizeof(T);  // of four channels, in a unit
  constexpr int kUnits = 8 / kChunks / NG, kWords = kChunks * NG / 2;  // of a lane; of a unit's codes
  const int p = threadIdx.x % NG;
  const RowPlace r = row_place<D>(a);
  if (r.t < 0) return;
  const Heads& dst = blockIdx.y ? a.t[1] : a.t[0];
  const long long at = r.t < token_count(a, r.b) ? cache_row(a, r.b, r.h, r.t) : -1;
  uint32_t w[kUnits][kWords] = {}, param[NG] = {};
  if (at >= 0) {
    const uint32_t* codes = reinterpret_cast<const uint32_t*>((blockIdx.y ? a.c.vc : a.c.kc) + at * (D / 2));
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const uint32_t* from = codes + (p + u * NG) * kWords;
      if constexpr (kWords == 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(from));
        w[u][0] = x.x; w[u][1] = x.y; w[u][2] = x.z; w[u][3] = x.w;
      } else if constexpr (kWords == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(from));
        w[u][0] = x.x; w[u][1] = x.y;
      } else {
        w[u][0] = __ldg(from);
      }
    }
#pragma unroll
    for (int k = 0; k < NG; ++k) param[k] = __ldg((blockIdx.y ? a.c.vp : a.c.kp) + at * NG + k);
  }
  T* row = reinterpret_cast<T*>(dst.ptr) + r.b * dst.sb + r.h * dst.sh + r.t * dst.sn;
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    const float s = low_half(param[k]), m = high_half(param[k]);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      float v[4 * kChunks];
#pragma unroll
      for (int i = 0; i < 4 * kChunks; ++i) {
        const int j = i / 4 * NG + k;  // the halfword of the unit
        // the nibble as 2^23 + n, an exact fp32
        const uint32_t n = (w[u][j / 2] >> (16 * (j & 1) + 4 * (i & 3)) & 15u) | 0x4b000000u;
        v[i] = fmaf(s, __uint_as_float(n) - 8388608.f, m);
      }
      store_span<4 * kChunks>(row + 32 * k + (p + u * NG) * 4 * kChunks, v);
    }
  }
}

// ------------------------------------------------------------------ decode

struct DecodeArgs {
  Problem p;
  Kv4 c;
  const float* S;  // scores
  Selection sel;   // lists of a selection made before; null where the kernel selects for itself
  const int32_t* seq_lens;
  const void* q;
  void* O;
  float* LSE;
  int grouped, splits;
  int inbox;  // with splits: where an Inbox lies in a CTA's dynamic shared memory
};

__device__ __forceinline__ int sequence_length(const DecodeArgs& a, int b) {
  if (!a.seq_lens) return a.p.N;
  const int L = __ldg(a.seq_lens + b);
  if (L < 0 || L > a.p.N) {
    set_error(a.c.err, GBS_ERR_INVALID_ARG);
    return L < 0 ? 0 : a.p.N;
  }
  return L;
}

// First cache row of block c of (b, kvh), or -1 for a page outside the pool.
__device__ __forceinline__ long long block_row(const DecodeArgs& a, int b, int kvh, int c) {
  if (!a.c.btab) return ((long long)b * a.p.Hkv + kvh) * a.c.cap + c * kBS;
  const int page = __ldg(a.c.btab + (size_t)b * a.c.max_blocks + c);
  if (page < 0 || page >= a.c.num_pages) {
    set_error(a.c.err, GBS_ERR_INVALID_ARG);
    return -1;
  }
  return ((long long)page * a.p.Hkv + kvh) * kBS;
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Selection of the decode (that of select.cu: the min(topk, r) largest of r scores, ties
// to the lower index, in threshold mode those whose gate reaches tau) by the 128 threads
// of a CTA. (The decode over unpacked caches keeps its lists from select.cu: its CTAs walk chunks
// of them, and rows of more than kSelectMax blocks need them here too. A change to what is kept
// is one to both.) The k-th largest key is found by bisection between the smallest and the
// largest, on scores first and on their ordered bits at the end, until a threshold has k
// keys on its upper side; no histogram, in which the few exponents of real scores would
// all meet. Rows of up to 2048 blocks first drop what cannot be among k <= 96 kept ones:
// at least k keys reach the k-th largest of the threads' own maxima, and those that reach
// it are few (some 60 of 2048 for k = 32), so that one warp finishes among them. Beyond either
// border every count is one of all threads, and rows of more than kSelectMax blocks are left to
// a kernel before, of a warp a row. Calls of 8 sequences with 32 heads, a selection for each /
// for four, in us: at 2047 earlier blocks, k = 32 25.5 / 16.6, 2048 25.7 / 16.8, 2049 32.8 / 22.5,
// 3071 35.5 / 25.8, 8192 50 / 37, 8193 601 / 570; at 2047, k = 96 57.8 / 28.9, 97 62.4 / 32.6,
// 128 77.3 / 39.7, 256 134 / 59.
struct SelectScratch {
  unsigned u[2][4], bound;
  float f[4];
  int32_t idx[GBS_MAX_TOPK];
  float score[GBS_MAX_TOPK];
};
constexpr int kSelectMax = 8192, kSelectRegs = 16;  // blocks of a row; keys a thread holds
constexpr int kSelectWork = 640;                   // least words of shared memory
constexpr int kMaxCluster = 16;  // splits of a row, which join their sums in one cluster

// A score as a key whose order is the scores'; 0 is left for "none" (only one NaN has it).
__device__ __forceinline__ uint32_t score_key(float score) { return max(ordered_key(score), 1u); }
__device__ __forceinline__ float key_score(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// Smallest threshold below the k-th largest key, by a warp whose lanes hold N keys each (0:
// none): keys above the result are kept, and the first *need_eq of those equal to it. At
// most `rounds` of bisection: a result of less is a bound that at least k keys reach.
template <int N>
__device__ __forceinline__ uint32_t warp_threshold(const uint32_t (&u)[N], int k, int rounds, int* need_eq) {
  uint32_t hi = 0u, lo = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    hi = max(hi, u[i]);
    if (u[i]) lo = min(lo, u[i]);
  }
  uint32_t T = __reduce_min_sync(0xffffffffu, lo), above = __reduce_max_sync(0xffffffffu, hi) + 1u;
  int n_above = 0;
  for (int it = 0; above - T > 1u && it < rounds; ++it) {
    uint32_t mid = T + (above - T) / 2;
    if (it < 14) {  // between the scores, where that is inside
      const uint32_t x = ordered_key(0.5f * key_score(T) + 0.5f * key_score(above - 1u));
      if (x > T && x < above) mid = x;
    }
    unsigned n = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) n += u[i] >= mid ? 1u : 0u;
    n = __reduce_add_sync(0xffffffffu, n);
    if ((int)n == k) {
      *need_eq = 0;
      return mid - 1u;
    }
    if ((int)n > k) T = mid;
    else above = mid, n_above = (int)n;
  }
  *need_eq = k - n_above;
  return T;
}

constexpr int kCandidates = 256;
static_assert(128 + 2 * kCandidates <= kSelectWork, "");

// The end of a selection, by a warp whose lane l holds keys l, l + 32, ... of n: of the k
// largest, idx(j) of the j-th key and its score go to sc where `write`; returns the
// logarithm of the sum of their exponentials over that of the largest score, top.
template <int N, typename Index>
__device__ __forceinline__ float keep_largest(const uint32_t (&v)[N], int n, int k, float top, bool write,
                                              SelectScratch& sc, Index idx) {
  const int lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
  int left = 0, out = 0;
  const uint32_t T = k < n ? warp_threshold(v, k, 1 << 20, &left) : 0u;  // (all of them are above 0)
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (32 * i >= n) break;
    const uint32_t is_eq = __ballot_sync(0xffffffffu, v[i] == T);
    const bool keep = v[i] > T || (v[i] == T && __popc(is_eq & below) < left);
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    if (keep) {
      const float score = key_score(v[i]);
      sum += expf(score - top);
      if (write) {
        const int j = out + __popc(kept & below);
        sc.idx[j] = idx(lane + 32 * i);
        sc.score[j] = score;
      }
    }
    out += __popc(kept);
    left -= min(left, __popc(is_eq));
  }
  return logf(warp_sum(sum));
}

// What a selection leaves beside the lists in its SelectScratch: how many blocks, their largest
// score and the logarithm of the sum of the exponentials over that one's. Log gates are (score -
// top) - log_sum: the sum of the two in fp32 would lose the logarithm beside large scores.
struct Kept {
  int n;
  float top, log_sum;
};

// select_here for r <= 256: every warp alone holds the row.
__device__ __forceinline__ Kept select_short(const float* __restrict__ srow, int r, int k, int mode, float log_tau,
                                             SelectScratch& sc) {
  const int lane = threadIdx.x & 31;
  uint32_t v[kCandidates / 32], hi = 0u;
#pragma unroll
  for (int i = 0; i < kCandidates / 32; ++i) {
    v[i] = lane + 32 * i < r ? score_key(__ldg(srow + lane + 32 * i)) : 0u;
    hi = max(hi, v[i]);
  }
  const float top = key_score(__reduce_max_sync(0xffffffffu, hi));
  if (mode == GBS_THRESHOLD) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kCandidates / 32; ++i) s += v[i] ? expf(key_score(v[i]) - top) : 0.f;
    const float all = top + logf(warp_sum(s));
    unsigned n = 0u;
#pragma unroll
    for (int i = 0; i < kCandidates / 32; ++i) n += v[i] && key_score(v[i]) - all >= log_tau ? 1u : 0u;
    k = min(k, (int)__reduce_add_sync(0xffffffffu, n));
    if (k == 0) return {};
  }
  const float log_sum = keep_largest(v, r, k, top, threadIdx.x < 32, sc, [](int j) { return j; });
  __syncthreads();
  return {k, top, log_sum};
}

// select_here for 256 < r <= 2048 and topk <= 96; n = -1 where too many keys are candidates.
__device__ __forceinline__ Kept select_fast(const float* __restrict__ srow, int r, int topk, int mode, float log_tau,
                                            uint32_t* work, SelectScratch& sc) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t *maxima = work, *cand_key = work + 128, *cand_idx = cand_key + kCandidates;
  // a warp holds a contiguous part of the row, 32 at a time
  const int part = (r + 127) / 128 * 32, c0 = warp * part + lane, c1 = min(r, warp * part + part);
  uint32_t u[kSelectRegs], hi = 0u;
#pragma unroll
  for (int i = 0; i < kSelectRegs; ++i) {
    u[i] = c0 + 32 * i < c1 ? score_key(__ldg(srow + c0 + 32 * i)) : 0u;
    hi = max(hi, u[i]);
  }
  maxima[tid] = hi;
  __syncthreads();
  uint32_t most[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) most[w] = maxima[32 * w + lane];
  const float top = key_score(__reduce_max_sync(0xffffffffu, max(max(most[0], most[1]), max(most[2], most[3]))));
  int k = topk;
  if (mode == GBS_THRESHOLD) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kSelectRegs; ++i) s += u[i] ? expf(key_score(u[i]) - top) : 0.f;
    s = warp_sum(s);
    if (lane == 0) sc.f[warp] = s;
    __syncthreads();
    const float all = top + logf(sc.f[0] + sc.f[1] + sc.f[2] + sc.f[3]);
    unsigned n = 0u;
#pragma unroll
    for (int i = 0; i < kSelectRegs; ++i) n += u[i] && key_score(u[i]) - all >= log_tau ? 1u : 0u;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) sc.u[1][warp] = n;
    __syncthreads();
    k = min(k, (int)(sc.u[1][0] + sc.u[1][1] + sc.u[1][2] + sc.u[1][3]));
    if (k == 0) return {};
  }
  if (warp == 0) {  // (one warp's instructions: the other CTAs of the SM use the rest)
    int need_eq;
    uint32_t t = warp_threshold(most, k, 5, &need_eq);
    if (need_eq > 0) t -= 1u;  // at least k keys are above it
    if (lane == 0) sc.bound = t;
  }
  __syncthreads();
  const uint32_t T = sc.bound;
  unsigned mine = 0u;
#pragma unroll
  for (int i = 0; i < kSelectRegs; ++i) mine += u[i] > T ? 1u : 0u;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) sc.u[0][warp] = mine;
  __syncthreads();
  unsigned at = 0u, n = 0u;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < warp) at += sc.u[0][w];
    n += sc.u[0][w];
  }
  if (n > kCandidates) return {-1};
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int i = 0; i < kSelectRegs; ++i) {
    const uint32_t is = __ballot_sync(0xffffffffu, u[i] > T);
    if (is == 0u) continue;
    if (u[i] > T) {
      const unsigned j = at + __popc(is & below);
      cand_key[j] = u[i];
      cand_idx[j] = c0 + 32 * i;
    }
    at += __popc(is);
  }
  __syncthreads();
  if (warp == 0) {
    const auto idx = [&](int j) { return (int)cand_idx[j]; };
    const auto key = [&](int j) { return j < (int)n ? cand_key[j] : 0u; };
    float sum;
    if (n <= 64) {
      const uint32_t v[2] = {key(lane), key(lane + 32)};
      sum = keep_largest(v, (int)n, k, top, true, sc, idx);
    } else {
      uint32_t v[kCandidates / 32];
#pragma unroll
      for (int i = 0; i < kCandidates / 32; ++i) v[i] = key(lane + 32 * i);
      sum = keep_largest(v, (int)n, k, top, true, sc, idx);
    }
    if (lane == 0) sc.f[0] = sum;
  }
  __syncthreads();
  return {k, top, sc.f[0]};
}

// sc.idx gets the kept blocks in ascending order and sc.score their scores. keys: r words of
// shared memory.
__device__ __forceinline__ Kept select_here(const float* __restrict__ srow, int r, int topk, int mode, float log_tau,
                                            uint32_t* keys, SelectScratch& sc) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int k = min(topk, r);
  if (k == 0) return {};
  if (r <= kCandidates) return select_short(srow, r, k, mode, log_tau, sc);
  if (r <= 128 * kSelectRegs && k <= 96) {
    const Kept fast = select_fast(srow, r, topk, mode, log_tau, keys, sc);
    if (fast.n >= 0) return fast;
    __syncthreads();
  }
  uint32_t u[kSelectRegs], hi = 0u, lo = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < kSelectRegs; ++i) {
    const int c = tid + 128 * i;
    u[i] = 0u;  // below every score's key
    if (c < r) {
      u[i] = score_key(__ldg(srow + c));
      lo = min(lo, u[i]);
    }
    hi = max(hi, u[i]);
  }
#pragma unroll
  for (int i = 0; i < kSelectRegs; ++i)
    if (tid + 128 * i < r) keys[tid + 128 * i] = u[i];
  for (int c = tid + 128 * kSelectRegs; c < r; c += 128) {
    const uint32_t x = score_key(__ldg(srow + c));
    keys[c] = x;
    lo = min(lo, x);
    hi = max(hi, x);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) sc.u[0][warp] = lo, sc.u[1][warp] = hi;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    lo = min(lo, sc.u[0][w]);
    hi = max(hi, sc.u[1][w]);
  }
  const float top = key_score(hi);
  __syncthreads();
  // the number of keys that `counts` is true of, and with it a float of each
  int round = 0;
  auto count = [&](auto counts) {
    unsigned n = 0u;
#pragma unroll
    for (int i = 0; i < kSelectRegs; ++i) n += counts(u[i]) ? 1u : 0u;
    for (int c = tid + 128 * kSelectRegs; c < r; c += 128) n += counts(keys[c]) ? 1u : 0u;
    n = __reduce_add_sync(0xffffffffu, n);
    unsigned* slot = sc.u[round++ & 1];
    if (lane == 0) slot[warp] = n;
    __syncthreads();
    return (int)(slot[0] + slot[1] + slot[2] + slot[3]);
  };
  if (mode == GBS_THRESHOLD) {
    float s = 0.f;
    for (int c = tid; c < r; c += 128) s += expf(key_score(keys[c]) - top);
    s = warp_sum(s);
    if (lane == 0) sc.f[warp] = s;
    __syncthreads();
    const float all = top + logf(sc.f[0] + sc.f[1] + sc.f[2] + sc.f[3]);
    k = min(k, count([&](uint32_t x) { return x != 0u && key_score(x) - all >= log_tau; }));
    if (k == 0) return {};
  }
  // keys above T are kept, and the first need_eq of those equal to it
  uint32_t T = lo - 1u;
  int need_eq = 0;
  if (k < r) {
    uint32_t above = hi + 1u;  // fewer than k keys reach it, at least k reach lo
    int n_above = 0;
    T = lo;
    need_eq = -1;
    for (int it = 0; above - T > 1u; ++it) {
      uint32_t mid = T + (above - T) / 2;
      if (it < 14) {  // between the scores, where that is inside
        const uint32_t x = ordered_key(0.5f * key_score(T) + 0.5f * key_score(above - 1u));
        if (x > T && x < above) mid = x;
      }
      const int n = count([&](uint32_t x) { return x >= mid; });
      if (n == k) {
        T = mid - 1u;
        need_eq = 0;
        break;
      }
      if (n > k) T = mid;
      else above = mid, n_above = n;
    }
    if (need_eq < 0) need_eq = k - n_above;
  }
  // each warp compacts a contiguous part of the row
  const int part = ((r + 31) / 32 + 3) / 4 * 32, c0 = warp * part, c1 = min(r, c0 + part);
  int gt = 0, eq = 0;
  for (int c = c0 + lane; c - lane < c1; c += 32) {
    const uint32_t x = c < c1 ? keys[c] : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, c < c1 && x > T));
    eq += __popc(__ballot_sync(0xffffffffu, c < c1 && x == T));
  }
  __syncthreads();  // the last count's slots are read
  if (lane == 0) sc.u[0][warp] = (unsigned)gt, sc.u[1][warp] = (unsigned)eq;
  __syncthreads();
  int at = 0, left = need_eq;
  for (int w = 0; w < warp; ++w) {
    const int e = min(left, (int)sc.u[1][w]);
    at += (int)sc.u[0][w] + e;
    left -= e;
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int c = c0 + lane; c - lane < c1; c += 32) {
    const uint32_t x = c < c1 ? keys[c] : 0u;
    const uint32_t is_eq = __ballot_sync(0xffffffffu, c < c1 && x == T);
    const bool keep = c < c1 && (x > T || (x == T && __popc(is_eq & below) < left));
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    if (keep) {
      const int j = at + __popc(kept & below);
      sc.idx[j] = c;
      sc.score[j] = key_score(x);
    }
    at += __popc(kept);
    left -= min(left, __popc(is_eq));
  }
  __syncthreads();
  float s = 0.f;
  for (int j = lane; j < k; j += 32) s += expf(sc.score[j] - top);
  return {k, top, logf(warp_sum(s))};
}

// The log gate of kept block e in powers of two. It stays finite, so that a maximum made of it
// does: a score of fp32's lowest, as masks have, would give -infinity (a weight of 0 either way).
__device__ __forceinline__ float log2_gate(const Kept& kept, const SelectScratch& sc, int e) {
  const float x = (sc.score[e] - kept.top - kept.log_sum) * GBS_LOG2E;
  return x < -1e30f ? -1e30f : x;
}

// A CTA's kept blocks, by its own selection or from the lists made before, into sc.
__device__ __forceinline__ Kept kept_blocks(const DecodeArgs& a, int srow, int cur, uint32_t* keys, SelectScratch& sc) {
  const float* scores = a.S + (size_t)srow * a.p.Nb;
  if (!a.sel.idx) return select_here(scores, cur, a.p.topk, a.p.mode, a.p.log_tau, keys, sc);
  const int n = cur > 0 ? dcheck(a.sel.cnt[srow], 0, min(a.p.topk, cur), a.c.err) : 0;
  for (int j = threadIdx.x; j < n; j += 128) {
    const int c = dcheck(a.sel.idx[(size_t)srow * a.p.topk + j], 0, cur - 1, a.c.err);
    sc.idx[j] = c;
    sc.score[j] = __ldg(scores + c);
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int j = threadIdx.x & 31; j < n; j += 32) top = fmaxf(top, sc.score[j]);
  top = warp_max(top);
  for (int j = threadIdx.x & 31; j < n; j += 32) sum += expf(sc.score[j] - top);
  return {n, top, logf(warp_sum(sum))};
}

// The splits of a row are a cluster and join their sums of n = heads * D channels: every
// CTA writes each 128 of its sums into the memory of the CTA that joins these 128, and the
// (maximum, sum) of the heads in them, so that after one barrier all reads are local (reading
// the others' memory, with a barrier on both sides, took about 1 us longer).
struct Inbox {
  float sums[kMaxCluster * 128];  // of split r, its x-th 128 of this CTA: at (x * splits + r) * 128
  float2 ml[kMaxCluster][4];
};
static_assert(sizeof(Inbox) % 16 == 0, "");
__device__ __forceinline__ void cluster_arrive_early() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Channel i's sum v, and its head's maximum M and sum l, to the CTA that joins it.
template <int D>
__device__ __forceinline__ void send_sum(const DecodeArgs& a, Inbox* inbox, int split, int i, float v, float M, float l) {
  const int chunk = i / 128;
  Inbox* to = cooperative_groups::this_cluster().map_shared_rank(inbox, chunk % a.splits);
  to->sums[(chunk / a.splits * a.splits + split) * 128 + i % 128] = v;
  if (i % D == 0) to->ml[split][i / D] = make_float2(M, l);
}

// The joined sums to output elements row0 * D + i. A row without a key (a length of 0) gives
// 0 and -infinity.
template <typename T, int D>
__device__ __forceinline__ void join_splits(const DecodeArgs& a, const Inbox* inbox, int n, int split, size_t row0) {
  cluster_arrive();
  cluster_wait();
  for (int i = split * 128 + threadIdx.x, x = 0; i < n; i += a.splits * 128, ++x) {
    const int h = i / D;
    float M = -INFINITY, l = 0.f, v = 0.f;
    for (int r = 0; r < a.splits; ++r) M = fmaxf(M, inbox->ml[r][h].x);
#pragma unroll 4
    for (int r = 0; r < a.splits; ++r) {
      const float2 ml = inbox->ml[r][h];
      const float f = ml.x == -INFINITY ? 1.f : exp2f(ml.x - M);
      l += ml.y * f;
      v += inbox->sums[(x * a.splits + r) * 128 + i % 128] * f;
    }
    store_out(reinterpret_cast<T*>(a.O) + row0 * D + i, l == 0.f ? 0.f : v / l);
    if (i % D == 0) a.LSE[row0 + h] = l == 0.f ? -INFINITY : (M + log2f(l)) * GBS_LN2;
  }
}

// fp32 queries: one query head and split per CTA, all in fp32, so queries keep their 24
// bits. A lane holds 32 channels of a row (16 code bytes), so D / 32 lanes hold a row and a
// warp 32 / (D / 32) rows. Bound by its arithmetic (every value is unpacked for one head);
// four uneven sequences of up to 4133 tokens, K = 8, take 10.4 us, most of it latency.
template <typename T, int D>
__global__ void __launch_bounds__(128) kv4_decode_simt_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int NG = D / 32, LANES = NG, ROWS = 128 / LANES;
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t* s_keys = reinterpret_cast<uint32_t*>(smem);
  __shared__ SelectScratch select;
  __shared__ float s_acc[4][D], s_m[4], s_l[4];
  const Problem& p = a.p;
  const int b = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq, split = blockIdx.y, kvh = hq / p.G;
  const int srow = a.grouped ? b * p.Hkv + kvh : blockIdx.x;
  const int lane = threadIdx.x % LANES, row_in = threadIdx.x / LANES;
  Inbox* inbox = reinterpret_cast<Inbox*>(reinterpret_cast<char*>(s_keys) + a.inbox);
  if (a.splits > 1) cluster_arrive_early();
  const int L = sequence_length(a, b), cur = L > 0 ? (L - 1) / kBS : 0;
  const Kept kept = kept_blocks(a, srow, cur, s_keys, select);
  const int n_hist = kept.n;
  const int n_ent = L > 0 ? n_hist + 1 : 0, per = (n_ent + a.splits - 1) / a.splits;
  const int e0 = split * per, e1 = min(n_ent, e0 + per);
  // 16-bit word 8 lane + i / 4 holds channels 4 chunk + i % 4 of group grp
  float q[32], acc[32] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int hw = 8 * lane + i / 4, c = 32 * (hw % NG) + 4 * (hw / NG) + i % 4;
    q[i] = to_f32<T>(reinterpret_cast<const T*>(a.q)[((size_t)b * p.Hq + hq) * D + c]) * p.scale_log2;
  }
  for (int e = e0; e < e1; ++e) {
    const bool is_cur = e == n_hist;
    const int c = is_cur ? cur : dcheck(select.idx[e], 0, cur - 1, a.c.err);
    const float bias = is_cur ? 0.f : log2_gate(kept, select, e);
    const long long row0 = block_row(a, b, kvh, c);
    if (row0 < 0) continue;
    const int nrows = is_cur ? L - cur * kBS : kBS;
    for (int r = row_in; r < kBS; r += ROWS) {
      float z = 0.f;
      const bool there = r < nrows;
      const long long at = row0 + (there ? r : 0);
      const uint4 kw = __ldg(reinterpret_cast<const uint4*>(a.c.kc + at * (D / 2)) + lane);
      const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
      float ks[NG], km[NG], vs[NG], vm[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t kp = __ldg(a.c.kp + at * NG + g), vp = __ldg(a.c.vp + at * NG + g);
        ks[g] = low_half(kp); km[g] = high_half(kp);
        vs[g] = low_half(vp); vm[g] = high_half(vp);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int g = (i / 4) % NG;
        z = fmaf(q[i], fmaf(ks[g], (float)(w[i / 8] >> (4 * (i % 8)) & 15u), km[g]), z);
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      if (!there) continue;
      z += bias;
      if (z > m) {
        const float f = exp2f(m - z);
        l *= f;
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[i] *= f;
        m = z;
      }
      // a NaN or infinite score leaves m where it was and makes the row's sum NaN
      const float pr = exp2f(z - m);
      l += pr;
      const uint4 vw = __ldg(reinterpret_cast<const uint4*>(a.c.vc + at * (D / 2)) + lane);
      const uint32_t x[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int g = (i / 4) % NG;
        acc[i] = fmaf(pr, fmaf(vs[g], (float)(x[i / 8] >> (4 * (i % 8)) & 15u), vm[g]), acc[i]);
      }
    }
  }
  // join the rows of a warp, then the warps
  float M = m;
#pragma unroll
  for (int o = LANES; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float f = m == -INFINITY ? 0.f : exp2f(m - M);
  l *= f;
#pragma unroll
  for (int o = LANES; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float v = m == -INFINITY ? acc[i] : acc[i] * f;
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int hw = 8 * lane + i / 4;
    if (threadIdx.x % 32 < LANES) s_acc[warp][32 * (hw % NG) + 4 * (hw / NG) + i % 4] = v;
  }
  if (threadIdx.x % 32 == 0) s_m[warp] = M, s_l[warp] = l;
  __syncthreads();
  float MM = -INFINITY, ll = 0.f;
  for (int w = 0; w < 4; ++w) MM = fmaxf(MM, s_m[w]);
  float fw[4];
  for (int w = 0; w < 4; ++w) {
    fw[w] = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - MM);
    ll += s_l[w] * (s_m[w] == -INFINITY ? 1.f : fw[w]);
  }
  const size_t row = (size_t)b * p.Hq + hq;
  if (a.splits > 1) cluster_wait();  // every CTA of the row has begun
  for (int c = threadIdx.x; c < D; c += 128) {
    float v = 0.f;
    for (int w = 0; w < 4; ++w) v += s_acc[w][c] * (s_m[w] == -INFINITY ? 1.f : fw[w]);
    if (a.splits > 1) send_sum<D>(a, inbox, split, c, v, MM, ll);
    else store_out(reinterpret_cast<T*>(a.O) + row * D + c, ll == 0.f ? 0.f : v / ll);
  }
  if (a.splits > 1) join_splits<T, D>(a, inbox, D, split, row);
  else if (threadIdx.x == 0) a.LSE[row] = ll == 0.f ? -INFINITY : (MM + log2f(ll)) * GBS_LN2;
}

// ------------------------------------------------------------ tensor-core decode
// bf16 queries. A CTA serves up to four query heads of one selection row (one head
// without a shared selection) over its share of the kept blocks. Each of its four warps
// works alone until the end, on every fourth half block: 32 keys, whose codes and
// parameters (5,120 bytes for d = 128) arrive by bulk copies into the warp's own ring of
// stages, issued by its first lanes when a stage has been read.
//
//   z[key, head] = sum_g s_g sum_{i in g} n_i q_i + sum_g m_g sum_{i in g} q_i
// The inner sums are m16n8k16 products of codes (rows: keys) and q as fp16, both exact: q
// is scaled by a power of two for each head so that it fits, scales are applied to the
// fp32 sums, and the minima's part is one more product, of the raw parameter words with
// the sums of q as two fp16 terms, which leaves 2^-23 of them: less than fp32 sums do.
//   O[channel, head] = sum_key n (s p) + sum_key m p
// with codes as rows again. Weights p and products s p go in as two fp16 terms each, which
// leaves 2^-21 of them, and sums are fp32: with one term (2^-12) one result in seven was a
// bf16 step beside the nearest, with two one in a hundred.
//
// A nibble masked out of a 32-bit word of codes stands for an fp16 pair as it is (kLow,
// kHigh below), one from a group 2 P (low half) and one from group 2 P + 1. Both go
// through a product together: its eight columns are four heads times the two groups of a
// pair, column c with zeros where the other group's factor would be. So codes need
// nothing but masks and one shift, the accumulators have no padding but unused heads, and
// the two groups' logits meet in one exchange between lanes. A CTA of one head takes groups
// as columns instead (ONE below).
//
// Bound with a selection for each head by memory and the beginnings of its CTAs (64 sequences
// x 131072, K = 32, d = 128: 679 MB that differ, 104 us at the copy rate): 131 us (5.2 TB/s),
// of which the products and softmaxes add 18 to the copies and selections alone (112, in which
// the first CTAs of all SMs select before anything is copied). With one for four heads: 53 us
// (178 MB, 27 us), the copies alone 31, selections 4, the rest instructions, most of them
// masks, factors and the softmax; the second terms take 8 (the products of them 1.4, the
// making of them the rest). Steps, calls per head /
// shared: one key a thread in fp32 393 / 371 us, products with heads as rows 299 / 101, keys
// and channels as rows 208 / 73, raw nibbles and a ring for each warp 189 / 70, both groups of
// a pair as columns 173 / 65, selection and join inside 157 / 50, one path for all scales
// 148 / 50, one warp ending the selection 142 / 47, one head a kernel of its own 128 / 46,
// whole bytes as operands 126 / 45, second terms of weights and products 129 / 52, nibbles apart
// again 131 / 53. Other shapes of it, each against its time's kernel: three
// CTAs an SM 178 / 74 (161 / 54), five with 96 registers 157 / 58 (148 / 51) and, of one head,
// 131 (127), three stages a warp 156 / 63 (141 / 47), the loop over channels rolled 167 / 57
// (151 / 53).
constexpr int kUnit = 32;  // keys of a warp's turn
template <int D>
struct Kv4Tile {
  static constexpr int NG = D / 32, RB = D / 2, PB = NG * 4;
  static constexpr int kKp = kUnit * RB, kV = kKp + kUnit * PB, kVp = kV + kKp;
  static constexpr int kStage = kVp + kUnit * PB;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kWarp = kStages * kStage, kBytes = 4 * kWarp;
  static_assert(kWarp >= 4 * D * 4, "a warp's sums go into its stages' memory");
  static_assert(kBytes >= 4 * 8192, "a row's keys are held in the stages' memory before copies begin");
};
constexpr int kMmaThreads = 128;
constexpr uint64_t kWaitNs = 4000000000ull;
// In the debug build a call whose error word already holds GBS_ERR_TIMEOUT takes its first waits
// for expired, once the copies have come: so tests reach what follows.
#ifdef GBS_DEBUG
__device__ __forceinline__ int starts_given_up(const unsigned int* err) { return *err == GBS_ERR_TIMEOUT; }
__device__ __forceinline__ bool gives_up(int abort) { return abort != 0; }
#else
__device__ __forceinline__ int starts_given_up(const unsigned int*) { return 0; }
__device__ __forceinline__ bool gives_up(int) { return false; }
#endif
// Weights are 2^(z - m), with m kLift below the largest z when it was set, and at most
// 2^kRoom; where scales reach 2^e, e > 0, both are e less. So no product of a weight and a
// scale leaves fp16, and its steps of 2^-24 are 2^-34 of the largest weight.
constexpr float kLift = 10.f, kRoom = 14.f;
// A nibble alone is the fp16 of its code times 2^-24 (low in its byte) or 2^-20 (high):
// products take it as it is, exactly, and the power of two goes into what it meets.
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
// (Whole bytes, low + 16 high, less the high nibbles at the end took an instruction less for
// the upper bytes of a word, 2 us of 131, but their sums are 17 times as large at equal codes
// and 241 times at 1 beside 15, and so are the steps of fp32: one low channel in ten was off.)

// c = a b, and c += a b
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma16816_add(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
__device__ __forceinline__ uint32_t as_word(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) { return as_word(__floats2half2_rn(lo, hi)); }
// What fp16 leaves of lo and hi, as fp16: *two gets their first terms.
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t* two) {
  const __half2 h = __floats2half2_rn(lo, hi);
  const float2 f = __half22float2(h);
  *two = as_word(h);
  return pack_half2(lo - f.x, hi - f.y);
}
// The product of (p + rest) and s as two fp16 terms: p s - top is exact (in steps of 2^-24).
__device__ __forceinline__ uint32_t product_rest(uint32_t p, uint32_t rest, uint32_t s, uint32_t* top) {
  const __half2 x = __hmul2(as_half2(p), as_half2(s));
  *top = as_word(x);
  return as_word(__hfma2(as_half2(rest), as_half2(s), __hfma2(as_half2(p), as_half2(s), __hneg2(x))));
}

// The transpose of an 8 x 8 matrix of fp16: a lane's word is row lane / 4, columns 2 (lane % 4) and the next.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t w) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
}

// N words of shared memory at an address and a constant offset from it.
template <int N>
__device__ __forceinline__ void load_words(uint32_t at, int off, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at + off));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at + off));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at + off));
}
__device__ __forceinline__ uint32_t load_word(uint32_t at, int off) {
  uint32_t w[1];
  load_words<1>(at, off, w);
  return w[0];
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ONE: a single head a CTA. Then the columns are the groups of a row (repeated where there
// are fewer than eight), so that the value products of all pairs of groups share their
// accumulators, and after the key products every lane holds the logit of one key of its own:
// one exponential, and the minima's part as products of its own, for 32 keys.
template <int D, bool ONE>
__global__ void __launch_bounds__(kMmaThreads, 4) kv4_decode_mma_kernel(const __grid_constant__ DecodeArgs a) {
  using Tile = Kv4Tile<D>;
  constexpr int NG = Tile::NG, NP = NG / 2, S = Tile::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full_all[4][S];
  __shared__ float bias_all[4][S], s_m[4][4], s_l[4][4];
  __shared__ int rows_all[4][S], s_abort;
  __shared__ SelectScratch select;
  Inbox* inbox = reinterpret_cast<Inbox*>(smem + a.inbox);
  if (a.splits > 1) cluster_arrive_early();
  const Problem& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* full = full_all[warp];
  float* s_bias = bias_all[warp];
  int* s_rows = rows_all[warp];
  uint8_t* ring = smem + warp * Tile::kWarp;

  // the CTA's selection row and heads
  int b, kvh, h0, nh, srow;
  if (a.grouped) {
    const int n_sub = (p.G + 3) / 4, sub = blockIdx.x % n_sub;
    srow = blockIdx.x / n_sub;
    b = srow / p.Hkv;
    kvh = srow % p.Hkv;
    h0 = kvh * p.G + sub * 4;
    nh = ONE ? 1 : min(4, p.G - sub * 4);
  } else {
    srow = blockIdx.x;
    b = srow / p.Hq;
    h0 = srow % p.Hq;
    kvh = h0 / p.G;
    nh = 1;
  }
  const int split = blockIdx.y;
  const int L = sequence_length(a, b), cur = L > 0 ? (L - 1) / kBS : 0;
  if (threadIdx.x == 0) s_abort = starts_given_up(a.c.err);
  const Kept kept = kept_blocks(a, srow, cur, reinterpret_cast<uint32_t*>(smem), select);
  const int n_hist = kept.n;
  if (!a.sel.idx) {
    sm100::fence_proxy_async_smem();  // copies will write over the keys
    __syncthreads();
  }
  const int n_ent = L > 0 ? n_hist + 1 : 0, per = (n_ent + a.splits - 1) / a.splits;
  const int e0 = split * per, e1 = min(n_ent, e0 + per);
  // this warp's blocks are first, first + 2, ...; it takes their keys half .. half + 31
  const int first = e0 + (warp >> 1), half = (warp & 1) * kUnit;
  const int turns = first < e1 ? (e1 - first + 1) / 2 : 0;

  if (lane == 0) {
    for (int s = 0; s < S; ++s) sm100::mbar_init(&full[s], 1);
    sm100::fence_barrier_init();
  }
  __syncwarp();

  // places of 32 of the warp's turns at once, a lane each, so that no copy waits for its
  // lookup: the half block's index among all of the cache's
  int my_unit = 0, my_rows = 0;
  float my_bias = 0.f;
  const uint8_t* copy_from = lane < 2 ? (lane ? (const uint8_t*)a.c.kp : a.c.kc) : (lane & 1 ? (const uint8_t*)a.c.vp : a.c.vc);
  const uint32_t copy_row = lane & 1 ? Tile::PB : Tile::RB;
  const uint32_t copy_to = (lane & 2 ? Tile::kV : 0) + (lane & 1 ? Tile::kKp : 0);
  auto look_up = [&](int turn) {
    const int e = first + 2 * turn;
    my_rows = 0;
    if (turn < turns) {
      const bool is_cur = e == n_hist;
      const int c = is_cur ? cur : dcheck(select.idx[e], 0, cur - 1, a.c.err);
      my_bias = is_cur ? 0.f : log2_gate(kept, select, e);
      const long long row = block_row(a, b, kvh, c);
      my_unit = (int)(row / kUnit) + (warp & 1);
      my_rows = row < 0 ? 0 : min(kUnit, is_cur ? L - cur * kBS - half : kUnit);
    }
  };
  auto issue = [&](int turn, int s) {
    if (turn > 0 && (turn & 31) == 0) look_up(turn + lane);
    const int unit = __shfl_sync(0xffffffffu, my_unit, turn & 31);
    const float bias = __shfl_sync(0xffffffffu, my_bias, turn & 31);
    const int n = __shfl_sync(0xffffffffu, my_rows, turn & 31);
    const uint32_t m = n > 0 ? (n + 1) & ~1 : 0;  // whole 16-byte units of the parameters too
    if (lane == 0) {
      s_bias[s] = bias;
      s_rows[s] = n;
      sm100::mbar_arrive_expect_tx(&full[s], 2 * m * (Tile::RB + Tile::PB));
    }
    __syncwarp();
    if (lane < 4 && m > 0)  // one of the four tensors each
      sm100::bulk_load(ring + s * Tile::kStage + copy_to, copy_from + (size_t)unit * (kUnit * copy_row), m * copy_row, &full[s]);
  };
  look_up(lane);
  for (int s = 0; s < S && s < turns; ++s) issue(s, s);

  const int g = lane >> 2, t = lane & 3;
  // q as fp16 times a power of two, the largest of a head in 2^8 .. 2^9: 2^-ex in two steps,
  // either of which fp32 can hold, and the logits' factor that undoes it (not 0, since keys
  // behind the sequence have -infinity times it)
  float down0, down1;
  auto fit = [&](float mx) {
    int ex = (int)(__float_as_uint(mx) >> 23) - 127 - 8;
    if (ex == 120) ex = 0;  // infinite: as it is
    down0 = ldexpf(1.f, -(ex / 2)), down1 = ldexpf(1.f, -(ex - ex / 2));
    return fmaxf(p.scale_log2 * ldexpf(1.f, ex / 2) * ldexpf(1.f, ex - ex / 2), 0x1p-126f);
  };
  auto load_q = [&](const __nv_bfloat16* q, bool there, float (&v)[8], float& mx) {
    const uint4 u = there ? __ldg(reinterpret_cast<const uint4*>(q)) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      mx = fmaxf(mx, fabsf(v[i]));
    }
  };
  // channel i of eight: nibble i % 4 of the lane's word i / 4. High nibbles count 16 times; of
  // q, whose largest is 2^8 or more, that rounds only steps below 2^-20: 2^-29 of the largest
  auto operand = [&](float v, int i, float& sum) {
    const __half x = __float2half_rn(v * down0 * down1);
    sum += __half2float(x);
    return (uint32_t)__half_as_ushort(i & 1 ? __hmul(x, __ushort_as_half(0x2c00)) : x);  // 2^-4
  };
  uint32_t qb[NP][8], qm0 = 0u, qm1 = 0u;
  float zs[2], q_sum[2];
  if constexpr (ONE) {
    // column g of a product: group g % NG; result columns 2 t and 2 t + 1: groups 2 t % NG and the next
    const int group = g & (NG - 1);
    float v[8], mx = 0.f, sum = 0.f;
    load_q(reinterpret_cast<const __nv_bfloat16*>(a.q) + ((size_t)b * p.Hq + h0) * D + 32 * group + 8 * t, true, v, mx);
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    zs[0] = fit(mx);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t bits = operand(v[i], i, sum);
#pragma unroll
      for (int P = 0; P < NP; ++P) qb[P][i] = group >> 1 == P ? bits << 16 * (group & 1) : 0u;
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
    for (int c = 0; c < 2; ++c) q_sum[c] = __shfl_sync(0xffffffffu, sum, 4 * ((2 * t & (NG - 1)) + c));
  } else {
    // column g of a product: head g & 3, group parity g >> 2; result columns 2 t and 2 t + 1:
    // heads 2 t & 3 and the next, parity t >> 1
    const int h = g & 3, par = g >> 2;
    float v[NP][8], mx = 0.f;
#pragma unroll
    for (int P = 0; P < NP; ++P)
      load_q(reinterpret_cast<const __nv_bfloat16*>(a.q) + ((size_t)b * p.Hq + h0 + h) * D + 32 * par + 8 * t + 64 * P,
             h < nh, v[P], mx);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    const float zscale = fit(mx);
    zs[0] = __shfl_sync(0xffffffffu, zscale, 4 * (2 * t & 3));
    zs[1] = __shfl_sync(0xffffffffu, zscale, 4 * (2 * t & 3) + 4);
    float qsum = 0.f;
#pragma unroll
    for (int P = 0; P < NP; ++P) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) qb[P][i] = operand(v[P][i], i, sum) << 16 * par;
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      // the minima's product takes parameter word t of a key as (s, m): group t's sum to m
      const float of_t = __shfl_sync(0xffffffffu, sum, 4 * (h + 4 * (t & 1)) + t);
      if (t >> 1 == P && par == 0) qsum = of_t;
    }
    const float hi = __half2float(__float2half_rn(qsum));
    qm0 = pack_half2(0.f, hi);
    qm1 = pack_half2(0.f, qsum - hi);
  }
  __syncthreads();  // s_abort is set

  // sums of the result columns' heads; a head that is not there never raises its maximum
  // (o in units of 2^-24 and 2^-20 of low and high nibbles; om: the minima's part, group g)
  // (ONE: om of a lane's own keys, for every group)
  constexpr int kSums = ONE ? 2 : NP * 2;
  float o[kSums][4], om[4] = {0.f, 0.f, 0.f, 0.f}, m[2], l[2] = {0.f, 0.f};
  const int hc = 2 * t & 3;  // head of column 2 t
  m[0] = ONE || hc < nh ? -INFINITY : INFINITY;
  m[1] = hc + 1 < nh ? -INFINITY : INFINITY;
#pragma unroll
  for (int i = 0; i < kSums; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

  // the product's row n is key n ^ (n >> 1 & 1) of eight, an order in which neither
  // kind of load meets a bank twice more than it must
  const int row_k = g ^ (g >> 1 & 1), row_v0 = 2 * t ^ (t & 1), row_v1 = (2 * t + 1) ^ (t & 1);
  const uint32_t ring_at = sm100::smem_u32(ring);
  const uint32_t at_k = row_k * Tile::RB + t * (Tile::RB / 4), at_kp = Tile::kKp + row_k * Tile::PB;
  const uint32_t at_v0 = Tile::kV + row_v0 * Tile::RB + g * (Tile::RB / 8);
  const uint32_t at_v1 = Tile::kV + row_v1 * Tile::RB + g * (Tile::RB / 8);
  const uint32_t at_vp0 = Tile::kVp + row_v0 * Tile::PB, at_vp1 = Tile::kVp + row_v1 * Tile::PB;
  const uint32_t par_k = 4 * (t >> 1), par_v = 4 * (g >> 2);
  // byte selectors that put the low or high half of a word into the half of column g's parity
  const uint32_t sel0 = g >> 2 ? 0x1044u : 0x4410u, sel1 = g >> 2 ? 0x3244u : 0x4432u;
  // ONE: a lane's own key among the 32, its column's group, and the selectors for that (or
  // nothing, for the other pairs of groups)
  const int my_key = 8 * t + row_k, group = g & (NG - 1);
  uint32_t lo_to[NP], hi_to[NP];
#pragma unroll
  for (int P = 0; P < NP; ++P) {
    lo_to[P] = group >> 1 != P ? 0x4444u : group & 1 ? 0x1044u : 0x4410u;
    hi_to[P] = group >> 1 != P ? 0x4444u : group & 1 ? 0x3244u : 0x4432u;
  }
  // what the value scales of 32 keys, a key's parameters to a lane, leave of kRoom
  auto room_for = [](const uint32_t (&params)[NG]) {
    uint32_t most = 0u;
#pragma unroll
    for (int k = 0; k < NG; ++k) most = max(most, params[k] & 0x7fffu);  // (a group whose minimum rounds up may have s < 0)
    most = __reduce_max_sync(0xffffffffu, most);
    return most >= 0x3c00u ? kRoom - (float)((int)(most >> 10) - 14) : kRoom;  // fp16 of 1 and more
  };
  int s = 0;
  uint32_t parity = 0;
  for (int turn = 0; turn < turns; ++turn) {
    if (!sm100::mbar_wait(&full[s], parity, &s_abort, a.c.err, kWaitNs) || gives_up(s_abort)) {
      // given up: no copy may be in flight when the CTA ends
      if (lane == 0)
        for (int i = turn; i < turns && i < turn + S; ++i) sm100::mbar_drain(&full[i % S], (i / S) & 1, 1000000ull);
      __syncwarp();
      break;
    }
    const uint32_t st = ring_at + s * Tile::kStage;
    const uint32_t lk = st + at_k, lkp = st + at_kp, lv0 = st + at_v0, lv1 = st + at_v1, lvp0 = st + at_vp0, lvp1 = st + at_vp1;
    const int rows = s_rows[s];
    if (rows > 0) {
      const bool ends = rows < kUnit;  // the sequence ends in these keys
      if (ends) {
        __syncwarp();  // (a branch of its own: it is seldom taken)
        if (lane >= rows)
#pragma unroll
          for (int k = 0; k < NG; ++k) {  // whatever lies behind the sequence stands for zeros
            uint32_t* params = reinterpret_cast<uint32_t*>(ring + s * Tile::kStage + Tile::kKp + lane * Tile::PB);
            params[k] = params[Tile::kV / 4 + k] = 0u;
          }
        __syncwarp();
      }
      if constexpr (ONE) {
        const float bias = s_bias[s];
        // the products of 16 keys y: c[y][0], c[y][1] of key row_k and c[y][2], c[y][3] of
        // row_k + 8, with the groups of columns 2 t and 2 t + 1
        float c[2][4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t kw[2][NG];
#pragma unroll
          for (int x = 0; x < 2; ++x) load_words<NG>(lk, (16 * y + 8 * x) * Tile::RB, kw[x]);
#pragma unroll
          for (int P = 0; P < NP; ++P)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w0 = kw[0][NP * j + P], w1 = kw[1][NP * j + P], h0 = w0 >> 8, h1 = w1 >> 8;
              if (P == 0 && j == 0) mma16816(c[y], w0 & kLow, w1 & kLow, w0 & kHigh, w1 & kHigh, qb[P][0], qb[P][1]);
              else mma16816_add(c[y], w0 & kLow, w1 & kLow, w0 & kHigh, w1 & kHigh, qb[P][4 * j], qb[P][4 * j + 1]);
              mma16816_add(c[y], h0 & kLow, h1 & kLow, h0 & kHigh, h1 & kHigh, qb[P][4 * j + 2], qb[P][4 * j + 3]);
            }
        }
        // the logit of the lane's own key, 16 (t / 2) + 8 (t % 2) + row_k
        const bool late = t >> 1, odd = t & 1;
        auto logit = [&](float c0, float c1, int key) {  // of a key's two groups
          uint32_t w[2];
          load_words<2>(st + Tile::kKp + key * Tile::PB + 4 * (2 * t & (NG - 1)), 0, w);
          return fmaf(fmaf(low_half(w[1]), c1, low_half(w[0]) * c0), 0x1p24f,
                      fmaf(high_half(w[1]), q_sum[1], high_half(w[0]) * q_sum[0]));
        };
        float z;
        const float c0 = late ? c[1][0] : c[0][0], c1 = late ? c[1][1] : c[0][1];
        const float c2 = late ? c[1][2] : c[0][2], c3 = late ? c[1][3] : c[0][3];
        if constexpr (NG == 4) {  // the lanes 2 and 2 + 1 of four hold two groups each
          const int key = 16 * (t >> 1) + row_k;
          const float z0 = logit(c0, c1, key), z1 = logit(c2, c3, key + 8);
          z = (odd ? z1 : z0) + __shfl_xor_sync(0xffffffffu, odd ? z0 : z1, 1);
        } else {
          z = logit(odd ? c2 : c0, odd ? c3 : c1, my_key);
        }
        if (my_key >= rows) z = -INFINITY;  // (the scale is not negative)
        uint32_t vp[NG];
        load_words<NG>(st + my_key * Tile::PB, Tile::kVp, vp);
        const float room = room_for(vp);
        float x = fmaf(z, zs[0], bias - m[0]);
        if (__any_sync(0xffffffffu, x > room)) {  // as below
          float mx = z;
#pragma unroll
          for (int w = 1; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          const float mn = fmaxf(m[0], fmaf(mx, zs[0], bias) + (kRoom - kLift - room));
          const float f = m[0] == mn ? 1.f : fast_exp2(m[0] - mn);
          m[0] = mn;
          l[0] *= f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            om[i] *= f;
            o[0][i] *= f;
            o[1][i] *= f;
          }
          x = fmaf(z, zs[0], bias - m[0]);
        }
        const float pr = fast_exp2(x);
        l[0] += pr;
#pragma unroll
        for (int k = 0; k < NG; ++k) om[k] = fmaf(pr, high_half(vp[k]), om[k]);
        // weights as two fp16 terms, of product rows 2 t and 2 t + 1 of each eight keys, in every
        // column: columns 0 to 3 take the products' first terms, 4 to 7 the rest
        const float other = __shfl_xor_sync(0xffffffffu, pr, 4);
        uint32_t two;
        const uint32_t rest = pack_rest(g & 1 ? other : pr, g & 1 ? pr : other, &two);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t pw = __shfl_sync(0xffffffffu, two, 8 * t + e), pl = __shfl_sync(0xffffffffu, rest, 8 * t + e);
          uint32_t vw[2][NP];
          load_words<NP>(lv0, 8 * e * Tile::RB, vw[0]);
          load_words<NP>(lv1, 8 * e * Tile::RB, vw[1]);
          const uint32_t sc = __byte_perm(load_word(lvp0 + 4 * group, 8 * e * Tile::PB),
                                          load_word(lvp1 + 4 * group, 8 * e * Tile::PB), 0x5410);
          uint32_t top;
          const uint32_t low = product_rest(pw, pl, sc, &top), ps = g >> 2 ? low : top;
#pragma unroll
          for (int P = 0; P < NP; ++P) {
            const uint32_t w0 = vw[0][P], w1 = vw[1][P], h0 = w0 >> 8, h1 = w1 >> 8;
            const uint32_t b0 = __byte_perm(ps, 0u, lo_to[P]), b1 = __byte_perm(ps, 0u, hi_to[P]);
            mma16816_add(o[0], w0 & kLow, w0 & kHigh, w1 & kLow, w1 & kHigh, b0, b1);
            mma16816_add(o[1], h0 & kLow, h0 & kHigh, h1 & kLow, h1 & kHigh, b0, b1);
          }
        }
      } else {
        // of 16 keys y: z of keys row_k (z[y][0], z[y][1]: heads 2 t, 2 t + 1) and row_k + 8
        float z[2][4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t kw[2][NG], km[2];
          float sc[2][NP];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = 16 * y + 8 * x;
            load_words<NG>(lk, r * Tile::RB, kw[x]);
#pragma unroll
            for (int P = 0; P < NP; ++P)  // (the codes' products are 2^-24 of what they stand for)
              sc[x][P] = low_half(load_word(lkp + par_k, r * Tile::PB + 8 * P)) * 0x1p24f;
            km[x] = t < NG ? load_word(lkp + 4 * t, r * Tile::PB) : 0u;
          }
          mma16816(z[y], km[0], km[1], km[0], km[1], qm0, qm1);
#pragma unroll
          for (int P = 0; P < NP; ++P) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 2; ++j) {  // four channels 2 t + j of both groups
              const uint32_t w0 = kw[0][NP * j + P], w1 = kw[1][NP * j + P], h0 = w0 >> 8, h1 = w1 >> 8;
              mma16816_add(c, w0 & kLow, w1 & kLow, w0 & kHigh, w1 & kHigh, qb[P][4 * j], qb[P][4 * j + 1]);
              mma16816_add(c, h0 & kLow, h1 & kLow, h0 & kHigh, h1 & kHigh, qb[P][4 * j + 2], qb[P][4 * j + 3]);
            }
            z[y][0] = fmaf(sc[0][P], c[0], z[y][0]);
            z[y][1] = fmaf(sc[0][P], c[1], z[y][1]);
            z[y][2] = fmaf(sc[1][P], c[2], z[y][2]);
            z[y][3] = fmaf(sc[1][P], c[3], z[y][3]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) z[y][i] += __shfl_xor_sync(0xffffffffu, z[y][i], 2);  // the other parity's
        }
        if (ends) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)  // scales of the heads are not negative
            if (row_k + 8 * (i >> 1) >= rows) z[i >> 2][i & 3] = -INFINITY;
        }
        uint32_t vp[NG];
        load_words<NG>(st + lane * Tile::PB, Tile::kVp, vp);
        const float room = room_for(vp);
        // logarithms of the weights; m is raised only where one would pass that, so the
        // exchange between lanes that a maximum takes is seldom needed
        const float bias = s_bias[s];
        float x[2][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i >> 2][i & 3] = fmaf(z[i >> 2][i & 3], zs[i & 1], bias - m[i & 1]);
        float mx[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) mx[c] = fmaxf(fmaxf(x[0][c], x[0][2 + c]), fmaxf(x[1][c], x[1][2 + c]));
        if (__any_sync(0xffffffffu, fmaxf(mx[0], mx[1]) > room)) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mx[c] = fmaxf(fmaxf(z[0][c], z[0][2 + c]), fmaxf(z[1][c], z[1][2 + c]));
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], w));
            const float mn = fmaxf(m[c], fmaf(mx[c], zs[c], bias) + (kRoom - kLift - room));
            const float f = m[c] == mn ? 1.f : fast_exp2(m[c] - mn);
            m[c] = mn;
            l[c] *= f;
            om[c] *= f;
#pragma unroll
            for (int i = 0; i < NP * 2; ++i) {
              o[i][c] *= f;
              o[i][2 + c] *= f;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i >> 2][i & 3] = fmaf(z[i >> 2][i & 3], zs[i & 1], bias - m[i & 1]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t pb[2], pl[2];  // head g, keys of the columns 2 t and 2 t + 1: both terms
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float p0 = fast_exp2(x[y][2 * v]), p1 = fast_exp2(x[y][2 * v + 1]);
            l[0] += p0;
            l[1] += p1;
            const uint32_t rest = pack_rest(p0, p1, &pb[v]);
            pb[v] = transpose8x8(pb[v]);
            pl[v] = transpose8x8(rest);
          }
          uint32_t vw[2][2][NP];  // of keys row_v0 and row_v1: four channels g of both groups of a pair
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int r = 16 * y + 8 * v;
            load_words<NP>(lv0, r * Tile::RB, vw[v][0]);
            load_words<NP>(lv1, r * Tile::RB, vw[v][1]);
          }
          uint32_t mi[2] = {0u, 0u};
          if (g < NG)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const int r = 16 * y + 8 * v;
              mi[v] = __byte_perm(load_word(lvp0 + 4 * g, r * Tile::PB), load_word(lvp1 + 4 * g, r * Tile::PB), 0x7632);
            }
          mma16816_add(om, mi[0], 0u, mi[1], 0u, pb[0], pb[1]);
          mma16816_add(om, mi[0], 0u, mi[1], 0u, pl[0], pl[1]);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int r = 16 * y + 8 * v;
#pragma unroll
            for (int P = 0; P < NP; ++P) {
              const uint32_t w0 = vw[v][0][P], w1 = vw[v][1][P], h0 = w0 >> 8, h1 = w1 >> 8;
              const int at = r * Tile::PB + 8 * P;
              const uint32_t sc = __byte_perm(load_word(lvp0 + par_v, at), load_word(lvp1 + par_v, at), 0x5410);
              uint32_t top;
              const uint32_t low = product_rest(pb[v], pl[v], sc, &top);
              const uint32_t b0 = __byte_perm(top, 0u, sel0), b1 = __byte_perm(top, 0u, sel1);
              const uint32_t c0 = __byte_perm(low, 0u, sel0), c1 = __byte_perm(low, 0u, sel1);
              mma16816_add(o[2 * P], w0 & kLow, w0 & kHigh, w1 & kLow, w1 & kHigh, b0, b1);
              mma16816_add(o[2 * P + 1], h0 & kLow, h0 & kHigh, h1 & kLow, h1 & kHigh, b0, b1);
              mma16816_add(o[2 * P], w0 & kLow, w0 & kHigh, w1 & kLow, w1 & kHigh, c0, c1);
              mma16816_add(o[2 * P + 1], h0 & kLow, h0 & kHigh, h1 & kLow, h1 & kHigh, c0, c1);
            }
          }
        }
      }
    }
    __syncwarp();
    if (turn + S < turns) issue(turn + S, s);
    if (++s == S) {
      s = 0;
      parity ^= 1u;
    }
  }
  // the warp's stages are all read: their memory takes its sums
  if constexpr (ONE) {
    l[0] = warp_sum(l[0]);
#pragma unroll
    for (int k = 0; k < NG; ++k) om[k] = warp_sum(om[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i)  // both terms' sums, of columns c and c + 4
      o[i >> 2][i & 3] += __shfl_xor_sync(0xffffffffu, o[i >> 2][i & 3], 2);
    if (t < NP)  // the columns of groups 2 t and 2 t + 1
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float least = t == 0 ? om[c] : om[2 + c];
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(ring) + 32 * (2 * t + c) + 4 * g) =
            make_float4(fmaf(o[0][c], 0x1p24f, least), fmaf(o[0][2 + c], 0x1p20f, least),
                        fmaf(o[1][c], 0x1p24f, least), fmaf(o[1][2 + c], 0x1p20f, least));
      }
    if (lane == 0) {
      s_m[warp][0] = m[0];
      s_l[warp][0] = l[0];
    }
  } else {
#pragma unroll
    for (int w = 4; w < 32; w <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], w);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], w);
    }
    float least[NP][2];
#pragma unroll
    for (int P = 0; P < NP; ++P)
#pragma unroll
      for (int c = 0; c < 2; ++c) least[P][c] = __shfl_sync(0xffffffffu, om[c], 4 * (2 * P + (t >> 1)) + t);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (hc + c < nh) {
        float* sum = reinterpret_cast<float*>(ring) + (hc + c) * D + 32 * (t >> 1) + 4 * g;
#pragma unroll
        for (int P = 0; P < NP; ++P)
          *reinterpret_cast<float4*>(sum + 64 * P) =
              make_float4(fmaf(o[2 * P][c], 0x1p24f, least[P][c]), fmaf(o[2 * P][2 + c], 0x1p20f, least[P][c]),
                          fmaf(o[2 * P + 1][c], 0x1p24f, least[P][c]), fmaf(o[2 * P + 1][2 + c], 0x1p20f, least[P][c]));
        if (g == 0 && t < 2) {
          s_m[warp][hc + c] = m[c];
          s_l[warp][hc + c] = l[c];
        }
      }
  }
  __syncthreads();
  // the warps' sums as one
  if (a.splits > 1) cluster_wait();  // every CTA of the row has begun
  for (int i = threadIdx.x; i < nh * D; i += kMmaThreads) {
    const int h = i / D;
    float M = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w][h]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = s_m[w][h] == -INFINITY ? 1.f : fast_exp2(s_m[w][h] - M);
      sum += s_l[w][h] * f;
      v += reinterpret_cast<const float*>(smem + w * Tile::kWarp)[i] * f;
    }
    if (s_abort) sum = NAN;  // a wait ran out: the row's results show it, beside the error word
    if (a.splits > 1) {
      send_sum<D>(a, inbox, split, i, v, M, sum);
    } else {
      const size_t row = (size_t)b * p.Hq + h0 + h;
      reinterpret_cast<__nv_bfloat16*>(a.O)[row * D + i % D] = __float2bfloat16_rn(sum == 0.f ? 0.f : v / sum);
      if (i % D == 0) a.LSE[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * GBS_LN2;
    }
  }
  if (a.splits > 1) join_splits<__nv_bfloat16, D>(a, inbox, nh * D, split, (size_t)b * p.Hq + h0);
}

// CTA rows of the tensor-core decode: selection rows, times slices of four heads.
int decode4_rows(const DecodeArgs& a) {
  return a.grouped ? a.p.B * a.p.Hkv * ((a.p.G + 3) / 4) : a.p.B * a.p.Hq;
}

// Splits of every CTA row's n_ent blocks, by a model of the call's time in blocks of a CTA
// that has an SM to itself. A CTA's selection, beginning and end take as long as 36 blocks
// (fp32 queries, whose blocks take four times as long: 6); where four CTAs share an SM,
// their blocks take twice (3 times) as long, and their beginnings and ends count as 12 (2)
// blocks more. The two meet as the root of the sum of squares. Beyond 7/8 of the places, the
// clusters of a row no longer all find places at once, so half a round more is counted.
// Microseconds at 1, 2, 4, 6, 8, 16 splits, the rule's own in brackets:
//   32 rows of 17 blocks    15.4 12.8 11.5 [10.8] 10.8 15.4
//   64 rows of 33, shared   27.9 20.2 16.6 15.5 16.8 34.9, [16.6] at 5
//   128 rows of 33          22.8 18.5 17.7 24.2 26.2 48.5, [17.1] at 3
//   192 rows of 33, shared  34.0 [27.2] 36.6 41.5 46.3 85.2
//   512 rows of 33          [41.3] 49.8 66.8 80.8 102 195
//   102 rows of 49, d = 64  24.9 19.0 15.6 23.4 23.1 36.7, [15.4] at 5
//   128 rows of 17, fp32    31.7 23.4 20.8 26.2 29.5 52.3, [20.3] at 3
int decode4_splits(int rows, int n_ent, int slots, bool fp32) {
  const float ends = fp32 ? 6.f : 36.f, crowd = fp32 ? 3.f : 2.f, more = fp32 ? 2.f : 12.f;
  int best = 1;
  float least = 0.f;
  for (int s = 1; s <= n_ent && s <= kMaxCluster; ++s) {
    const float share = (float)((n_ent + s - 1) / s), load = (float)rows * s / slots;
    const float alone = share + ends, full = (load <= 0.875f ? load : load + 0.5f) * crowd * (share + more);
    const float cost = alone * alone + full * full;
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

// SMs of a device, asked for once.
cudaError_t sm_count(int device, int* sms) {
  static std::atomic<int> known[64];
  if (device < 64 && (*sms = known[device].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  const cudaError_t e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess && device < 64) known[device].store(*sms, std::memory_order_relaxed);
  return e;
}

// One launch: rows x splits CTAs, the splits of a row a cluster.
template <typename T, int D, bool ONE>
cudaError_t launch_decode4(DecodeArgs& a, int device, cudaStream_t st) {
  constexpr bool kMma = sizeof(T) == 2;
  void (*kernel)(DecodeArgs);
  size_t smem;
  if constexpr (kMma) {
    kernel = kv4_decode_mma_kernel<D, ONE>;
    smem = Kv4Tile<D>::kBytes;
  } else {
    kernel = kv4_decode_simt_kernel<T, D>;
    smem = a.sel.idx ? 0 : 4 * (size_t)(a.p.Nb > kSelectWork ? a.p.Nb : kSelectWork);
  }
  a.inbox = (int)((smem + 15) / 16 * 16);
  constexpr int kMost = kMma ? Kv4Tile<D>::kBytes : 4 * (kSelectMax + 4);
  if (a.splits > 1) smem = a.inbox + sizeof(Inbox);
  cudaError_t e;
  static std::atomic<unsigned long long> ready{0};  // devices whose kernel may use large clusters and its memory
  if (device >= 64 || !(ready.load(std::memory_order_acquire) >> device & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost + (int)sizeof(Inbox));
    if (e != cudaSuccess) return e;
    if (device < 64) ready.fetch_or(1ull << device, std::memory_order_release);
  }
  cudaLaunchConfig_t launch{};
  launch.gridDim = dim3(kMma ? decode4_rows(a) : a.p.B * a.p.Hq, a.splits);
  launch.blockDim = dim3(128);
  launch.dynamicSmemBytes = smem;
  launch.stream = st;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = 1;
  cluster.val.clusterDim.y = a.splits;
  cluster.val.clusterDim.z = 1;
  launch.attrs = &cluster;
  launch.numAttrs = a.splits > 1 ? 1 : 0;
  timer_begin(GBS_OP_DECODE, st);
  e = cudaLaunchKernelEx(&launch, kernel, a);
  timer_end(GBS_OP_DECODE, st);
  if (e != cudaSuccess) cudaGetLastError();  // not left for a later launch to find
  else note_launch();
  return e;
}

// ------------------------------------------------------------------ arguments

gbs_status resolve_cache(const Problem& p, const gbs_kv4_cache* in, Kv4* out) {
  if (!in) return fail_status(GBS_ERR_INVALID_ARG, "cache is NULL");
  const void* ptrs[] = {in->kc, in->kp, in->vc, in->vp};
  const char* names[] = {"kc", "kp", "vc", "vp"};
  for (int i = 0; i < 4; ++i) {
    if (!ptrs[i]) return fail_status(GBS_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if ((uintptr_t)ptrs[i] & 15u) return fail_status(GBS_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  if (in->block_table) {
    if (in->max_blocks < p.Nb)
      return fail_status(GBS_ERR_INVALID_ARG, "max_blocks (%d) is below ceil(N / block) = %d", in->max_blocks, p.Nb);
    if (in->num_pages <= 0) return fail_status(GBS_ERR_INVALID_ARG, "num_pages must be positive");
    if ((long long)in->num_pages * p.Hkv > INT32_MAX / 2)  // half blocks are counted in 32 bits
      return fail_status(GBS_ERR_INVALID_ARG, "num_pages * Hkv must be below 2^30");
    if ((uintptr_t)in->block_table & 3u)
      return fail_status(GBS_ERR_INVALID_ARG, "block_table is not 4-byte aligned");
  } else if (in->cap < p.N || in->cap % p.bs) {
    return fail_status(GBS_ERR_INVALID_ARG, "cap (%d) must be a multiple of block and at least N = %d", in->cap, p.N);
  } else if ((long long)p.B * p.Hkv * (in->cap / p.bs) > INT32_MAX / 2) {
    return fail_status(GBS_ERR_INVALID_ARG, "B * Hkv * cap / block must be below 2^30");
  }
  out->kc = static_cast<uint8_t*>(in->kc);
  out->kp = static_cast<uint32_t*>(in->kp);
  out->vc = static_cast<uint8_t*>(in->vc);
  out->vp = static_cast<uint32_t*>(in->vp);
  out->btab = in->block_table;
  out->max_blocks = in->max_blocks;
  out->num_pages = in->num_pages;
  out->cap = in->cap;
  return GBS_OK;
}

gbs_status cuda_done(cudaError_t e, const char* where) {
  return e == cudaSuccess ? GBS_OK : fail_status(GBS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

// Append (READ = false) and read share everything but their kernel.
template <bool READ>
gbs_status rows_call(const char* where, const gbs_params* in, const gbs_kv4_cache* cache, const gbs_heads* K,
                     const gbs_heads* V, int T, const int32_t* start, const int32_t* count, void* ws,
                     void* stream) {
  set_last_error("");
  Problem p{};
  gbs_status s = resolve_kv4_params(in, &p);
  if (s != GBS_OK) return s;
  RowArgs a{};
  if ((s = resolve_cache(p, cache, &a.c)) != GBS_OK) return s;
  const int es = p.dtype == GBS_BF16 ? 2 : 4;
  if ((s = resolve_heads(K, "K", es, false, &a.t[0])) != GBS_OK) return s;
  if ((s = resolve_heads(V, "V", es, false, &a.t[1])) != GBS_OK) return s;
  if (T < 0) return fail_status(GBS_ERR_INVALID_ARG, "T must not be negative");
  if (!start) return fail_status(GBS_ERR_INVALID_ARG, "start is NULL");
  if (((uintptr_t)start | (uintptr_t)count) & 3u)
    return fail_status(GBS_ERR_INVALID_ARG, "start or count is not 4-byte aligned");
  if ((uintptr_t)ws & 255u) return fail_status(GBS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  const long long rows = (long long)p.B * p.Hkv * T;
  if (rows > INT32_MAX) return fail_status(GBS_ERR_INVALID_ARG, "problem too large: B * Hkv * T must be below 2^31");
  if (rows == 0) return GBS_OK;
  if (READ && share_memory(a.t[0], p.Hkv, a.t[1], p.Hkv, p.B, T, p.d, es))
    return fail_status(GBS_ERR_INVALID_ARG, "K and V share memory");
  a.B = p.B; a.Hkv = p.Hkv; a.T = T; a.N = p.N;
  a.start = start; a.count = count;
  a.c.err = static_cast<unsigned int*>(ws);
  const int rows_per_cta = 256 / (p.d / 32);
  const dim3 grid((unsigned)((rows + rows_per_cta - 1) / rows_per_cta), 2);
  cudaStream_t st = (cudaStream_t)stream;
#define GBS_ROWS(T_, D_)                                       \
  do {                                                         \
    if (READ) kv4_read_kernel<T_, D_><<<grid, 256, 0, st>>>(a); \
    else kv4_append_kernel<T_, D_><<<grid, 256, 0, st>>>(a);   \
  } while (0)
  if (p.dtype == GBS_BF16) {
    if (p.d == 64) GBS_ROWS(__nv_bfloat16, 64);
    else GBS_ROWS(__nv_bfloat16, 128);
  } else {
    if (p.d == 64) GBS_ROWS(float, 64);
    else GBS_ROWS(float, 128);
  }
#undef GBS_ROWS
  note_launch();
  return cuda_done(cudaGetLastError(), where);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The error word and, for rows too long for the decode to select from, the lists.
size_t carve_kv4(const Problem& p, char* base, DecodeArgs* a) {
  size_t off = 256;
  if ((p.N - 1) / p.bs <= kSelectMax) return off;
  const size_t rows = (size_t)p.B * p.Hq;
  auto take = [&](size_t bytes) {
    char* at = base + off;
    off += up256(bytes);
    return at;
  };
  a->sel.idx = reinterpret_cast<int32_t*>(take(rows * p.topk * 4));
  a->sel.cnt = reinterpret_cast<int32_t*>(take(rows * 4));
  a->sel.logg = reinterpret_cast<float*>(take(rows * p.topk * 4));
  return off;
}

}  // namespace
}  // namespace gbs

using namespace gbs;

extern "C" gbs_status gbs_kv4_append(const gbs_params* p, const gbs_kv4_cache* cache, const gbs_heads* K,
                                     const gbs_heads* V, int T, const int32_t* start, const int32_t* count,
                                     void* ws, void* stream) {
  return rows_call<false>("gbs_kv4_append", p, cache, K, V, T, start, count, ws, stream);
}

extern "C" gbs_status gbs_kv4_read(const gbs_params* p, const gbs_kv4_cache* cache, const gbs_heads* K,
                                   const gbs_heads* V, int T, const int32_t* start, const int32_t* count,
                                   void* ws, void* stream) {
  return rows_call<true>("gbs_kv4_read", p, cache, K, V, T, start, count, ws, stream);
}

extern "C" size_t gbs_kv4_workspace_bytes(const gbs_params* in) {
  set_last_error("");
  Problem p{};
  if (resolve_kv4_params(in, &p) != GBS_OK) return 0;
  DecodeArgs a{};
  return carve_kv4(p, nullptr, &a);
}

extern "C" gbs_status gbs_kv4_decode(const gbs_params* in, const gbs_kv4_cache* cache, const int32_t* seq_lens,
                                     int group_shared, const void* q, const float* S, void* O, float* LSE,
                                     int num_splits, void* ws, size_t ws_bytes, void* stream) {
  set_last_error("");
  DecodeArgs a{};
  Problem& p = a.p;
  gbs_status s = resolve_kv4_params(in, &p);
  if (s != GBS_OK) return s;
  if ((s = resolve_cache(p, cache, &a.c)) != GBS_OK) return s;
  const void* ptrs[] = {q, S, O, LSE};
  const char* names[] = {"q", "S", "O", "LSE"};
  for (int i = 0; i < 4; ++i) {
    if (!ptrs[i]) return fail_status(GBS_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if ((uintptr_t)ptrs[i] & 15u) return fail_status(GBS_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  if (num_splits < 0 || num_splits > kMaxDecodeSplits)
    return fail_status(GBS_ERR_INVALID_ARG, "num_splits %d outside [0, %d]", num_splits, kMaxDecodeSplits);
  if (group_shared != 0 && group_shared != 1) return fail_status(GBS_ERR_INVALID_ARG, "group_shared must be 0 or 1");
  if ((uintptr_t)seq_lens & 3u) return fail_status(GBS_ERR_INVALID_ARG, "seq_lens is not 4-byte aligned");
  const size_t need = carve_kv4(p, static_cast<char*>(ws), &a);
  if (!ws) return fail_status(GBS_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
  if ((uintptr_t)ws & 255u) return fail_status(GBS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < need) return fail_status(GBS_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  a.c.err = static_cast<unsigned int*>(ws);
  a.seq_lens = seq_lens;
  a.q = q; a.O = O; a.LSE = LSE;
  a.grouped = group_shared;
  cudaStream_t st = (cudaStream_t)stream;
  const int cur_max = (p.N - 1) / p.bs;
  SeqLens seq;
  seq.lens = seq_lens;
  seq.rows_per_seq = group_shared ? p.Hkv : p.Hq;
  seq.max_len = p.N;
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = sm_count(device, &sms);
  if (e != cudaSuccess) return cuda_done(e, "gbs_kv4_decode/device");
  a.S = S;
  if (cur_max > kSelectMax) {
    e = launch_select(S, p.B * seq.rows_per_seq, p.Nb, 1, seq_lens ? -1 : cur_max, p.topk, p.mode, p.log_tau, a.sel.idx,
                      a.sel.cnt, a.sel.logg, nullptr, st, nullptr, nullptr, 0, seq);
    if (e != cudaSuccess) return cuda_done(e, "gbs_kv4_decode/select");
  }
  const int n_ent = (p.topk < cur_max ? p.topk : cur_max) + 1;
  a.splits = num_splits;
  if (a.splits == 0) a.splits = decode4_splits(p.dtype == GBS_BF16 ? decode4_rows(a) : p.B * p.Hq, n_ent, 4 * sms, p.dtype != GBS_BF16);
  if (a.splits > n_ent) a.splits = n_ent;
  if (a.splits > kMaxCluster) a.splits = kMaxCluster;
  cudaError_t (*launch)(DecodeArgs&, int, cudaStream_t);
  if (p.dtype != GBS_BF16) launch = p.d == 64 ? launch_decode4<float, 64, true> : launch_decode4<float, 128, true>;
  else if (!a.grouped || p.G == 1) launch = p.d == 64 ? launch_decode4<__nv_bfloat16, 64, true> : launch_decode4<__nv_bfloat16, 128, true>;
  else launch = p.d == 64 ? launch_decode4<__nv_bfloat16, 64, false> : launch_decode4<__nv_bfloat16, 128, false>;
  e = launch(a, device, st);
  return cuda_done(e, "gbs_kv4_decode");
}
