// qkv_rope.cu — norms of queries and keys for each head and rotary positions in
// one pass, from a projection's layout to the attention's, and the backward.
//
// One row (token, head) of d channels is held by d / 8 lanes, eight channels to
// a lane: four and their rotation partners, so that a pair never leaves its lane
// (halves: channels 4 l .. 4 l + 3 and rot / 2 + 4 l ..; neighbours, and channels
// that are not rotated: 8 l .. 8 l + 7). The norm's sums go over the row's lanes
// by shuffles. A row is read once and written once, and the cos and sin of a
// token stay in registers for all of its heads, so the pass is bound by memory. A
// CTA works on one tensor: its 16 lane groups (d = 128) walk along the heads of 16
// adjacent tokens, which is 8 KB in a row in the projection for each group (32 heads)
// and 4 KB in a row in every head's plane for all of them; with four groups to a token
// the forward took 342 us instead of 305.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gbs {
namespace {

using namespace sm100;  // f32x2

constexpr int kThreads = 256;
// Rows whose loads a lane group has in flight before any arithmetic. Two, with the
// registers held to four (backward: three) CTAs an SM and the lines of the next two asked
// for in L2, measured best: forward of 65536 tokens (32 + 16 heads, d = 128, bf16) 272 us
// (5.9 TB/s) against 312 without the prefetch, 299 with one four rounds ahead, and 342
// with eight rows in flight and two CTAs; backward of 8192 tokens 70 us against 80 without.
constexpr int kRows = 2;

struct RopeArgs {
  int B, N, Hq, Hkv, half, interleaved, n_axes, max_pos, norm, w_bf16;
  int per_token[2];  // lane groups that share a token's heads: of q; of k and v
  int ctas[3];       // CTAs of q, k, v, in this order
  float eps;
  const void *wq, *wk;
  const float *cos_tab, *sin_tab;
  const int32_t* pos;
  Heads in[3], out[3];  // q, k, v and what becomes of them (backward: dQ, dK, dV -> dq, dk, dv)
  Heads x[2];           // backward: q, k
  float* part;          // backward: [CTAs of q and k][d] partial sums of dwq, dwk
  unsigned int* err;
  alignas(4) unsigned char axis[64];
};

// Eight channels of a lane as two vectors of first (p) and second (r) members of four
// pairs, in packed fp32 pairs (two lanes of arithmetic an instruction).
struct Pairs {
  f32x2 p[2], r[2];
};

template <typename T> struct Quad;  // four channels as one load
template <> struct Quad<float> {
  using type = float4;
  static __device__ __forceinline__ type ones() { return make_float4(1.f, 1.f, 1.f, 1.f); }
};
template <> struct Quad<__nv_bfloat16> {
  using type = uint2;
  static __device__ __forceinline__ type ones() { return make_uint2(0x3f803f80u, 0x3f803f80u); }
};

__device__ __forceinline__ f32x2 make2(uint32_t lo, uint32_t hi) {
  return f2_make(__uint_as_float(lo), __uint_as_float(hi));
}
// INTER: pairs are neighbours; else pair i is (a[i], b[i]).
template <bool INTER>
__device__ __forceinline__ Pairs widen(const float4& a, const float4& b) {
  if (INTER) return {{f2_make(a.x, a.z), f2_make(b.x, b.z)}, {f2_make(a.y, a.w), f2_make(b.y, b.w)}};
  return {{f2_make(a.x, a.y), f2_make(a.z, a.w)}, {f2_make(b.x, b.y), f2_make(b.z, b.w)}};
}
template <bool INTER>
__device__ __forceinline__ Pairs widen(const uint2& a, const uint2& b) {
  constexpr uint32_t H = 0xffff0000u;
  if (INTER)
    return {{make2(a.x << 16, a.y << 16), make2(b.x << 16, b.y << 16)}, {make2(a.x & H, a.y & H), make2(b.x & H, b.y & H)}};
  return {{make2(a.x << 16, a.x & H), make2(a.y << 16, a.y & H)}, {make2(b.x << 16, b.x & H), make2(b.y << 16, b.y & H)}};
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool INTER>
__device__ __forceinline__ void narrow(const Pairs& v, float4* a, float4* b) {
  float p[4], r[4];
  f2_split(v.p[0], p[0], p[1]); f2_split(v.p[1], p[2], p[3]);
  f2_split(v.r[0], r[0], r[1]); f2_split(v.r[1], r[2], r[3]);
  *a = INTER ? make_float4(p[0], r[0], p[1], r[1]) : make_float4(p[0], p[1], p[2], p[3]);
  *b = INTER ? make_float4(p[2], r[2], p[3], r[3]) : make_float4(r[0], r[1], r[2], r[3]);
}
template <bool INTER>
__device__ __forceinline__ void narrow(const Pairs& v, uint2* a, uint2* b) {
  float4 x, y;
  narrow<INTER>(v, &x, &y);
  *a = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
  *b = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
}
// sum of the products of all channels
__device__ __forceinline__ float dot(const Pairs& x, const Pairs& y) {
  const f32x2 s = f2_fma(x.r[1], y.r[1], f2_fma(x.r[0], y.r[0], f2_fma(x.p[1], y.p[1], f2_mul(x.p[0], y.p[0]))));
  float lo, hi;
  f2_split(s, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ Pairs times(const Pairs& x, const Pairs& y) {
  return {{f2_mul(x.p[0], y.p[0]), f2_mul(x.p[1], y.p[1])}, {f2_mul(x.r[0], y.r[0]), f2_mul(x.r[1], y.r[1])}};
}
__device__ __forceinline__ Pairs times(const Pairs& x, float f) {
  const f32x2 y = f2_make(f, f);
  return {{f2_mul(x.p[0], y), f2_mul(x.p[1], y)}, {f2_mul(x.r[0], y), f2_mul(x.r[1], y)}};
}
// x y + z and f x + z
__device__ __forceinline__ Pairs fma(const Pairs& x, const Pairs& y, const Pairs& z) {
  return {{f2_fma(x.p[0], y.p[0], z.p[0]), f2_fma(x.p[1], y.p[1], z.p[1])},
          {f2_fma(x.r[0], y.r[0], z.r[0]), f2_fma(x.r[1], y.r[1], z.r[1])}};
}
__device__ __forceinline__ Pairs fma(float f, const Pairs& x, const Pairs& z) {
  const f32x2 y = f2_make(f, f);
  return {{f2_fma(x.p[0], y, z.p[0]), f2_fma(x.p[1], y, z.p[1])}, {f2_fma(x.r[0], y, z.r[0]), f2_fma(x.r[1], y, z.r[1])}};
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(x): of fp32 rows rounded to nearest, as their results keep all of its bits.
template <typename T>
__device__ __forceinline__ float inv_root(float x) {
  return sizeof(T) == 4 ? __frsqrt_rn(x) : rsqrtf(x);
}

// What a lane keeps of its token: the angles of its four pairs, sin with either sign.
struct Angles {
  f32x2 c[2], s[2], minus_s[2];
};

__device__ __forceinline__ int table_row(const RopeArgs& a, long long token, int axis) {
  int p = __ldg(a.pos + token * a.n_axes + axis);
  if (p < 0 || p >= a.max_pos) {
    set_error(a.err, GBS_ERR_INVALID_ARG);
    p = p < 0 ? 0 : a.max_pos - 1;
  }
  return p;
}

// axes: the axes of the lane's four pairs, a byte each. Called for lanes that rotate.
__device__ __forceinline__ Angles load_angles(const RopeArgs& a, long long token, int lane, uint32_t axes) {
  float4 c, s;
  const int i0 = 4 * lane;
  if (axes == (axes & 0xffu) * 0x01010101u) {
    const size_t at = (size_t)table_row(a, token, axes & 0xffu) * a.half + i0;
    c = __ldg(reinterpret_cast<const float4*>(a.cos_tab + at));
    s = __ldg(reinterpret_cast<const float4*>(a.sin_tab + at));
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t at = (size_t)table_row(a, token, axes >> (8 * i) & 0xffu) * a.half + i0 + i;
      v[i] = __ldg(a.cos_tab + at);
      v[4 + i] = __ldg(a.sin_tab + at);
    }
    c = make_float4(v[0], v[1], v[2], v[3]);
    s = make_float4(v[4], v[5], v[6], v[7]);
  }
  return {{f2_make(c.x, c.y), f2_make(c.z, c.w)}, {f2_make(s.x, s.y), f2_make(s.z, s.w)},
          {f2_make(-s.x, -s.y), f2_make(-s.z, -s.w)}};
}

// Rotates by the angles (BACK: by their negatives).
template <bool BACK>
__device__ __forceinline__ void rotate(Pairs& v, const Angles& t) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 p = v.p[i], r = v.r[i];
    v.p[i] = f2_fma(r, BACK ? t.s[i] : t.minus_s[i], f2_mul(p, t.c[i]));
    v.r[i] = f2_fma(p, BACK ? t.minus_s[i] : t.s[i], f2_mul(r, t.c[i]));
  }
}

__device__ __forceinline__ bool lane_rotates(const RopeArgs& a, int lane) { return 4 * lane < a.half; }
__device__ __forceinline__ uint32_t lane_axes(const RopeArgs& a, int lane) {
  return lane_rotates(a, lane) ? *reinterpret_cast<const uint32_t*>(a.axis + 4 * lane) : 0u;
}

// Asks for the lines of a row that is loaded a little later.
template <typename T, int D>
__device__ __forceinline__ void prefetch_row(const T* row, int lane, bool there) {
  constexpr int kLines = D * (int)sizeof(T) / 128;
  if (there && lane < kLines) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + lane * (128 / (int)sizeof(T))));
}

// First channels of a lane's two quads.
template <bool INTER>
__device__ __forceinline__ void quad_offsets(const RopeArgs& a, int lane, int* off) {
  const bool apart = !INTER && lane_rotates(a, lane);
  off[0] = apart ? 4 * lane : 8 * lane;
  off[1] = apart ? a.half + 4 * lane : 8 * lane + 4;
}

template <bool INTER>
__device__ __forceinline__ Pairs load_weights(const RopeArgs& a, const void* w, const int* off) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = off[i >> 2] + (i & 3);
    v[i] = !w ? 1.f
              : (a.w_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[c])
                          : reinterpret_cast<const float*>(w)[c]);
  }
  return widen<INTER>(make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7]));
}

// Which of the three tensors a CTA works on, its place among that tensor's CTAs, and their number.
struct Role {
  int which, index, count, per_token;
};
__device__ __forceinline__ Role cta_role(const RopeArgs& a) {
  int x = blockIdx.x;
  if (x < a.ctas[0]) return {0, x, a.ctas[0], a.per_token[0]};
  x -= a.ctas[0];
  if (x < a.ctas[1]) return {1, x, a.ctas[1], a.per_token[1]};
  return {2, x - a.ctas[1], a.ctas[2], a.per_token[1]};
}

// One of the three tensors of a token: heads h = sub, sub + per_token, ...
// WHICH: 0 = q, 1 = k (norm and rotation), 2 = v (moved).
template <typename T, int D, int WHICH, bool INTER>
__device__ __forceinline__ void forward_tensor(const RopeArgs& a, const Role& role) {
  using Q4 = typename Quad<T>::type;
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, sub = group % role.per_token;
  const long long token = (long long)role.index * (GROUPS / role.per_token) + group / role.per_token;
  const bool valid = token < (long long)a.B * a.N;
  const int b = valid ? (int)token / a.N : 0, n = valid ? (int)token - b * a.N : 0;
  int off[2] = {8 * lane, 8 * lane + 4};
  if (WHICH < 2) quad_offsets<INTER>(a, lane, off);
  const int H = valid ? (WHICH == 0 ? a.Hq : a.Hkv) : 0;
  const long long in_step = role.per_token * a.in[WHICH].sh, out_step = role.per_token * a.out[WHICH].sh;
  const T* src = reinterpret_cast<const T*>(a.in[WHICH].ptr) + b * a.in[WHICH].sb + n * a.in[WHICH].sn + sub * a.in[WHICH].sh;
  T* dst = reinterpret_cast<T*>(a.out[WHICH].ptr) + b * a.out[WHICH].sb + n * a.out[WHICH].sn + sub * a.out[WHICH].sh;
  const int rounds = ((WHICH == 0 ? a.Hq : a.Hkv) + role.per_token * kRows - 1) / (role.per_token * kRows);
  const bool rotates = WHICH < 2 && lane_rotates(a, lane);
  Angles ang;
  Pairs w;
  for (int it = 0, h = sub; it < rounds; ++it) {
    Q4 raw[kRows][2];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      raw[u][0] = raw[u][1] = Q4{};
      if (h + u * role.per_token < H) {
        raw[u][0] = __ldg(reinterpret_cast<const Q4*>(src + off[0]));
        raw[u][1] = __ldg(reinterpret_cast<const Q4*>(src + off[1]));
      }
      prefetch_row<T, D>(src + kRows * in_step, lane, h + (u + kRows) * role.per_token < H);
      src += in_step;
    }
    if (WHICH < 2 && it == 0) {  // behind the rows' loads, which need not wait for the position
      if (rotates) ang = load_angles(a, valid ? token : 0, lane, lane_axes(a, lane));
      w = load_weights<INTER>(a, WHICH == 0 ? a.wq : a.wk, off);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u, h += role.per_token) {
      if (WHICH < 2) {
        Pairs v = widen<INTER>(raw[u][0], raw[u][1]);
        if (a.norm) v = times(v, times(w, inv_root<T>(row_sum<LANES>(dot(v, v)) * (1.f / D) + a.eps)));
        if (rotates) rotate<false>(v, ang);
        narrow<INTER>(v, &raw[u][0], &raw[u][1]);
      }
      if (h < H) {
        *reinterpret_cast<Q4*>(dst + off[0]) = raw[u][0];
        *reinterpret_cast<Q4*>(dst + off[1]) = raw[u][1];
      }
      dst += out_step;
    }
  }
}

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
  const Role r = cta_role(a);
  if (r.which == 0) forward_tensor<T, D, 0, INTER>(a, r);
  else if (r.which == 1) forward_tensor<T, D, 1, INTER>(a, r);
  else forward_tensor<T, D, 2, INTER>(a, r);
}

// dx from x and dz, and this lane's share of dw.
template <typename T, int D, int WHICH, bool INTER>
__device__ __forceinline__ void backward_tensor(const RopeArgs& a, const Role& role) {
  using Q4 = typename Quad<T>::type;
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, sub = group % role.per_token;
  const int tokens_per_cta = GROUPS / role.per_token;
  const long long tokens = (long long)a.B * a.N;
  int off[2] = {8 * lane, 8 * lane + 4};
  const f32x2 zero = f2_make(0.f, 0.f);
  Pairs w, dw = {{zero, zero}, {zero, zero}};
  const uint32_t axes = lane_axes(a, lane);
  const bool rotates = WHICH < 2 && lane_rotates(a, lane);
  if (WHICH < 2) {
    quad_offsets<INTER>(a, lane, off);
    w = load_weights<INTER>(a, WHICH == 0 ? a.wq : a.wk, off);
  }
  const Heads& tx = a.x[WHICH < 2 ? WHICH : 0];
  const long long in_step = role.per_token * a.in[WHICH].sh, out_step = role.per_token * a.out[WHICH].sh;
  const long long x_step = role.per_token * tx.sh;
  const int rounds = ((WHICH == 0 ? a.Hq : a.Hkv) + role.per_token * kRows - 1) / (role.per_token * kRows);
  // a CTA takes every count-th run of tokens, so that few partial sums of dw are left
  for (long long first = (long long)role.index * tokens_per_cta; first < tokens; first += (long long)role.count * tokens_per_cta) {
    const long long token = first + group / role.per_token;
    const bool valid = token < tokens;
    const int b = valid ? (int)token / a.N : 0, n = valid ? (int)token - b * a.N : 0;
    const int H = valid ? (WHICH == 0 ? a.Hq : a.Hkv) : 0;
    const T* dz = reinterpret_cast<const T*>(a.in[WHICH].ptr) + b * a.in[WHICH].sb + n * a.in[WHICH].sn + sub * a.in[WHICH].sh;
    const T* x = reinterpret_cast<const T*>(tx.ptr) + b * tx.sb + n * tx.sn + sub * tx.sh;
    T* dx = reinterpret_cast<T*>(a.out[WHICH].ptr) + b * a.out[WHICH].sb + n * a.out[WHICH].sn + sub * a.out[WHICH].sh;
    Angles ang;
    for (int it = 0, h = sub; it < rounds; ++it) {
      Q4 rz[kRows][2], rx[kRows][2];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        rz[u][0] = rz[u][1] = Q4{};
        rx[u][0] = rx[u][1] = Quad<T>::ones();  // a row that is not there: r has to be finite with eps = 0
        if (h + u * role.per_token < H) {
          rz[u][0] = __ldg(reinterpret_cast<const Q4*>(dz + off[0]));
          rz[u][1] = __ldg(reinterpret_cast<const Q4*>(dz + off[1]));
          if (WHICH < 2 && a.norm) {
            rx[u][0] = __ldg(reinterpret_cast<const Q4*>(x + off[0]));
            rx[u][1] = __ldg(reinterpret_cast<const Q4*>(x + off[1]));
          }
        }
        const bool next = h + (u + kRows) * role.per_token < H;
        prefetch_row<T, D>(dz + kRows * in_step, lane, next);
        if (WHICH < 2) prefetch_row<T, D>(x + kRows * x_step, lane, next && a.norm);
        dz += in_step;
        x += x_step;
      }
      // (a token that is not there counts as zeros: its angles only have to be finite)
      if (it == 0 && rotates) ang = load_angles(a, valid ? token : 0, lane, axes);
#pragma unroll
      for (int u = 0; u < kRows; ++u, h += role.per_token) {
        if (WHICH < 2) {
          Pairs g = widen<INTER>(rz[u][0], rz[u][1]);
          if (rotates) rotate<true>(g, ang);
          if (a.norm) {
            const Pairs v = widen<INTER>(rx[u][0], rx[u][1]), hw = times(g, w);
            const float r = inv_root<T>(row_sum<LANES>(dot(v, v)) * (1.f / D) + a.eps);
            // mean(h xh) xh = x r^2 mean(h x)
            const float back = row_sum<LANES>(dot(hw, v)) * (1.f / D) * r * r;
            dw = fma(times(g, r), v, dw);  // rows left out have g = 0
            g = times(fma(-back, v, hw), r);
          }
          narrow<INTER>(g, &rz[u][0], &rz[u][1]);
        }
        if (h < H) {
          *reinterpret_cast<Q4*>(dx + off[0]) = rz[u][0];
          *reinterpret_cast<Q4*>(dx + off[1]) = rz[u][1];
        }
        dx += out_step;
      }
    }
  }
  if constexpr (WHICH < 2) {
    if (!a.norm) return;
    __shared__ float sums[GROUPS][D];
    float4 lo, hi;
    narrow<INTER>(dw, &lo, &hi);
    *reinterpret_cast<float4*>(&sums[group][off[0]]) = lo;
    *reinterpret_cast<float4*>(&sums[group][off[1]]) = hi;
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kThreads) {
      float s = 0.f;
      for (int g = 0; g < GROUPS; ++g) s += sums[g][c];
      a.part[(size_t)blockIdx.x * D + c] = s;
    }
  }
}

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  const Role r = cta_role(a);
  if (r.which == 0) backward_tensor<T, D, 0, INTER>(a, r);
  else if (r.which == 1) backward_tensor<T, D, 1, INTER>(a, r);
  else backward_tensor<T, D, 2, INTER>(a, r);
}

// dw[c] = sum of the CTAs' partial sums, in a fixed order: blockIdx.y 0 for q, 1 for k.
__global__ void __launch_bounds__(1024)
rope_dw_kernel(const float* __restrict__ part, int n_q, int n_k, int d, float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float s_sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  const int begin = blockIdx.y ? n_q : 0, end = blockIdx.y ? n_q + n_k : n_q;
  float s = 0.f;
#pragma unroll 8
  for (int r = begin + warp; r < end; r += 32) s += part[(size_t)r * d + col];
  s_sum[warp][lane] = s;
  __syncthreads();
  const float v = warp_sum(s_sum[lane][warp]);  // warp w: column w of the 32
  if (lane == 0) (blockIdx.y ? dwk : dwq)[blockIdx.x * 32 + warp] = v;
}

gbs_status resolve_rope(const gbs_rope_params* in, RopeArgs* a) {
  if (!in) return fail_status(GBS_ERR_INVALID_ARG, "params is NULL");
  const gbs_rope_params& p = *in;
  if (p.B <= 0 || p.N <= 0 || p.Hq <= 0 || p.Hkv <= 0)
    return fail_status(GBS_ERR_INVALID_ARG, "B, N, Hq and Hkv must be positive");
  if (p.d != 64 && p.d != 128) return fail_status(GBS_ERR_UNSUPPORTED, "d %d: only 64 and 128 are built", p.d);
  if (p.rot < 0 || p.rot > p.d || p.rot % 8)
    return fail_status(GBS_ERR_INVALID_ARG, "rot %d must be a multiple of 8 in [0, d = %d]", p.rot, p.d);
  if (p.interleaved != 0 && p.interleaved != 1)
    return fail_status(GBS_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (p.dtype != GBS_BF16 && p.dtype != GBS_F32) return fail_status(GBS_ERR_INVALID_ARG, "dtype %d unknown", p.dtype);
  if (p.w_dtype != GBS_BF16 && p.w_dtype != GBS_F32)
    return fail_status(GBS_ERR_INVALID_ARG, "w_dtype %d unknown", p.w_dtype);
  if (!(p.eps >= 0.f) || isinf(p.eps)) return fail_status(GBS_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (p.n_axes < 1 || p.n_axes > 4) return fail_status(GBS_ERR_INVALID_ARG, "n_axes %d outside [1, 4]", p.n_axes);
  if (p.rot && p.max_pos < 1) return fail_status(GBS_ERR_INVALID_ARG, "max_pos must be positive");
  for (int i = 0; i < p.rot / 2; ++i)
    if (p.axis[i] >= p.n_axes)
      return fail_status(GBS_ERR_INVALID_ARG, "axis[%d] = %d is not below n_axes = %d", i, (int)p.axis[i], p.n_axes);
  if ((long long)p.B * p.N > INT32_MAX / 4 || p.Hq > 65536 || p.Hkv > 65536)
    return fail_status(GBS_ERR_INVALID_ARG, "problem too large: B * N must be below 2^29 and heads at most 65536");
  *a = RopeArgs{};
  a->B = p.B; a->N = p.N; a->Hq = p.Hq; a->Hkv = p.Hkv;
  a->half = p.rot / 2; a->interleaved = p.interleaved; a->n_axes = p.n_axes;
  a->max_pos = p.max_pos; a->eps = p.eps; a->w_bf16 = p.w_dtype == GBS_BF16;
  memcpy(a->axis, p.axis, sizeof(a->axis));
  return GBS_OK;
}

gbs_status check_side(const RopeArgs& a, const void* wq, const void* wk, const float* cos_tab,
                      const float* sin_tab, const int32_t* pos) {
  if (!wq != !wk) return fail_status(GBS_ERR_INVALID_ARG, "give both weights or neither");
  if (((uintptr_t)wq | (uintptr_t)wk) & (a.w_bf16 ? 1u : 3u))
    return fail_status(GBS_ERR_INVALID_ARG, "a weight is not aligned to its elements");
  if (a.half && (!cos_tab || !sin_tab || !pos))
    return fail_status(GBS_ERR_INVALID_ARG, "cos_tab, sin_tab or pos is NULL");
  if (((uintptr_t)cos_tab | (uintptr_t)sin_tab) & 15u)
    return fail_status(GBS_ERR_INVALID_ARG, "cos_tab or sin_tab is not 16-byte aligned");
  if ((uintptr_t)pos & 3u) return fail_status(GBS_ERR_INVALID_ARG, "pos is not 4-byte aligned");
  return GBS_OK;
}

// That no output shares memory with an input or another output: in (n_in of them, heads[i] each)
// and out, of which the pointers that are null are left out.
gbs_status check_apart(const gbs_rope_params& p, int n_in, const Heads* in, const int* in_heads, const char* const* in_names,
                       const Heads* out, const char* const* out_names) {
  const int es = p.dtype == GBS_BF16 ? 2 : 4, out_heads[] = {p.Hq, p.Hkv, p.Hkv};
  for (int o = 0; o < 3; ++o) {
    if (!out[o].ptr) continue;
    for (int i = 0; i < n_in; ++i)
      if (in[i].ptr && share_memory(out[o], out_heads[o], in[i], in_heads[i], p.B, p.N, p.d, es))
        return fail_status(GBS_ERR_INVALID_ARG, "%s and %s share memory", in_names[i], out_names[o]);
    for (int i = 0; i < o; ++i)
      if (out[i].ptr && share_memory(out[o], out_heads[o], out[i], out_heads[i], p.B, p.N, p.d, es))
        return fail_status(GBS_ERR_INVALID_ARG, "%s and %s share memory", out_names[i], out_names[o]);
  }
  return GBS_OK;
}

constexpr int kSms = 148;
constexpr int kMaxBwdCtas = 512;  // of a tensor

// Lane groups that share a token's heads (a power of two): one while there are tokens
// enough to fill the GPU, so that a group walks along a token's heads and the groups of
// a CTA meet in adjacent rows of every head.
int groups_per_token(long long tokens, int heads, int groups) {
  int g = 1;
  while (g < groups && g < heads && tokens * g / groups < kSms) g *= 2;
  return g;
}

template <typename T>
cudaError_t launch_rope(RopeArgs& a, int d, bool backward, float* dwq, float* dwk, cudaStream_t st) {
  const int groups = kThreads / (d / 8);
  const long long tokens = (long long)a.B * a.N;
  const int heads[3] = {a.Hq, a.Hkv, a.in[2].ptr ? a.Hkv : 0};
  for (int i = 0; i < 2; ++i) a.per_token[i] = groups_per_token(tokens, heads[i], groups);
  for (int i = 0; i < 3; ++i) {
    const int tokens_per_cta = groups / a.per_token[i ? 1 : 0];
    long long n = heads[i] ? (tokens + tokens_per_cta - 1) / tokens_per_cta : 0;
    // the backward's CTAs take equal numbers of runs of tokens, so that at most kMaxBwdCtas
    // partial sums of dw are left
    const long long runs = (n + kMaxBwdCtas - 1) / kMaxBwdCtas;
    a.ctas[i] = (int)(backward && n ? (n + runs - 1) / runs : n);
  }
  const unsigned grid = (unsigned)(a.ctas[0] + a.ctas[1] + a.ctas[2]);
  void (*const fwd[])(RopeArgs) = {rope_fwd_kernel<T, 64, false>, rope_fwd_kernel<T, 64, true>,
                                   rope_fwd_kernel<T, 128, false>, rope_fwd_kernel<T, 128, true>};
  void (*const bwd[])(RopeArgs) = {rope_bwd_kernel<T, 64, false>, rope_bwd_kernel<T, 64, true>,
                                   rope_bwd_kernel<T, 128, false>, rope_bwd_kernel<T, 128, true>};
  const int kind = (d == 128 ? 2 : 0) + a.interleaved;
  (backward ? bwd : fwd)[kind]<<<grid, kThreads, 0, st>>>(a);
  note_launch();
  if (!backward) return cudaGetLastError();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.norm) return e;
  rope_dw_kernel<<<dim3(d / 32, 2), 1024, 0, st>>>(a.part, a.ctas[0], a.ctas[1], d, dwq, dwk);
  note_launch();
  return cudaGetLastError();
}

gbs_status done(cudaError_t e, const char* where) {
  return e == cudaSuccess ? GBS_OK : fail_status(GBS_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

}  // namespace
}  // namespace gbs

using namespace gbs;

extern "C" size_t gbs_qkv_rope_workspace_bytes(const gbs_rope_params* p) {
  set_last_error("");
  RopeArgs a;
  if (resolve_rope(p, &a) != GBS_OK) return 0;
  return 256 + (size_t)2 * kMaxBwdCtas * p->d * sizeof(float);
}

extern "C" gbs_status gbs_qkv_rope_fwd(const gbs_rope_params* p, const gbs_heads* q, const gbs_heads* k,
                                       const gbs_heads* v, const void* wq, const void* wk,
                                       const float* cos_tab, const float* sin_tab, const int32_t* pos,
                                       const gbs_heads* Q, const gbs_heads* K, const gbs_heads* V, void* ws,
                                       void* stream) {
  set_last_error("");
  RopeArgs a;
  gbs_status s = resolve_rope(p, &a);
  if (s != GBS_OK) return s;
  const int es = p->dtype == GBS_BF16 ? 2 : 4;
  if (!v != !V) return fail_status(GBS_ERR_INVALID_ARG, "give both v and V or neither");
  const gbs_heads* in[] = {q, k, v};
  const gbs_heads* out[] = {Q, K, V};
  const char* names[] = {"q", "k", "v", "Q", "K", "V"};
  for (int i = 0; i < 3; ++i) {
    if ((s = resolve_heads(in[i], names[i], es, i == 2, &a.in[i])) != GBS_OK) return s;
    if ((s = resolve_heads(out[i], names[3 + i], es, i == 2, &a.out[i])) != GBS_OK) return s;
  }
  if ((s = check_side(a, wq, wk, cos_tab, sin_tab, pos)) != GBS_OK) return s;
  if ((uintptr_t)ws & 255u) return fail_status(GBS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  const int in_heads[] = {p->Hq, p->Hkv, p->Hkv};
  if ((s = check_apart(*p, 3, a.in, in_heads, names, a.out, names + 3)) != GBS_OK) return s;
  a.wq = wq; a.wk = wk; a.norm = wq != nullptr;
  a.cos_tab = cos_tab; a.sin_tab = sin_tab; a.pos = pos;
  a.err = static_cast<unsigned int*>(ws);
  cudaStream_t st = (cudaStream_t)stream;
  return done(p->dtype == GBS_BF16 ? launch_rope<__nv_bfloat16>(a, p->d, false, nullptr, nullptr, st)
                                   : launch_rope<float>(a, p->d, false, nullptr, nullptr, st),
              "gbs_qkv_rope_fwd");
}

extern "C" gbs_status gbs_qkv_rope_bwd(const gbs_rope_params* p, const gbs_heads* q, const gbs_heads* k,
                                       const void* wq, const void* wk, const float* cos_tab,
                                       const float* sin_tab, const int32_t* pos, const gbs_heads* dQ,
                                       const gbs_heads* dK, const gbs_heads* dV, const gbs_heads* dq,
                                       const gbs_heads* dk, const gbs_heads* dv, float* dwq, float* dwk,
                                       void* ws, size_t ws_bytes, void* stream) {
  set_last_error("");
  RopeArgs a;
  gbs_status s = resolve_rope(p, &a);
  if (s != GBS_OK) return s;
  const int es = p->dtype == GBS_BF16 ? 2 : 4;
  if (!dV != !dv) return fail_status(GBS_ERR_INVALID_ARG, "give both dV and dv or neither");
  const gbs_heads* in[] = {dQ, dK, dV};
  const gbs_heads* out[] = {dq, dk, dv};
  const gbs_heads* x[] = {q, k};
  const char* names[] = {"dQ", "dK", "dV", "dq", "dk", "dv", "q", "k"};
  for (int i = 0; i < 3; ++i) {
    if ((s = resolve_heads(in[i], names[i], es, i == 2, &a.in[i])) != GBS_OK) return s;
    if ((s = resolve_heads(out[i], names[3 + i], es, i == 2, &a.out[i])) != GBS_OK) return s;
    // the inputs of the forward are read for the norm only
    if (i < 2 && (s = resolve_heads(x[i], names[6 + i], es, wq == nullptr, &a.x[i])) != GBS_OK) return s;
  }
  if ((s = check_side(a, wq, wk, cos_tab, sin_tab, pos)) != GBS_OK) return s;
  if (wq && (!dwq || !dwk)) return fail_status(GBS_ERR_INVALID_ARG, "dwq or dwk is NULL");
  if (((uintptr_t)dwq | (uintptr_t)dwk) & 3u)
    return fail_status(GBS_ERR_INVALID_ARG, "dwq or dwk is not 4-byte aligned");
  const size_t need = gbs_qkv_rope_workspace_bytes(p);
  if (!ws) return fail_status(GBS_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
  if ((uintptr_t)ws & 255u) return fail_status(GBS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < need) return fail_status(GBS_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  const Heads read[] = {a.in[0], a.in[1], a.in[2], a.x[0], a.x[1]};
  const int in_heads[] = {p->Hq, p->Hkv, p->Hkv, p->Hq, p->Hkv};
  const char* read_names[] = {"dQ", "dK", "dV", "q", "k"};
  if ((s = check_apart(*p, wq ? 5 : 3, read, in_heads, read_names, a.out, names + 3)) != GBS_OK) return s;
  a.wq = wq; a.wk = wk; a.norm = wq != nullptr;
  a.cos_tab = cos_tab; a.sin_tab = sin_tab; a.pos = pos;
  a.err = static_cast<unsigned int*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  cudaStream_t st = (cudaStream_t)stream;
  return done(p->dtype == GBS_BF16 ? launch_rope<__nv_bfloat16>(a, p->d, true, dwq, dwk, st)
                                   : launch_rope<float>(a, p->d, true, dwq, dwk, st),
              "gbs_qkv_rope_bwd");
}
