// qkv_rope.cu — norms of queries and keys for each head and rotary positions in
// one pass, from a projection's layout to the attention's, and the backward.
//
// One row (token, head) of d channels is held by d / 8 lanes, eight channels to
// a lane: four and their rotation partners, so that a pair never leaves its lane
// (halves: channels 4 l .. 4 l + 3 and rot / 2 + 4 l ..; neighbours, and channels
// that are not rotated: 8 l .. 8 l + 7). The norm's sums go over the row's lanes
// by shuffles. A row is read once and written once, and the cos and sin of a
// token stay in registers for all of its heads, so the pass is bound by memory.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace gbs {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows whose loads are in flight before any arithmetic

struct RopeArgs {
  int B, N, Hq, Hkv, half, interleaved, n_axes, max_pos, norm, w_bf16;
  int per_token;  // lane groups that share a token's heads
  float eps;
  const void *wq, *wk;
  const float *cos_tab, *sin_tab;
  const int32_t* pos;
  Heads in[3], out[3];  // q, k, v and what becomes of them (backward: dQ, dK, dV -> dq, dk, dv)
  Heads x[2];           // backward: q, k
  float* part;          // backward: [CTAs][2][d] partial sums of dwq, dwk
  unsigned int* err;
  unsigned char axis[64];
};

template <typename T> struct Quad;  // four channels as one load
template <> struct Quad<float> { using type = float4; };
template <> struct Quad<__nv_bfloat16> { using type = uint2; };

__device__ __forceinline__ void widen(const float4& u, float* v) {
  v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
}
__device__ __forceinline__ void widen(const uint2& u, float* v) {
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void narrow(const float* v, float4* u) {
  *u = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void narrow(const float* v, uint2* u) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What a lane keeps of its token: the angles of its four pairs.
struct Angles {
  float c[4], s[4];
  int mode;  // 0: not rotated, 1: pairs (v[i], v[4 + i]), 2: pairs (v[2 i], v[2 i + 1])
};

__device__ __forceinline__ Angles load_angles(const RopeArgs& a, long long token, int lane, bool valid) {
  Angles r;
  const int i0 = 4 * lane;
  r.mode = i0 < a.half ? (a.interleaved ? 2 : 1) : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.c[i] = 1.f, r.s[i] = 0.f;
  if (r.mode && valid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int p = __ldg(a.pos + token * a.n_axes + a.axis[i0 + i]);
      if (p < 0 || p >= a.max_pos) {
        set_error(a.err, GBS_ERR_INVALID_ARG);
        p = p < 0 ? 0 : a.max_pos - 1;
      }
      r.c[i] = __ldg(a.cos_tab + (size_t)p * a.half + i0 + i);
      r.s[i] = __ldg(a.sin_tab + (size_t)p * a.half + i0 + i);
    }
  }
  return r;
}

// Rotates eight channels by the angles (SIGN = -1: by their negatives).
template <int SIGN>
__device__ __forceinline__ void rotate(float (&v)[8], const Angles& r) {
  if (r.mode == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[i], y = v[4 + i], s = SIGN * r.s[i];
      v[i] = x * r.c[i] - y * s;
      v[4 + i] = y * r.c[i] + x * s;
    }
  } else if (r.mode == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[2 * i], y = v[2 * i + 1], s = SIGN * r.s[i];
      v[2 * i] = x * r.c[i] - y * s;
      v[2 * i + 1] = y * r.c[i] + x * s;
    }
  }
}

// First channels of a lane's two quads.
__device__ __forceinline__ void quad_offsets(const RopeArgs& a, int lane, int* off) {
  if (!a.interleaved && 4 * lane < a.half) {
    off[0] = 4 * lane;
    off[1] = a.half + 4 * lane;
  } else {
    off[0] = 8 * lane;
    off[1] = 8 * lane + 4;
  }
}

__device__ __forceinline__ void load_weights(const RopeArgs& a, const void* w, const int* off, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = off[i >> 2] + (i & 3);
    v[i] = !w ? 1.f
              : (a.w_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[c])
                          : reinterpret_cast<const float*>(w)[c]);
  }
}

template <typename T>
__device__ __forceinline__ T* row_ptr(const Heads& t, int b, int h, int n) {
  return reinterpret_cast<T*>(t.ptr) + b * t.sb + h * t.sh + n * t.sn;
}

// One of the three tensors of a token: heads h = sub, sub + per_token, ...
// WHICH: 0 = q, 1 = k (norm and rotation), 2 = v (moved).
template <typename T, int D, int WHICH>
__device__ __forceinline__ void forward_heads(const RopeArgs& a, int b, int n, int sub, bool valid,
                                              const Angles& ang, const int* off) {
  using Q4 = typename Quad<T>::type;
  const int H = WHICH == 0 ? a.Hq : a.Hkv;
  float w[8];
  if (WHICH < 2) load_weights(a, WHICH == 0 ? a.wq : a.wk, off, w);
  const int rounds = (H + a.per_token * kUnroll - 1) / (a.per_token * kUnroll);
  for (int it = 0; it < rounds; ++it) {
    Q4 raw[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = sub + (it * kUnroll + u) * a.per_token;
      if (valid && h < H) {
        const T* src = row_ptr<T>(a.in[WHICH], b, h, n);
#pragma unroll
        for (int j = 0; j < 2; ++j) raw[u][j] = __ldg(reinterpret_cast<const Q4*>(src + off[j]));
      } else {
        raw[u][0] = raw[u][1] = Q4{};
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = sub + (it * kUnroll + u) * a.per_token;
      if (WHICH < 2) {
        float v[8];
        widen(raw[u][0], v);
        widen(raw[u][1], v + 4);
        if (a.norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
          const float r = rsqrtf(row_sum<D / 8>(ss) * (1.f / D) + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= r * w[i];
        }
        rotate<1>(v, ang);
        narrow(v, &raw[u][0]);
        narrow(v + 4, &raw[u][1]);
      }
      if (valid && h < H) {
        T* dst = row_ptr<T>(a.out[WHICH], b, h, n);
#pragma unroll
        for (int j = 0; j < 2; ++j) *reinterpret_cast<Q4*>(dst + off[j]) = raw[u][j];
      }
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int tokens_per_cta = GROUPS / a.per_token;
  const long long tokens = (long long)a.B * a.N;
  const long long token = (long long)blockIdx.x * tokens_per_cta + group / a.per_token;
  const int sub = group % a.per_token;
  const bool valid = token < tokens;
  const int b = valid ? (int)(token / a.N) : 0, n = valid ? (int)(token - (long long)b * a.N) : 0;
  const Angles ang = load_angles(a, token, lane, valid);
  int off[2];
  quad_offsets(a, lane, off);
  forward_heads<T, D, 0>(a, b, n, sub, valid, ang, off);
  forward_heads<T, D, 1>(a, b, n, sub, valid, ang, off);
  if (a.in[2].ptr) {
    int straight[2] = {8 * lane, 8 * lane + 4};
    forward_heads<T, D, 2>(a, b, n, sub, valid, ang, straight);
  }
}

// Backward of q (WHICH 0), k (1): dx from x and dz, and this lane's share of dw.
template <typename T, int D, int WHICH>
__device__ __forceinline__ void backward_heads(const RopeArgs& a, int b, int n, int sub, bool valid,
                                               const Angles& ang, const int* off, const float (&w)[8],
                                               float (&dw)[8]) {
  using Q4 = typename Quad<T>::type;
  constexpr int kRows = 2;  // two rows of x and dz in flight
  const int H = WHICH == 0 ? a.Hq : a.Hkv;
  const int rounds = (H + a.per_token * kRows - 1) / (a.per_token * kRows);
  for (int it = 0; it < rounds; ++it) {
    Q4 rz[kRows][2], rx[kRows][2];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int h = sub + (it * kRows + u) * a.per_token;
      rz[u][0] = rz[u][1] = rx[u][0] = rx[u][1] = Q4{};
      if (valid && h < H) {
        const T* dz = row_ptr<T>(a.in[WHICH], b, h, n);
#pragma unroll
        for (int j = 0; j < 2; ++j) rz[u][j] = __ldg(reinterpret_cast<const Q4*>(dz + off[j]));
        if (WHICH < 2 && a.norm) {
          const T* x = row_ptr<T>(a.x[WHICH], b, h, n);
#pragma unroll
          for (int j = 0; j < 2; ++j) rx[u][j] = __ldg(reinterpret_cast<const Q4*>(x + off[j]));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int h = sub + (it * kRows + u) * a.per_token;
      if (WHICH < 2) {
        float g[8];
        widen(rz[u][0], g);
        widen(rz[u][1], g + 4);
        rotate<-1>(g, ang);
        if (a.norm) {
          float x[8], ss = 0.f, hx = 0.f;
          widen(rx[u][0], x);
          widen(rx[u][1], x + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(x[i], x[i], ss);
            hx = fmaf(g[i] * w[i], x[i], hx);
          }
          const float r = rsqrtf(row_sum<D / 8>(ss) * (1.f / D) + a.eps);
          // mean(h xh) xh = x r^2 mean(h x)
          const float back = row_sum<D / 8>(hx) * (1.f / D) * r * r;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dw[i] = fmaf(g[i] * r, x[i], dw[i]);  // rows left out have g = x = 0
            g[i] = r * (g[i] * w[i] - x[i] * back);
          }
        }
        narrow(g, &rz[u][0]);
        narrow(g + 4, &rz[u][1]);
      }
      if (valid && h < H) {
        T* dx = row_ptr<T>(a.out[WHICH], b, h, n);
#pragma unroll
        for (int j = 0; j < 2; ++j) *reinterpret_cast<Q4*>(dx + off[j]) = rz[u][j];
      }
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
  __shared__ float sums[GROUPS][D];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int tokens_per_cta = GROUPS / a.per_token;
  const long long tokens = (long long)a.B * a.N;
  const int sub = group % a.per_token;
  int off[2], straight[2] = {8 * lane, 8 * lane + 4};
  quad_offsets(a, lane, off);
  float wq[8], wk[8], dwq[8] = {}, dwk[8] = {};
  load_weights(a, a.wq, off, wq);
  load_weights(a, a.wk, off, wk);
  // a CTA takes every gridDim.x-th run of tokens, so that few partial sums of dw are left
  for (long long first = (long long)blockIdx.x * tokens_per_cta; first < tokens;
       first += (long long)gridDim.x * tokens_per_cta) {
    const long long token = first + group / a.per_token;
    const bool valid = token < tokens;
    const int b = valid ? (int)(token / a.N) : 0, n = valid ? (int)(token - (long long)b * a.N) : 0;
    const Angles ang = load_angles(a, token, lane, valid);
    backward_heads<T, D, 0>(a, b, n, sub, valid, ang, off, wq, dwq);
    backward_heads<T, D, 1>(a, b, n, sub, valid, ang, off, wk, dwk);
    if (a.in[2].ptr) backward_heads<T, D, 2>(a, b, n, sub, valid, ang, straight, wk, dwk);
  }
  if (!a.norm) return;
  for (int t = 0; t < 2; ++t) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[group][off[i >> 2] + (i & 3)] = t ? dwk[i] : dwq[i];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kThreads) {
      float s = 0.f;
      for (int g = 0; g < GROUPS; ++g) s += sums[g][c];
      a.part[((size_t)blockIdx.x * 2 + t) * D + c] = s;
    }
  }
}

// dw[t][c] = sum of the CTAs' partial sums, in a fixed order.
__global__ void __launch_bounds__(256)
rope_dw_kernel(const float* __restrict__ part, int n, int d, float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float s_sum[8][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), row0 = threadIdx.x >> 5;
  float s = 0.f;
  for (int r = row0; r < n; r += 8) s += part[(size_t)r * 2 * d + col];
  s_sum[row0][threadIdx.x & 31] = s;
  __syncthreads();
  if (row0 == 0) {
    float v = 0.f;
    for (int r = 0; r < 8; ++r) v += s_sum[r][threadIdx.x];
    (col < d ? dwq[col] : dwk[col - d]) = v;
  }
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
  if ((long long)p.B * p.N > INT32_MAX || (long long)p.B * p.N * ((long long)p.Hq + p.Hkv) > ((long long)1 << 40))
    return fail_status(GBS_ERR_INVALID_ARG, "problem too large: B * N must be below 2^31");
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
  if (((uintptr_t)wq | (uintptr_t)wk) & 3u) return fail_status(GBS_ERR_INVALID_ARG, "a weight is not 4-byte aligned");
  if (a.half && (!cos_tab || !sin_tab || !pos))
    return fail_status(GBS_ERR_INVALID_ARG, "cos_tab, sin_tab or pos is NULL");
  if (((uintptr_t)cos_tab | (uintptr_t)sin_tab | (uintptr_t)pos) & 3u)
    return fail_status(GBS_ERR_INVALID_ARG, "cos_tab, sin_tab or pos is not 4-byte aligned");
  return GBS_OK;
}

// Lane groups that share a token's heads: as many as a CTA has while there are
// too few tokens to fill the GPU, and one when there are many.
int groups_per_token(const RopeArgs& a, int groups, int want_ctas) {
  const long long tokens = (long long)a.B * a.N;
  int g = 1;
  while (g < groups && tokens * g / groups < want_ctas) g *= 2;
  return g;
}

constexpr int kMaxBwdCtas = 148 * 4;

int bwd_ctas(const RopeArgs& a, int d, int per_token) {
  const int tokens_per_cta = kThreads / (d / 8) / per_token;
  const long long n = ((long long)a.B * a.N + tokens_per_cta - 1) / tokens_per_cta;
  return (int)(n < kMaxBwdCtas ? n : kMaxBwdCtas);
}

template <typename T>
cudaError_t launch_rope(RopeArgs& a, int d, bool backward, float* dwq, float* dwk, cudaStream_t st) {
  const int groups = kThreads / (d / 8);
  a.per_token = groups_per_token(a, groups, kMaxBwdCtas);
  const int tokens_per_cta = groups / a.per_token;
  if (!backward) {
    const unsigned grid = (unsigned)(((long long)a.B * a.N + tokens_per_cta - 1) / tokens_per_cta);
    if (d == 64) rope_fwd_kernel<T, 64><<<grid, kThreads, 0, st>>>(a);
    else rope_fwd_kernel<T, 128><<<grid, kThreads, 0, st>>>(a);
    note_launch();
    return cudaGetLastError();
  }
  const int grid = bwd_ctas(a, d, a.per_token);
  if (d == 64) rope_bwd_kernel<T, 64><<<grid, kThreads, 0, st>>>(a);
  else rope_bwd_kernel<T, 128><<<grid, kThreads, 0, st>>>(a);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.norm) return e;
  rope_dw_kernel<<<2 * d / 32, 256, 0, st>>>(a.part, grid, d, dwq, dwk);
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
  return 256 + (size_t)kMaxBwdCtas * 2 * p->d * sizeof(float);
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
  a.wq = wq; a.wk = wk; a.norm = wq != nullptr;
  a.cos_tab = cos_tab; a.sin_tab = sin_tab; a.pos = pos;
  a.err = static_cast<unsigned int*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  cudaStream_t st = (cudaStream_t)stream;
  return done(p->dtype == GBS_BF16 ? launch_rope<__nv_bfloat16>(a, p->d, true, dwq, dwk, st)
                                   : launch_rope<float>(a, p->d, true, dwq, dwk, st),
              "gbs_qkv_rope_bwd");
}
