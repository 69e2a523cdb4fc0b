// qk_norm_rope.cu — RMS norm of every query and key head, and the position
// rotation, in one pass over q and k; and its backward.
//
//   n = x / sqrt(mean(x^2) + eps) * w,  then the first `rot` features of the
//   head are rotated in pairs (a, b) by the angle position * inv_freq[i]:
//   a' = a cos - b sin,  b' = b cos + a sin.
// Pairs are (i, i + rot / 2), or (2i, 2i + 1) with `interleaved`.
//
// Backward, with r = 1 / sqrt(mean(x^2) + eps) and g the gradient turned back:
//   dw = sum over rows of g * x * r,
//   dx = r * (w g - x r^2 mean(x w g)).
//
// Bound by memory: one read and one write of every element (the backward reads
// x and dy and writes dx).  A thread holds 16 features of a row as two pieces
// of 8, chosen so that both members of each of its 8 pairs are its own: no
// exchange for the rotation, and 16-byte accesses.  A row is a group of G
// lanes, the norm's sums are log2(G) shuffles.  The angles of a token are
// computed once per CTA and shared by all its heads; they are formed in 64
// bits, in turns, since a far position times a frequency has no correct bits
// left below the point in 32.  This file is built without fast math: with fp32
// rows the outputs are compared at fp32's own steps.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "diffattn.h"
#include "kernels.h"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 1024;     // angles of a CTA's batch of tokens
constexpr int kBwdCtas = 148 * 2; // workspace rows; fixed, so that the size query needs no device

struct NormArgs {
  const void* x[2];  // q, k
  int64_t x_tok[2];  // token strides in elements
  void* y[2];        // forward: rows out
  int64_t y_tok[2];
  const float* dy[2];  // backward
  int64_t dy_tok[2];
  float* dx[2];  // dense
  const float* w[2];
  const int* positions;
  const float* inv_freq;
  float* partial;  // [gridDim.x][2][d]
  int tokens, heads[2], d, rot, tok_log2;  // 1 << tok_log2 tokens per batch
  float eps;
};

__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  x[0] = bf16lo(u.x), x[1] = bf16hi(u.x), x[2] = bf16lo(u.y), x[3] = bf16hi(u.y);
  x[4] = bf16lo(u.z), x[5] = bf16hi(u.z), x[6] = bf16lo(u.w), x[7] = bf16hi(u.w);
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                            pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Offsets of a thread's two pieces; `turned` says whether they are rotated.
template <bool kInterleaved>
__device__ __forceinline__ void pieces(int j, int rot, int& o0, int& o1, bool& turned) {
  const int n = rot >> 4;
  turned = j < n;
  if (!kInterleaved && turned) {
    o0 = 8 * j;
    o1 = o0 + (rot >> 1);
  } else {
    o0 = 16 * j;
    o1 = o0 + 8;
  }
}

// x[0..7] and x[8..15] rotated by the 8 angles; sign -1 turns back.
template <bool kInterleaved>
__device__ __forceinline__ void rotate(float (&x)[16], const float (&c)[8], const float (&s)[8],
                                       float sign) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& a = x[kInterleaved ? 2 * i : i];
    float& b = x[kInterleaved ? 2 * i + 1 : 8 + i];
    const float sn = sign * s[i];
    const float a0 = a, b0 = b;
    a = a0 * c[i] - b0 * sn;
    b = b0 * c[i] + a0 * sn;
  }
}

// cos and sin of the batch's tokens.  The product of a 32-bit position and an
// fp32 frequency is formed in 64 bits and reduced to a part of one turn there.
__device__ __forceinline__ void angles(const NormArgs& a, int tok0, float* cs, float* sn) {
  const int half = a.rot >> 1, n = half << a.tok_log2;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int t = i / half, p = i - t * half;
    if (tok0 + t >= a.tokens) break;
    double turns = (double)a.positions[tok0 + t] * (double)a.inv_freq[p] * 0.15915494309189535;
    turns -= rint(turns);
    float s, c;
    sincospif((float)(2.0 * turns), &s, &c);
    cs[i] = c;
    sn[i] = s;
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = 1; off < G; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ void load_angles(const float* cs, const float* sn, float (&c)[8],
                                            float (&s)[8]) {
  load8(cs, c);
  load8(sn, s);
}

// The weights and the token's angles as coefficients of a thread's 8 pairs:
// a' = r (a ac - b bs), b' = r (b bc + a as).
struct Coefs {
  float ac[8], bs[8], bc[8], as[8];
};

template <bool kInterleaved>
__device__ __forceinline__ void fold(const float* w, int o0, int o1, const float (&c)[8],
                                     const float (&s)[8], Coefs& f) {
  float g[16];
  if (w) {
    load8(w + o0, g);
    load8(w + o1, g + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = 1.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float wa = g[kInterleaved ? 2 * i : i], wb = g[kInterleaved ? 2 * i + 1 : 8 + i];
    f.ac[i] = wa * c[i], f.bs[i] = wb * s[i], f.bc[i] = wb * c[i], f.as[i] = wa * s[i];
  }
}

template <typename T>
struct Row {
  uint4 v[sizeof(T)];  // 16 features: two pieces of 8
};

template <typename T, int G, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2)
    qk_norm_rope_kernel(const NormArgs a) {
  __shared__ __align__(16) float cs[kAngles];
  __shared__ __align__(16) float sn[kAngles];
  const int j = threadIdx.x % G, g = threadIdx.x / G;
  const int per_tok = (kThreads / G) >> a.tok_log2;  // groups of a token
  const int t = g / per_tok;
  const int tok = ((int)blockIdx.x << a.tok_log2) + t;
  const int heads = a.heads[0] + a.heads[1];
  const int step = per_tok * (int)gridDim.y;
  int h = g % per_tok + per_tok * (int)blockIdx.y;
  const bool mine = tok < a.tokens && j * 16 < a.d;
  int o0, o1;
  bool turned;
  pieces<kInterleaved>(j, a.rot, o0, o1, turned);
  constexpr int kHalf = sizeof(T) / 2;  // 16-byte words of a piece
  auto fetch = [&](int head) {
    Row<T> r{};
    if (mine && head < heads) {
      const int kind = head >= a.heads[0];
      const T* p = static_cast<const T*>(a.x[kind]) + tok * a.x_tok[kind] +
                   (int64_t)(head - (kind ? a.heads[0] : 0)) * a.d;
#pragma unroll
      for (int i = 0; i < kHalf; ++i) {
        r.v[i] = reinterpret_cast<const uint4*>(p + o0)[i];
        r.v[kHalf + i] = reinterpret_cast<const uint4*>(p + o1)[i];
      }
    }
    return r;
  };
  Row<T> next = fetch(h);  // in flight while the angles are computed
  angles(a, (int)blockIdx.x << a.tok_log2, cs, sn);
  __syncthreads();
  float c[8], s[8];
  if (turned) {
    load_angles(cs + t * (a.rot >> 1) + 8 * j, sn + t * (a.rot >> 1) + 8 * j, c, s);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  }
  Coefs f;
  int kind = -1;
  const float inv_d = 1.0f / (float)a.d;
  // Every group of the CTA takes the same number of turns: the shuffles of a
  // warp need all its lanes.
  const int first = per_tok * (int)blockIdx.y;
  for (int base = first; base < heads; base += step, h += step) {
    float x[16];
    load8(reinterpret_cast<const T*>(&next.v[0]), x);
    load8(reinterpret_cast<const T*>(&next.v[kHalf]), x + 8);
    if (base + step < heads) next = fetch(h + step);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
    const float r = rsqrtf(group_sum<G>(ss) * inv_d + a.eps);
    if (mine && h < heads) {
      const int k = h >= a.heads[0];
      if (k != kind) {  // once for the queries, once for the keys
        kind = k;
        fold<kInterleaved>(a.w[k], o0, o1, c, s, f);
      }
      float y[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = x[kInterleaved ? 2 * i : i], v = x[kInterleaved ? 2 * i + 1 : 8 + i];
        y[kInterleaved ? 2 * i : i] = r * (u * f.ac[i] - v * f.bs[i]);
        y[kInterleaved ? 2 * i + 1 : 8 + i] = r * (v * f.bc[i] + u * f.as[i]);
      }
      T* p = static_cast<T*>(a.y[k]) + tok * a.y_tok[k] +
             (int64_t)(h - (k ? a.heads[0] : 0)) * a.d;
      store8(p + o0, y);
      store8(p + o1, y + 8);
    }
  }
}

// Backward.  CTAs walk over batches of tokens and keep the weights' gradient
// of their own rows in registers (fp32: a thread adds a few hundred rows at
// most); each writes one row of sums, and the second kernel adds those in 64
// bits.  The order depends on the sizes alone.
template <typename T, int G, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_rope_bwd_kernel(const NormArgs a) {
  __shared__ __align__(16) float cs[2][kAngles];
  __shared__ __align__(16) float sn[2][kAngles];
  __shared__ float sums[kThreads / 32][2 * 256];
  const int j = threadIdx.x % G, g = threadIdx.x / G;
  const int per_tok = (kThreads / G) >> a.tok_log2;
  const int t = g / per_tok;
  const int heads = a.heads[0] + a.heads[1];
  const bool in_row = j * 16 < a.d;
  int o0, o1;
  bool turned;
  pieces<kInterleaved>(j, a.rot, o0, o1, turned);
  float acc[2][16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.f;
  const int batches = (a.tokens + (1 << a.tok_log2) - 1) >> a.tok_log2;
  angles(a, (int)blockIdx.x << a.tok_log2, cs[0], sn[0]);
  for (int batch = blockIdx.x, turn = 0; batch < batches; batch += gridDim.x, ++turn) {
    const int tok = (batch << a.tok_log2) + t;
    const int buf = turn & 1;
    __syncthreads();  // this batch's angles are there, the other buffer is free
    if (batch + (int)gridDim.x < batches)
      angles(a, (batch + (int)gridDim.x) << a.tok_log2, cs[buf ^ 1], sn[buf ^ 1]);
    float c[8], s[8];
    if (turned) {
      load_angles(cs[buf] + t * (a.rot >> 1) + 8 * j, sn[buf] + t * (a.rot >> 1) + 8 * j, c, s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    }
    const bool mine = tok < a.tokens && in_row;
    for (int base = 0; base < heads; base += per_tok) {
      const int h = base + g % per_tok;
      const bool live = mine && h < heads;
      const int kind = h >= a.heads[0];
      const int hk = h - (kind ? a.heads[0] : 0);
      float x[16], dy[16], w[16];
      if (live) {
        const T* p = static_cast<const T*>(a.x[kind]) + tok * a.x_tok[kind] + (int64_t)hk * a.d;
        load8(p + o0, x);
        load8(p + o1, x + 8);
        const float* q = a.dy[kind] + tok * a.dy_tok[kind] + (int64_t)hk * a.d;
        load8(q + o0, dy);
        load8(q + o1, dy + 8);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = dy[i] = 0.f;
      }
      if (in_row && a.w[kind]) {
        load8(a.w[kind] + o0, w);
        load8(a.w[kind] + o1, w + 8);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = 1.f;
      }
      if (turned && live) rotate<kInterleaved>(dy, c, s, -1.f);  // no angles past the last token
      float ss = 0.f, sg = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        ss = fmaf(x[i], x[i], ss);
        sg = fmaf(x[i] * w[i], dy[i], sg);
      }
      const float inv_d = 1.0f / (float)a.d;
      float r = rsqrtf(group_sum<G>(ss) * inv_d + a.eps);
      if (!live) r = 0.f;  // with eps = 0 it is an infinity here
      const float m = group_sum<G>(sg) * r * inv_d;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float n = x[i] * r;
        if (kind) acc[1][i] = fmaf(dy[i], n, acc[1][i]);
        else acc[0][i] = fmaf(dy[i], n, acc[0][i]);
        x[i] = r * (w[i] * dy[i] - n * m);
      }
      if (live) {
        float* p = a.dx[kind] + ((int64_t)tok * a.heads[kind] + hk) * a.d;
        store8(p + o0, x);
        store8(p + o1, x + 8);
      }
    }
  }
  // Sum over the warp's groups, then over the warps.
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int off = G; off < 32; off <<= 1)
        acc[k][i] += __shfl_xor_sync(0xffffffffu, acc[k][i], off);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane < G && in_row) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        sums[warp][k * a.d + (i < 8 ? o0 + i : o1 + i - 8)] = acc[k][i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += sums[w][i];
    a.partial[(size_t)blockIdx.x * 2 * a.d + i] = v;
  }
}

// Columns of the CTAs' sums: a block adds 32 of them, 8 rows at a time.
__global__ void __launch_bounds__(256) qk_norm_dweight_kernel(const float* partial, int rows,
                                                              int d, float* dwq, float* dwk) {
  __shared__ double sh[8][32];
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  double v = 0.0;
  if (col < 2 * d) {
#pragma unroll 8
    for (int r = y; r < rows; r += 8) v += (double)partial[(size_t)r * 2 * d + col];
  }
  sh[y][lane] = v;
  __syncthreads();
  if (y == 0 && col < 2 * d) {
    for (int i = 1; i < 8; ++i) v += sh[i][lane];
    float* out = col < d ? dwq : dwk;
    if (out) out[col < d ? col : col - d] = (float)v;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Lanes of a row: the power of two from ceil(d / 16).
int lanes_of(int d) {
  int g = 1;
  while (g * 16 < d) g <<= 1;
  return g;
}

int check(const void* q, const void* k, long long q_tok, long long k_tok, da_dtype dtype,
          int tokens, int n_q, int n_k, int d, int rot, const int* positions,
          const float* inv_freq, const float* wq, const float* wk, float eps) {
  if (dtype != DA_BF16 && dtype != DA_FP32) return DA_ERR_INVALID_ARG;
  if (tokens < 0 || n_q < 1 || n_k < 0 || d < 1 || rot < 0 || rot > d) return DA_ERR_INVALID_ARG;
  if (!(eps >= 0.f)) return DA_ERR_INVALID_ARG;
  if (d % 16 || d > 256 || rot % 16) return DA_ERR_UNSUPPORTED;
  if (n_q > (1 << 20) || n_k > (1 << 20)) return DA_ERR_UNSUPPORTED;
  if (tokens == 0) return DA_OK;
  if (!q || (n_k > 0 && !k) || (rot > 0 && (!positions || !inv_freq))) return DA_ERR_INVALID_ARG;
  if (q_tok < (long long)n_q * d || (n_k > 0 && k_tok < (long long)n_k * d))
    return DA_ERR_INVALID_ARG;
  const int per16 = dtype == DA_BF16 ? 8 : 4;
  if (q_tok % per16 || (n_k > 0 && k_tok % per16)) return DA_ERR_ALIGNMENT;
  if (!aligned16(q) || (n_k > 0 && !aligned16(k)) || !aligned16(wq) || !aligned16(wk))
    return DA_ERR_ALIGNMENT;
  return DA_OK;
}

// Calls f with the template arguments of (dtype, lanes, pairing).
template <typename F>
void dispatch(da_dtype dtype, int lanes, bool interleaved, F&& f) {
  auto with_lanes = [&](auto t, auto il) {
    switch (lanes) {
      case 1: f(t, std::integral_constant<int, 1>{}, il); break;
      case 2: f(t, std::integral_constant<int, 2>{}, il); break;
      case 4: f(t, std::integral_constant<int, 4>{}, il); break;
      case 8: f(t, std::integral_constant<int, 8>{}, il); break;
      default: f(t, std::integral_constant<int, 16>{}, il); break;
    }
  };
  auto with_type = [&](auto t) {
    if (interleaved) with_lanes(t, std::true_type{});
    else with_lanes(t, std::false_type{});
  };
  if (dtype == DA_BF16) with_type(__nv_bfloat16{});
  else with_type(float{});
}

// Tokens of a CTA's batch (log2): as many as give every group of lanes a head,
// while 148 CTAs are left; then up to four where `enough` CTAs are left, so
// that more heads share a thread's angles.
int batch_log2(int tokens, int heads, int lanes, int rot, int enough) {
  const int groups = kThreads / lanes;
  int lg = 0;
  auto room = [&](int ctas) {
    return (rot << lg) <= kAngles && (tokens >> (lg + 1)) >= ctas && (groups >> (lg + 1)) >= 1;
  };
  while (room(148) && (groups >> (lg + 1)) >= heads) ++lg;
  while (lg < 2 && room(enough)) ++lg;
  return lg;
}

}  // namespace
}  // namespace da

extern "C" int diffattn_qk_norm_rope(const void* q, long long q_token_stride, const void* k,
                                     long long k_token_stride, da_dtype dtype, int tokens,
                                     int n_q_heads, int n_k_heads, int head_dim,
                                     const float* q_weight, const float* k_weight,
                                     float norm_eps, const int* positions,
                                     const float* inv_freq, int rot_dim, int interleaved,
                                     void* q_out, long long q_out_token_stride, void* k_out,
                                     long long k_out_token_stride, void* stream) {
  const int st = da::check(q, k, q_token_stride, k_token_stride, dtype, tokens, n_q_heads,
                           n_k_heads, head_dim, rot_dim, positions, inv_freq, q_weight, k_weight,
                           norm_eps);
  if (st != DA_OK || tokens == 0) return st;
  if (!q_out || (n_k_heads > 0 && !k_out)) return DA_ERR_INVALID_ARG;
  if (q_out_token_stride < (long long)n_q_heads * head_dim ||
      (n_k_heads > 0 && k_out_token_stride < (long long)n_k_heads * head_dim))
    return DA_ERR_INVALID_ARG;
  const int per16 = dtype == DA_BF16 ? 8 : 4;
  if (q_out_token_stride % per16 || (n_k_heads > 0 && k_out_token_stride % per16))
    return DA_ERR_ALIGNMENT;
  if (!da::aligned16(q_out) || (n_k_heads > 0 && !da::aligned16(k_out)))
    return DA_ERR_ALIGNMENT;
  da::NormArgs a{};
  a.x[0] = q, a.x[1] = k;
  a.x_tok[0] = q_token_stride, a.x_tok[1] = k_token_stride;
  a.y[0] = q_out, a.y[1] = k_out;
  a.y_tok[0] = q_out_token_stride, a.y_tok[1] = k_out_token_stride;
  a.w[0] = q_weight, a.w[1] = k_weight;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.tokens = tokens;
  a.heads[0] = n_q_heads, a.heads[1] = n_k_heads;
  a.d = head_dim;
  a.rot = rot_dim;
  a.eps = norm_eps;
  const int heads = n_q_heads + n_k_heads, lanes = da::lanes_of(head_dim);
  a.tok_log2 = da::batch_log2(tokens, heads, lanes, rot_dim, 148 * 8);
  const int per_tok = (da::kThreads / lanes) >> a.tok_log2;
  dim3 grid((unsigned)(((long long)tokens + (1 << a.tok_log2) - 1) >> a.tok_log2), 1, 1);
  // Few tokens: a token's heads are split over CTAs too.
  const int turns = (heads + per_tok - 1) / per_tok;
  while (grid.y < (unsigned)turns && (long long)grid.x * grid.y < 148 * 4) ++grid.y;
  if (grid.y > 65535u) grid.y = 65535u;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  da::dispatch(dtype, lanes, interleaved != 0, [&](auto t, auto g, auto il) {
    da::qk_norm_rope_kernel<decltype(t), decltype(g)::value, decltype(il)::value>
        <<<grid, da::kThreads, 0, cs>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

extern "C" size_t diffattn_qk_norm_rope_bwd_workspace_size(int tokens, int n_q_heads,
                                                           int n_k_heads, int head_dim) {
  if (tokens < 0 || n_q_heads < 1 || n_k_heads < 0 || head_dim < 16 || head_dim > 256 ||
      head_dim % 16)
    return 0;
  const int ctas = tokens < da::kBwdCtas ? tokens : da::kBwdCtas;
  return (size_t)(ctas < 1 ? 1 : ctas) * 2 * head_dim * sizeof(float);
}

extern "C" int diffattn_qk_norm_rope_bwd(
    const void* q, long long q_token_stride, const void* k, long long k_token_stride,
    da_dtype dtype, const float* dq_out, long long dq_out_token_stride, const float* dk_out,
    long long dk_out_token_stride, int tokens, int n_q_heads, int n_k_heads, int head_dim,
    const float* q_weight, const float* k_weight, float norm_eps, const int* positions,
    const float* inv_freq, int rot_dim, int interleaved, float* dq, float* dk, float* dq_weight,
    float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = da::check(q, k, q_token_stride, k_token_stride, dtype, tokens, n_q_heads,
                           n_k_heads, head_dim, rot_dim, positions, inv_freq, q_weight, k_weight,
                           norm_eps);
  if (st != DA_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {  // the weights' gradients are sums over no rows
    const size_t n = (size_t)head_dim * sizeof(float);
    if (dq_weight && cudaMemsetAsync(dq_weight, 0, n, cs) != cudaSuccess) return DA_ERR_CUDA;
    if (dk_weight && cudaMemsetAsync(dk_weight, 0, n, cs) != cudaSuccess) return DA_ERR_CUDA;
    return DA_OK;
  }
  if (!dq_out || !dq || (n_k_heads > 0 && (!dk_out || !dk))) return DA_ERR_INVALID_ARG;
  if (dq_out_token_stride < (long long)n_q_heads * head_dim ||
      (n_k_heads > 0 && dk_out_token_stride < (long long)n_k_heads * head_dim))
    return DA_ERR_INVALID_ARG;
  if (dq_out_token_stride % 4 || (n_k_heads > 0 && dk_out_token_stride % 4))
    return DA_ERR_ALIGNMENT;
  if (!da::aligned16(dq_out) || !da::aligned16(dq) ||
      (n_k_heads > 0 && (!da::aligned16(dk_out) || !da::aligned16(dk))))
    return DA_ERR_ALIGNMENT;
  if (!workspace ||
      workspace_bytes <
          diffattn_qk_norm_rope_bwd_workspace_size(tokens, n_q_heads, n_k_heads, head_dim))
    return DA_ERR_WORKSPACE;
  if (!da::aligned16(workspace)) return DA_ERR_ALIGNMENT;
  da::NormArgs a{};
  a.x[0] = q, a.x[1] = k;
  a.x_tok[0] = q_token_stride, a.x_tok[1] = k_token_stride;
  a.dy[0] = dq_out, a.dy[1] = dk_out;
  a.dy_tok[0] = dq_out_token_stride, a.dy_tok[1] = dk_out_token_stride;
  a.dx[0] = dq, a.dx[1] = dk;
  a.w[0] = q_weight, a.w[1] = k_weight;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.partial = static_cast<float*>(workspace);
  a.tokens = tokens;
  a.heads[0] = n_q_heads, a.heads[1] = n_k_heads;
  a.d = head_dim;
  a.rot = rot_dim;
  a.eps = norm_eps;
  const int heads = n_q_heads + n_k_heads, lanes = da::lanes_of(head_dim);
  a.tok_log2 = da::batch_log2(tokens, heads, lanes, rot_dim, da::kBwdCtas);
  const int batches = (int)(((long long)tokens + (1 << a.tok_log2) - 1) >> a.tok_log2);
  const int ctas = batches < da::kBwdCtas ? batches : da::kBwdCtas;
  da::dispatch(dtype, lanes, interleaved != 0, [&](auto t, auto g, auto il) {
    da::qk_norm_rope_bwd_kernel<decltype(t), decltype(g)::value, decltype(il)::value>
        <<<ctas, da::kThreads, 0, cs>>>(a);
  });
  if (cudaGetLastError() != cudaSuccess) return DA_ERR_CUDA;
  if (dq_weight || dk_weight) {
    da::qk_norm_dweight_kernel<<<(2 * head_dim + 31) / 32, 256, 0, cs>>>(
        a.partial, ctas, head_dim, dq_weight, dk_weight);
    if (cudaGetLastError() != cudaSuccess) return DA_ERR_CUDA;
  }
  return DA_OK;
}
