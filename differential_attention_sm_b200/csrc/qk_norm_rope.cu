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
// left below the point in 32.  CTAs are persistent (two an SM) and rows are on
// their way through shared memory several turns ahead: registers alone held
// too few bytes in flight (72 us where this takes 58).  This file is built
// without fast math: with fp32 rows the outputs are compared at fp32's own steps.
// Measured: 16384 tokens of 40 heads of 128 58 to 60 us, 0.85 to 0.88 of the copy
// rate; the backward, 64 heads of 64, 116 to 118 us, 0.87.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "diffattn.h"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 2;
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
__device__ __forceinline__ void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
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
// fp32 frequency is formed in 64 bits and reduced to a part of one turn there;
// rounding that part to fp32 moves the angle by pi * 2^-25 at most.
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
// a' = r (a wa cos - b wb sin), b' = r (b wb cos + a wa sin).  Held two by two
// for the packed fp32 instructions, which halve the arithmetic: at one
// instruction a feature it took as long as the memory (71 us for 16384 tokens
// of 40 heads where the bytes take 51).
//  halves:      words 0 .. 3 make a' of two pairs each, words 4 .. 7 b'
//  interleaved: word i makes (a', b') of pair i
// out[i] = r (own[i] c[i] + other[i] s[i])
struct Coefs {
  uint64_t c[8], s[8];
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
  if (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f.c[i] = f2pack(g[2 * i] * c[i], g[2 * i + 1] * c[i]);
      f.s[i] = f2pack(-g[2 * i + 1] * s[i], g[2 * i] * s[i]);
    }
  } else {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int i = 2 * m, k = i + 1;
      f.c[m] = f2pack(g[i] * c[i], g[k] * c[k]);
      f.s[m] = f2pack(-g[8 + i] * s[i], -g[8 + k] * s[k]);
      f.c[4 + m] = f2pack(g[8 + i] * c[i], g[8 + k] * c[k]);
      f.s[4 + m] = f2pack(g[i] * s[i], g[k] * s[k]);
    }
  }
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t swapped(uint64_t x) { return (x << 32) | (x >> 32); }

// Sixteen features as held, and as fp32 pairs.
template <typename T>
struct Row {
  uint4 v[sizeof(T)];
};
__device__ __forceinline__ void unpack(const Row<__nv_bfloat16>& r, uint64_t (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[4 * i + j] = f2pack(bf16lo(u[j]), bf16hi(u[j]));
  }
}
__device__ __forceinline__ void unpack(const Row<float>& r, uint64_t (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = f2pack(__uint_as_float(r.v[i].x), __uint_as_float(r.v[i].y));
    x[2 * i + 1] = f2pack(__uint_as_float(r.v[i].z), __uint_as_float(r.v[i].w));
  }
}
__device__ __forceinline__ void store_pairs(__nv_bfloat16* p, const uint64_t* y) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2unpack(y[i], lo, hi);
    u[i] = pack_bf16(lo, hi);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store_pairs(float* p, const uint64_t* y) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float4 f;
    f2unpack(y[2 * i], f.x, f.y);
    f2unpack(y[2 * i + 1], f.z, f.w);
    reinterpret_cast<float4*>(p)[i] = f;
  }
}

// Through L1: of fp32 rows a thread's 8 features are two copies of half a sector
// each (past L1 the backward took 150 us for 107).
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// CTAs walk over batches of tokens (blockIdx.y: over the heads of a token, when
// tokens are few).  While a batch's rows pass through, the next batch's angles
// are computed into the other buffer, and a thread's next rows are in flight.
// kPart: some features are not rotated.  Their way around an infinity is left out
// where all are: 16384 tokens of 40 heads of 128 took 61 us with it for 60, and
// with half of the features rotated take 57.8 for 57.4 (interleaved 59.0).
template <typename T, int G, bool kInterleaved, bool kPart>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) qk_norm_rope_kernel(const NormArgs a) {
  __shared__ __align__(16) float cs[2][kAngles];
  __shared__ __align__(16) float sn[2][kAngles];
  let_next_start();
  after_previous();
  const int j = threadIdx.x % G, g = threadIdx.x / G;
  const int per_tok = (kThreads / G) >> a.tok_log2;  // groups of a token
  const int t = g / per_tok;
  const int n_q = a.heads[0], heads = n_q + a.heads[1];
  const int step = per_tok * (int)gridDim.y;
  const int first = per_tok * (int)blockIdx.y;  // of the CTA
  const int h0 = first + g % per_tok;
  const bool in_row = j * 16 < a.d;
  int o0, o1;
  bool turned;
  pieces<kInterleaved>(j, a.rot, o0, o1, turned);
  // Rows of head 0 of the queries, and of the keys as if they followed them.
  const int64_t back = (int64_t)n_q * a.d;
  const T* src0 = static_cast<const T*>(a.x[0]) + o0;
  const T* src1 = static_cast<const T*>(a.x[1]) - back + o0;
  T* dst0 = static_cast<T*>(a.y[0]) + o0;
  T* dst1 = static_cast<T*>(a.y[1]) - back + o0;
  const int apart = o1 - o0;
  const int batches = (a.tokens + (1 << a.tok_log2) - 1) >> a.tok_log2;
  const float inv_d = 1.0f / (float)a.d;
  // The thread's own rows on their way: it copies and reads only its own 16
  // bytes of each, so no one else has to be waited for.
  constexpr int kWords = sizeof(T);  // 16-byte words of a thread's part of a row
  constexpr int kDepth = 8 / kWords;
  __shared__ uint4 ring[kDepth][kWords][kThreads];
  int p_batch = (int)blockIdx.x, p_base = first;  // next row to ask for
  auto push = [&](int slot) {
    const int tok = (p_batch << a.tok_log2) + t, head = p_base + g % per_tok;
    if (p_batch < batches && tok < a.tokens && in_row && head < heads) {
      const T* p = (head >= n_q ? src1 + tok * a.x_tok[1] : src0 + tok * a.x_tok[0]) + head * a.d;
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {
        copy16(&ring[slot][i][threadIdx.x], reinterpret_cast<const uint4*>(p) + i);
        copy16(&ring[slot][kWords / 2 + i][threadIdx.x],
               reinterpret_cast<const uint4*>(p + apart) + i);
      }
    }
    copy_commit();
    p_base += step;
    if (p_base >= heads) {
      p_base = first;
      p_batch += (int)gridDim.x;
    }
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) push(k);
  int slot = 0;
  int batch = (int)blockIdx.x;
  angles(a, batch << a.tok_log2, cs[0], sn[0]);
  for (int buf = 0; batch < batches; buf ^= 1) {
    const int tok = (batch << a.tok_log2) + t;
    batch += (int)gridDim.x;
    __syncthreads();  // this batch's angles are there, the other buffer is free
    if (batch < batches) angles(a, batch << a.tok_log2, cs[buf ^ 1], sn[buf ^ 1]);
    float c[8], s[8];
    if (turned) {
      load_angles(cs[buf] + t * (a.rot >> 1) + 8 * j, sn[buf] + t * (a.rot >> 1) + 8 * j, c, s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    }
    Coefs f;
    int kind = -1;
    // Every group of the CTA takes the same number of turns: the shuffles of a
    // warp need all its lanes.
    for (int base = first, h = h0; base < heads; base += step, h += step) {
      push(slot == 0 ? kDepth - 1 : slot - 1);
      copy_wait<kDepth - 1>();
      Row<T> row{};  // lanes past the row's end add nothing to its sum
      if (in_row) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) row.v[i] = ring[slot][i][threadIdx.x];
      }
      if (++slot == kDepth) slot = 0;
      uint64_t x[8];
      unpack(row, x);
      uint64_t sq = mul2(x[0], x[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) sq = fma2(x[i], x[i], sq);
      float lo, hi;
      f2unpack(sq, lo, hi);
      const float r = rsqrtf(group_sum<G>(lo + hi) * inv_d + a.eps);
      if (tok < a.tokens && in_row && h < heads) {
        const int k = h >= n_q;
        if (k != kind) {  // once for the queries, once for the keys
          kind = k;
          fold<kInterleaved>(a.w[k], o0, o1, c, s, f);
        }
        const uint64_t r2 = f2pack(r, r);
        uint64_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t other = kInterleaved ? swapped(x[i]) : x[i ^ 4];
          y[i] = mul2(r2, fma2(x[i], f.c[i], mul2(other, f.s[i])));
        }
        // A row that holds an infinity: what is not rotated has no partner, and
        // the partner's product with a sine of 0 would be a NaN.
        if (kPart && r == 0.f && !turned) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = mul2(r2, mul2(x[i], f.c[i]));
        }
        T* p = (k ? dst1 + tok * a.y_tok[1] : dst0 + tok * a.y_tok[0]) + h * a.d;
        store_pairs(p, y);
        store_pairs(p + apart, y + 4);
      }
    }
  }
}

// Backward.  CTAs walk over batches of tokens as above and keep the weights'
// gradient of their own rows in registers, in fp32 for up to kFoldRows rows of a
// thread.  With more (kMany; 1.2 million rows of 128), a warp adds those up in 64
// bits in shared memory and begins anew, so that the error does not grow with
// the rows; 8 million rows of 128 take 1.71 ms with it and 1.66 without, and
// 16384 tokens of 64 heads of 64, which need none, 117 and 116 us.  Each CTA writes
// one row of sums, and the second kernel adds those in 64 bits.  The order depends
// on the sizes alone.
constexpr int kBwdDepth = 2;  // rows of a thread in shared memory (3: 114 us for 110)
constexpr int kFoldRows = 128;
template <typename T>
struct BwdSmem {
  float cs[2][kAngles], sn[2][kAngles];
  union {
    uint4 ring[kBwdDepth][sizeof(T) + 4][kThreads];  // words of x, then of dy
    float sums[kThreads / 32][2 * 256];              // the warps' last rows
  };
  // and with kMany double [kThreads / 32][2 * d] behind it: their rows before those
};
template <typename T>
constexpr int bwd_smem_of(int d, bool many) {
  return (int)sizeof(BwdSmem<T>) + (many ? kThreads / 32 * 2 * d * (int)sizeof(double) : 0);
}

template <typename T, int G, bool kInterleaved, bool kMany>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) qk_norm_rope_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  BwdSmem<T>& sh = *reinterpret_cast<BwdSmem<T>*>(smem);
  double* const folded = reinterpret_cast<double*>(smem + sizeof(BwdSmem<T>));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  let_next_start();
  after_previous();
  const int j = threadIdx.x % G, g = threadIdx.x / G;
  const int per_tok = (kThreads / G) >> a.tok_log2;
  const int t = g / per_tok;
  const int n_q = a.heads[0], heads = n_q + a.heads[1];
  const bool in_row = j * 16 < a.d;
  int o0, o1;
  bool turned;
  pieces<kInterleaved>(j, a.rot, o0, o1, turned);
  const int64_t back = (int64_t)n_q * a.d;
  const T* x0 = static_cast<const T*>(a.x[0]) + o0;
  const T* x1 = static_cast<const T*>(a.x[1]) - back + o0;
  const float* dy0 = a.dy[0] + o0;
  const float* dy1 = a.dy[1] - back + o0;
  const int apart = o1 - o0;
  const int batches = (a.tokens + (1 << a.tok_log2) - 1) >> a.tok_log2;
  constexpr int kWords = sizeof(T);
  int p_batch = (int)blockIdx.x, p_head = g % per_tok;  // next row to ask for
  auto push = [&](int slot) {
    const int tok = (p_batch << a.tok_log2) + t;
    if (p_batch < batches && tok < a.tokens && in_row && p_head < heads) {
      const bool k = p_head >= n_q;
      const T* p = (k ? x1 + tok * a.x_tok[1] : x0 + tok * a.x_tok[0]) + p_head * a.d;
      const float* q = (k ? dy1 + tok * a.dy_tok[1] : dy0 + tok * a.dy_tok[0]) + p_head * a.d;
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {
        copy16(&sh.ring[slot][i][threadIdx.x], reinterpret_cast<const uint4*>(p) + i);
        copy16(&sh.ring[slot][kWords / 2 + i][threadIdx.x],
               reinterpret_cast<const uint4*>(p + apart) + i);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        copy16(&sh.ring[slot][kWords + i][threadIdx.x], reinterpret_cast<const uint4*>(q) + i);
        copy16(&sh.ring[slot][kWords + 2 + i][threadIdx.x],
               reinterpret_cast<const uint4*>(q + apart) + i);
      }
    }
    copy_commit();
    p_head += per_tok;
    if (p_head - g % per_tok >= heads) {
      p_head = g % per_tok;
      p_batch += (int)gridDim.x;
    }
  };
#pragma unroll
  for (int k = 0; k < kBwdDepth - 1; ++k) push(k);
  int slot = 0;
  float acc[2][16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.f;
  // The sums of the warp's groups, in every lane.
  auto add_groups = [&] {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int off = G; off < 32; off <<= 1)
          acc[k][i] += __shfl_xor_sync(0xffffffffu, acc[k][i], off);
  };
  int rows = 0;         // in acc
  bool more = false;    // `folded` holds some
  auto fold = [&] {
    add_groups();
    if (lane < G && in_row) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          double* p = folded + (warp * 2 + k) * a.d + (half ? o1 : o0);
          double v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = more ? p[i] : 0.0;
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = v[i] + (double)acc[k][8 * half + i];
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.f;
    rows = 0;
    more = true;
  };
  angles(a, (int)blockIdx.x << a.tok_log2, sh.cs[0], sh.sn[0]);
  int buf = 0;
  for (int batch = blockIdx.x; batch < batches; batch += gridDim.x, buf ^= 1) {
    const int tok = (batch << a.tok_log2) + t;
    __syncthreads();  // this batch's angles are there, the other buffer is free
    if (batch + (int)gridDim.x < batches)
      angles(a, (batch + (int)gridDim.x) << a.tok_log2, sh.cs[buf ^ 1], sh.sn[buf ^ 1]);
    float c[8], s[8];
    if (turned) {
      load_angles(sh.cs[buf] + t * (a.rot >> 1) + 8 * j, sh.sn[buf] + t * (a.rot >> 1) + 8 * j, c,
                  s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    }
    const bool mine = tok < a.tokens && in_row;
    for (int base = 0; base < heads; base += per_tok) {
      push(slot == 0 ? kBwdDepth - 1 : slot - 1);
      copy_wait<kBwdDepth - 1>();
      const int h = base + g % per_tok;
      const bool live = mine && h < heads;
      const int kind = h >= n_q;
      float x[16], dy[16], w[16];
      if (live) {
        Row<T> row;
        Row<float> grad;
#pragma unroll
        for (int i = 0; i < kWords; ++i) row.v[i] = sh.ring[slot][i][threadIdx.x];
#pragma unroll
        for (int i = 0; i < 4; ++i) grad.v[i] = sh.ring[slot][kWords + i][threadIdx.x];
        uint64_t p[8];
        unpack(row, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) f2unpack(p[i], x[2 * i], x[2 * i + 1]);
        unpack(grad, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) f2unpack(p[i], dy[2 * i], dy[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = dy[i] = 0.f;
      }
      if (++slot == kBwdDepth) slot = 0;
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
        float* p = a.dx[kind] + ((int64_t)tok * a.heads[kind] + h - (kind ? n_q : 0)) * a.d;
        store8(p + o0, x);
        store8(p + o1, x + 8);
      }
      if (kMany && ++rows == kFoldRows) fold();  // all lanes: the CTA's groups take the same turns
    }
  }
  copy_wait<0>();
  __syncthreads();  // the ring's place is taken by the sums
  // Sum over the warp's groups, then over the warps.
  add_groups();
  if (lane < G && in_row) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        sh.sums[warp][k * a.d + (i < 8 ? o0 + i : o1 + i - 8)] = acc[k][i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += sh.sums[w][i];
    if (kMany && more) {
      double all = v;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) all += folded[w * 2 * a.d + i];
      v = (float)all;
    }
    a.partial[(size_t)blockIdx.x * 2 * a.d + i] = v;
  }
}

// Columns of the CTAs' sums: a block adds 32 of them, 32 rows at a time.
__global__ void __launch_bounds__(1024) qk_norm_dweight_kernel(const float* partial, int rows,
                                                               int d, float* dwq, float* dwk) {
  __shared__ double sh[32][33];
  let_next_start();
  after_previous();
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  double v = 0.0;
  if (col < 2 * d) {
#pragma unroll 10
    for (int r = y; r < rows; r += 32) v += (double)partial[(size_t)r * 2 * d + col];
  }
  sh[y][lane] = v;
  __syncthreads();
  // Warp y adds column y.
  v = sh[lane][y];
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  const int mine = blockIdx.x * 32 + y;
  if (lane == 0 && mine < 2 * d) {
    float* out = mine < d ? dwq : dwk;
    if (out) out[mine < d ? mine : mine - d] = (float)v;
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
  if (tokens > (1 << 30) || n_q > (1 << 20) || n_k > (1 << 20)) return DA_ERR_UNSUPPORTED;
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

// Tokens of a CTA's batch (log2), for the fewest turns of the busiest CTA: a
// batch costs ceil(heads / groups of a token) turns and about half of one for
// its angles and coefficients.  More tokens share the threads of a CTA where there
// are few heads, and let a thread use its coefficients for more rows; fewer
// spread better over the GPU, and above `most` turns a batch nothing is gained
// (backward, 16384 tokens of 64 heads: 1, 4, 8 turns 118, 107, 110 us; forward,
// 40 heads: 5, 10, 20 turns 61, 57, 66 us).
int batch_log2(int tokens, int heads, int lanes, int rot, int most) {
  const int groups = kThreads / lanes;
  int best = 0;
  long long best_cost = 0;
  for (int lg = 0; (groups >> lg) >= 1 && ((rot / 2) << lg) <= kAngles; ++lg) {
    const int per_tok = groups >> lg;
    const long long batches = ((long long)tokens + (1 << lg) - 1) >> lg;
    const long long rounds = (batches + 148 * kCtasPerSm - 1) / (148 * kCtasPerSm);
    const int turns = (heads + per_tok - 1) / per_tok;
    const long long cost = rounds * (2 * turns + 1);
    if (lg == 0 || (turns <= most && cost < best_cost)) best = lg, best_cost = cost;
  }
  return best;
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
  a.tok_log2 = da::batch_log2(tokens, heads, lanes, rot_dim, 10);
  const int per_tok = (da::kThreads / lanes) >> a.tok_log2;
  const long long batches = ((long long)tokens + (1 << a.tok_log2) - 1) >> a.tok_log2;
  dim3 grid((unsigned)(batches < 148 * da::kCtasPerSm ? batches : 148 * da::kCtasPerSm), 1, 1);
  // Few tokens: a token's heads are split over CTAs too.
  const int turns = (heads + per_tok - 1) / per_tok;
  while (grid.y < (unsigned)turns && (long long)grid.x * grid.y < 148 * da::kCtasPerSm / 2) ++grid.y;
  if (grid.y > 65535u) grid.y = 65535u;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  auto run = [&](auto t, auto g, auto il, auto part) {
    e = da::launch_after(da::qk_norm_rope_kernel<decltype(t), decltype(g)::value,
                                                 decltype(il)::value, decltype(part)::value>,
                         grid, da::kThreads, 0, cs, a);
  };
  da::dispatch(dtype, lanes, interleaved != 0, [&](auto t, auto g, auto il) {
    if (rot_dim < head_dim) run(t, g, il, std::true_type{});
    else run(t, g, il, std::false_type{});
  });
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
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
  a.tok_log2 = da::batch_log2(tokens, heads, lanes, rot_dim, 4);
  const int batches = (int)(((long long)tokens + (1 << a.tok_log2) - 1) >> a.tok_log2);
  const int ctas = batches < da::kBwdCtas ? batches : da::kBwdCtas;
  const int per_tok = (da::kThreads / lanes) >> a.tok_log2;
  const long long rows = (long long)((batches + ctas - 1) / ctas) * ((heads + per_tok - 1) / per_tok);
  cudaError_t e = cudaSuccess;
  auto run = [&](auto t, auto g, auto il, auto many) {
    auto kernel = da::qk_norm_rope_bwd_kernel<decltype(t), decltype(g)::value,
                                              decltype(il)::value, decltype(many)::value>;
    const int bytes = da::bwd_smem_of<decltype(t)>(head_dim, decltype(many)::value);
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             da::bwd_smem_of<decltype(t)>(256, decltype(many)::value));
    if (e == cudaSuccess) e = da::launch_after(kernel, dim3(ctas), da::kThreads, bytes, cs, a);
  };
  da::dispatch(dtype, lanes, interleaved != 0, [&](auto t, auto g, auto il) {
    if (rows > da::kFoldRows) run(t, g, il, std::true_type{});
    else run(t, g, il, std::false_type{});
  });
  if (e != cudaSuccess) return DA_ERR_CUDA;
  if ((dq_weight || dk_weight) &&
      da::launch_after(da::qk_norm_dweight_kernel, dim3((2 * head_dim + 31) / 32), 1024, 0, cs,
                       a.partial, ctas, head_dim, dq_weight, dk_weight) != cudaSuccess)
    return DA_ERR_CUDA;
  return DA_OK;
}
