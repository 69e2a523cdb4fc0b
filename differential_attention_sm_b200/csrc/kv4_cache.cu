// kv4_cache.cu — writing rows into the 4-bit paged KV cache and reading them
// back (formats and layout: kv4.cuh).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "diffattn.h"
#include "kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;

struct CacheArgs {
  const void* k;  // rows in (append)
  const void* v;
  int64_t k_tok, v_tok;  // token strides in elements
  void* k_out;           // rows out (read), dense
  void* v_out;
  const int* slots;
  uint8_t* cache;
  int64_t n_slots;  // n_pages * page_size
  int tokens, heads, page_shift;
  int* dev_status;
};

// Sixteen consecutive channels as fp32.
__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = reinterpret_cast<const float4*>(p)[i];
    x[4 * i] = f.x;
    x[4 * i + 1] = f.y;
    x[4 * i + 2] = f.z;
    x[4 * i + 3] = f.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = bf16lo(u[j]);
      x[8 * i + 2 * j + 1] = bf16hi(u[j]);
    }
  }
}
__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] =
        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<uint4*>(p)[i] =
        make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                   pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
}

// Block scale: amax / 6 rounded to the nearest scale (ties to even).  The
// correctly rounded quotient decides as the exact one would: amax and 6 *
// (midpoint of two scales) are fp32 numbers, so unless they are equal they
// differ by an fp32 step of amax, which is more than the quotient's rounding.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return (uint32_t)kKv4BadScale;
  const float t = __fdiv_rn(__uint_as_float(amax_bits), 6.0f);
  uint32_t b;
  if (t < 6.103515625e-5f) {  // below 2^-14 the scales are multiples of 2^-17
    b = (uint32_t)__float2int_rn(t * 131072.0f);
  } else {
    uint32_t u = __float_as_uint(t);
    u += 0x7FFFFu + ((u >> 20) & 1u);
    b = (u >> 20) - ((127u - 15u) << 3);
  }
  return b > (uint32_t)kKv4MaxScale ? (uint32_t)kKv4MaxScale : b;
}

__device__ __forceinline__ uint8_t* tile_of(const CacheArgs& a, int slot, int head) {
  const int ps = 1 << a.page_shift;
  const int64_t page = slot >> a.page_shift;
  const int tile = (slot & (ps - 1)) >> 4;
  return a.cache + ((page * a.heads + head) * (ps >> 4) + tile) * kKv4TileBytes;
}

// One thread per block of 16 channels of a (token, head)'s K and V row.
// A code is x / scale rounded to the nearest level (ties to the even code).
// As above, the correctly rounded quotient falls on the same side of a border
// as the exact one: border * scale has 7 significant bits.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const CacheArgs a) {
  const int blk = threadIdx.x & 7;
  const int kv = (threadIdx.x >> 3) & 1;
  const unsigned th = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  const int tok = (int)(th / (unsigned)a.heads);
  if (tok >= a.tokens) return;
  const int head = (int)(th - (unsigned)tok * (unsigned)a.heads);
  const int slot = a.slots[tok];
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    report(a.dev_status, DA_ERR_PAGE);
    return;
  }
  float x[16];
  const T* src = kv ? static_cast<const T*>(a.v) + tok * a.v_tok
                    : static_cast<const T*>(a.k) + tok * a.k_tok;
  load16(src + head * kKv4Row + blk * 16, x);
  uint32_t amax = 0u;  // as bits: infinities and NaN order above every finite magnitude
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  const uint32_t sb = scale_byte(amax);
  const float s = kv4_scale_value(sb);
  uint32_t w[2] = {0u, 0u};
  if (sb != 0u && sb != (uint32_t)kKv4BadScale) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 2] |= f32x2_to_e2m1(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s))
                   << (8 * (i & 3));
  }
  uint8_t* tile = tile_of(a, slot, head);
  const int t = slot & 15;
  if (kv == 0) {
    *reinterpret_cast<uint2*>(tile + t * 64 + blk * 8) = make_uint2(w[0], w[1]);
    tile[kKv4KScales + 16 * (t & 7) + 4 * (blk >> 1) + 2 * (t >> 3) + (blk & 1)] = (uint8_t)sb;
  } else {
    *reinterpret_cast<uint2*>(tile + kKv4VCodes + 512 * (t >> 3) + 64 * blk +
                              16 * ((t & 7) >> 1) + 8 * (t & 1)) = make_uint2(w[0], w[1]);
    tile[kKv4VScales + 16 * blk + 4 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1)] = (uint8_t)sb;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const CacheArgs a) {
  const int blk = threadIdx.x & 7;
  const int kv = (threadIdx.x >> 3) & 1;
  const unsigned th = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  const int tok = (int)(th / (unsigned)a.heads);
  if (tok >= a.tokens) return;
  const int head = (int)(th - (unsigned)tok * (unsigned)a.heads);
  const int slot = a.slots[tok];
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    report(a.dev_status, DA_ERR_PAGE);
    return;
  }
  const uint8_t* tile = tile_of(a, slot, head);
  const int t = slot & 15;
  uint2 w;
  uint32_t sb;
  if (kv == 0) {
    w = *reinterpret_cast<const uint2*>(tile + t * 64 + blk * 8);
    sb = tile[kKv4KScales + 16 * (t & 7) + 4 * (blk >> 1) + 2 * (t >> 3) + (blk & 1)];
  } else {
    w = *reinterpret_cast<const uint2*>(tile + kKv4VCodes + 512 * (t >> 3) + 64 * blk +
                                        16 * ((t & 7) >> 1) + 8 * (t & 1));
    sb = tile[kKv4VScales + 16 * blk + 4 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1)];
  }
  const float s = kv4_scale_value(sb);
  uint32_t h[8];
  e2m1x8_to_f16x2(w.x, h[0], h[1], h[2], h[3]);
  e2m1x8_to_f16x2(w.y, h[4], h[5], h[6], h[7]);
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
  T* dst = static_cast<T*>(kv ? a.v_out : a.k_out);
  store16(dst + ((int64_t)tok * a.heads + head) * kKv4Row + blk * 16, x);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks shared by both calls; returns DA_OK, or the error.
int check(const int* slots, int tokens, int heads, int head_dim, const void* cache, int n_pages,
          int page_size, da_dtype dtype) {
  if (dtype != DA_BF16 && dtype != DA_FP32) return DA_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 1 || head_dim < 1 || n_pages < 1 || page_size < 1)
    return DA_ERR_INVALID_ARG;
  if (!cache || (tokens > 0 && !slots)) return DA_ERR_INVALID_ARG;
  if (head_dim != kKv4Row || !kv4_page_size_ok(page_size)) return DA_ERR_UNSUPPORTED;
  if ((long long)n_pages * page_size >= (1LL << 31)) return DA_ERR_UNSUPPORTED;
  if ((long long)tokens * heads >= (1LL << 31)) return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

unsigned blocks_for(int tokens, int heads) {
  return (unsigned)(((long long)tokens * heads * 16 + kThreads - 1) / kThreads);
}

}  // namespace
}  // namespace da

using da::CacheArgs;

extern "C" size_t diffattn_kv4_page_bytes(int n_kv_heads, int head_dim, int page_size) {
  if (n_kv_heads < 1 || head_dim != da::kKv4Row || page_size < 1 ||
      !da::kv4_page_size_ok(page_size))
    return 0;
  return (size_t)n_kv_heads * (page_size / da::kKv4Tile) * da::kKv4TileBytes;
}

extern "C" int diffattn_kv4_append(const void* k, long long k_token_stride, const void* v,
                                   long long v_token_stride, da_dtype dtype, const int* slots,
                                   int tokens, int n_kv_heads, int head_dim, void* cache,
                                   int n_pages, int page_size, int* dev_status, void* stream) {
  const int st = da::check(slots, tokens, n_kv_heads, head_dim, cache, n_pages, page_size, dtype);
  if (st != DA_OK) return st;
  if (tokens == 0) return DA_OK;
  if (!k || !v) return DA_ERR_INVALID_ARG;
  const long long row = (long long)n_kv_heads * head_dim;
  if (k_token_stride < row || v_token_stride < row) return DA_ERR_INVALID_ARG;
  const int per16 = dtype == DA_BF16 ? 8 : 4;
  if (k_token_stride % per16 || v_token_stride % per16) return DA_ERR_ALIGNMENT;
  if (!da::aligned16(k) || !da::aligned16(v) || !da::aligned16(cache)) return DA_ERR_ALIGNMENT;
  CacheArgs a{};
  a.k = k;
  a.v = v;
  a.k_tok = k_token_stride;
  a.v_tok = v_token_stride;
  a.slots = slots;
  a.cache = static_cast<uint8_t*>(cache);
  a.n_slots = (int64_t)n_pages * page_size;
  a.tokens = tokens;
  a.heads = n_kv_heads;
  a.page_shift = da::kv4_shift(page_size);
  a.dev_status = dev_status;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const unsigned grid = da::blocks_for(tokens, n_kv_heads);
  if (dtype == DA_BF16)
    da::kv4_append_kernel<__nv_bfloat16><<<grid, da::kThreads, 0, cs>>>(a);
  else
    da::kv4_append_kernel<float><<<grid, da::kThreads, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

extern "C" int diffattn_kv4_read(const void* cache, int n_pages, int page_size, const int* slots,
                                 int tokens, int n_kv_heads, int head_dim, void* k, void* v,
                                 da_dtype dtype, int* dev_status, void* stream) {
  const int st = da::check(slots, tokens, n_kv_heads, head_dim, cache, n_pages, page_size, dtype);
  if (st != DA_OK) return st;
  if (tokens == 0) return DA_OK;
  if (!k || !v) return DA_ERR_INVALID_ARG;
  if (!da::aligned16(k) || !da::aligned16(v) || !da::aligned16(cache)) return DA_ERR_ALIGNMENT;
  CacheArgs a{};
  a.k_out = k;
  a.v_out = v;
  a.slots = slots;
  a.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  a.n_slots = (int64_t)n_pages * page_size;
  a.tokens = tokens;
  a.heads = n_kv_heads;
  a.page_shift = da::kv4_shift(page_size);
  a.dev_status = dev_status;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const unsigned grid = da::blocks_for(tokens, n_kv_heads);
  if (dtype == DA_BF16)
    da::kv4_read_kernel<__nv_bfloat16><<<grid, da::kThreads, 0, cs>>>(a);
  else
    da::kv4_read_kernel<float><<<grid, da::kThreads, 0, cs>>>(a);
  return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}
