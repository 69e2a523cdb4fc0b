// kv4_cache.cu — writing rows into the 4-bit paged KV cache and reading them
// back (formats and layout: kv4.cuh).  Both are bound by memory: the rows
// (256 bytes of bf16 a token and head, K and V each) once, 72 bytes held once.
// Measured, 16383 tokens of 8 heads: append and read 33 us together, 0.79 of the
// copy rate; 64 tokens: 3.4 us both.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "diffattn.h"
#include "kernels.h"
#include "kv4.cuh"
#include "launch.cuh"
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

// Sixteen consecutive channels as they are held, and as fp32 pairs.
template <typename T>
struct Block {
  uint4 v[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Block<T> load_block(const T* p) {
  Block<T> b;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) b.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return b;
}
__device__ __forceinline__ void unpack(const Block<float>& b, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[4 * i] = __uint_as_float(b.v[i].x), x[4 * i + 1] = __uint_as_float(b.v[i].y);
    x[4 * i + 2] = __uint_as_float(b.v[i].z), x[4 * i + 3] = __uint_as_float(b.v[i].w);
  }
}
__device__ __forceinline__ void unpack(const Block<__nv_bfloat16>& b, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u[4] = {b.v[i].x, b.v[i].y, b.v[i].z, b.v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[8 * i + 2 * j] = bf16lo(u[j]), x[8 * i + 2 * j + 1] = bf16hi(u[j]);
  }
}
// Bits of the largest magnitude: infinities and NaN order above every number.
__device__ __forceinline__ uint32_t amax_bits(const Block<float>& b) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = max(max(m, max(b.v[i].x & 0x7FFFFFFFu, b.v[i].y & 0x7FFFFFFFu)),
            max(b.v[i].z & 0x7FFFFFFFu, b.v[i].w & 0x7FFFFFFFu));
  return m;
}
__device__ __forceinline__ uint32_t amax_bits(const Block<__nv_bfloat16>& b) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m = __vmaxu2(m, __vmaxu2(b.v[i].x & 0x7FFF7FFFu, b.v[i].y & 0x7FFF7FFFu));
    m = __vmaxu2(m, __vmaxu2(b.v[i].z & 0x7FFF7FFFu, b.v[i].w & 0x7FFF7FFFu));
  }
  return max(m << 16, m & 0xFFFF0000u);
}

// fp32 (a scale before its rounding, >= 0) to the nearest scale's byte, ties to
// even.
__device__ __forceinline__ uint32_t scale_byte(float t) {
  uint32_t b;
  if (t < 6.103515625e-5f) {  // below 2^-14 the scales are multiples of 2^-17
    b = (uint32_t)__float2int_rn(t * 131072.0f);
  } else {
    uint32_t u = __float_as_uint(t);
    u += 0x7FFFFu + ((u >> 20) & 1u);
    b = (u >> 20) - ((127u - 15u) << 3);
  }
  return min(b, (uint32_t)kKv4MaxScale);
}

// Quotients near enough that rounding them gives what rounding the exact ones
// gives.  A quotient on a border between two scales or levels belongs to an
// amax (x) of 7 significant bits: 6 * border has 7, border * scale 3 + 4.
//  bf16 rows (8 bits): whatever is not on a border is off it by 2^-9 of it or
//  more, so a product with the reciprocal (off by less than 2^-21 of itself)
//  is rounded to some 12 bits, which puts ties back on the border and moves
//  nothing across one.
//  fp32 rows: a value may be one step off a border.  The correctly rounded
//  quotient is on the border only if the exact one is, since the step is more
//  than half a step of the quotient.
__device__ __forceinline__ float sixth(float amax, const __nv_bfloat16*) {
  return __uint_as_float((__float_as_uint(amax * (1.0f / 6.0f)) + 0x400u) & 0xFFFFF800u);
}
__device__ __forceinline__ float sixth(float amax, const float*) { return __fdiv_rn(amax, 6.0f); }

// Sixteen codes of a block with scale s, 8 bytes.
__device__ __forceinline__ uint2 codes_of(const Block<__nv_bfloat16>& b, float s) {
  float x[16];
  unpack(b, x);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  constexpr float kAway = 1.5f * 2048.0f;  // its neighbours are 2^-12 apart
  const uint64_t inv2 = f2pack(inv, inv), up = f2pack(kAway, kAway), down = f2pack(-kAway, -kAway);
  float y[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // to multiples of 2^-12
    uint64_t v = fma2(f2pack(x[2 * i], x[2 * i + 1]), inv2, f2pack(-0.f, -0.f));
    v = add2(add2(v, up), down);
    f2unpack(v, y[2 * i], y[2 * i + 1]);
  }
  return make_uint2(f32x8_to_e2m1(y), f32x8_to_e2m1(y + 8));
}
__device__ __forceinline__ uint2 codes_of(const Block<float>& b, float s) {
  float x[16];
  unpack(b, x);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], s);
  return make_uint2(f32x8_to_e2m1(x), f32x8_to_e2m1(x + 8));
}

// Work of both kernels: a CTA takes 16 tokens and walks over the KV heads.
// A warp has 8 tokens and 4 of the 8 blocks of a row of K or of V, so that 4
// lanes read 128 bytes in a row and, where the 8 tokens lie in a row of slots,
// the codes of V are written 64 bytes in a row.
constexpr int kTokens = 16;

struct Lane {
  int tok, blk, t;   // token, block, place in the tile
  bool is_v;
  uint32_t codes, scale;  // bytes of the tile
  uint8_t* tile;     // of KV head 0
  int64_t head_bytes;
  __device__ __forceinline__ Lane() {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    is_v = warp & 1;
    blk = 4 * ((warp >> 1) & 1) + (lane & 3);
    tok = (int)blockIdx.x * kTokens + 8 * (warp >> 2) + (lane >> 2);
  }
  // Where the token is held; false if there is nothing to do for it.
  __device__ __forceinline__ bool find(const CacheArgs& a, int slot) {
    if (slot < 0) return false;
    if (slot >= a.n_slots) {
      report(a.dev_status, DA_ERR_PAGE);
      return false;
    }
    const int sh = a.page_shift - 4;
    const int64_t page = slot >> a.page_shift;
    const int in_page = (slot >> 4) & ((1 << sh) - 1);
    head_bytes = (int64_t)kKv4TileBytes << sh;
    tile = a.cache + page * a.heads * head_bytes + in_page * kKv4TileBytes;
    t = slot & 15;
    codes = is_v ? kKv4VCodes + 512 * (t >> 3) + 64 * blk + 16 * ((t & 7) >> 1) + 8 * (t & 1)
                 : t * 64 + blk * 8;
    scale = is_v ? kKv4VScales + 16 * blk + 4 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1)
                 : kKv4KScales + 16 * (t & 7) + 4 * (blk >> 1) + 2 * (t >> 3) + (blk & 1);
    return true;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const CacheArgs a) {
  let_next_start();
  after_previous();
  Lane w;
  if (w.tok >= a.tokens) return;
  const T* src = (w.is_v ? static_cast<const T*>(a.v) + w.tok * a.v_tok
                         : static_cast<const T*>(a.k) + w.tok * a.k_tok) + w.blk * 16;
  const int slot = a.slots[w.tok];
  int h = blockIdx.y;
  Block<T> next = load_block(src + (int64_t)h * kKv4Row);  // not held up by the slot
  if (!w.find(a, slot)) return;
  for (; h < a.heads; h += gridDim.y) {
    const Block<T> b = next;
    if (h + (int)gridDim.y < a.heads)
      next = load_block(src + (int64_t)(h + gridDim.y) * kKv4Row);
    const uint32_t top = amax_bits(b);
    const uint32_t sb = top >= 0x7F800000u
                            ? (uint32_t)kKv4BadScale
                            : scale_byte(sixth(__uint_as_float(top), (const T*)nullptr));
    uint2 c = make_uint2(0u, 0u);
    if (sb != 0u && sb != (uint32_t)kKv4BadScale) c = codes_of(b, kv4_scale_value(sb));
    uint8_t* tile = w.tile + h * w.head_bytes;
    *reinterpret_cast<uint2*>(tile + w.codes) = c;
    tile[w.scale] = (uint8_t)sb;
  }
}

// 32 bytes in one store (kWide: p is a multiple of 32), or in two: a store of
// every other 16 bytes leaves half of each sector to the next one (reading
// 16383 tokens of 8 heads: 23 us for 15).
template <bool kWide>
__device__ __forceinline__ void store32(void* p, const uint32_t (&u)[8]) {
  if (kWide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]),
                 "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    static_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}
template <bool kWide>
__device__ __forceinline__ void store_block(float* p, const uint32_t (&h)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[4 * i + j]));
      u[2 * j] = __float_as_uint(f.x), u[2 * j + 1] = __float_as_uint(f.y);
    }
    store32<kWide>(p + 8 * i, u);
  }
}
template <bool kWide>
__device__ __forceinline__ void store_block(__nv_bfloat16* p, const uint32_t (&h)[8]) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    u[i] = pack_bf16(f.x, f.y);
  }
  store32<kWide>(p, u);
}

template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const CacheArgs a) {
  constexpr int kAtOnce = 4;  // heads asked for together
  let_next_start();
  after_previous();
  Lane w;
  if (w.tok >= a.tokens || !w.find(a, a.slots[w.tok])) return;
  T* dst = static_cast<T*>(w.is_v ? a.v_out : a.k_out) + (int64_t)w.tok * a.heads * kKv4Row +
           w.blk * 16;
  const int step = (int)gridDim.y;
  for (int h0 = blockIdx.y; h0 < a.heads; h0 += kAtOnce * step) {
    uint2 c[kAtOnce];
    uint32_t s[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int h = h0 + k * step;
      c[k] = make_uint2(0u, 0u), s[k] = 0u;
      if (h < a.heads) {
        const uint8_t* tile = w.tile + h * w.head_bytes;
        c[k] = *reinterpret_cast<const uint2*>(tile + w.codes);
        s[k] = tile[w.scale];
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int h = h0 + k * step;
      if (h >= a.heads) break;
      const uint32_t s2 = (s[k] << 7) * 0x10001u;  // the scale twice, fp16
      uint32_t x[8];
      e2m1x8_to_f16x2(c[k].x, x[0], x[1], x[2], x[3]);
      e2m1x8_to_f16x2(c[k].y, x[4], x[5], x[6], x[7]);
#pragma unroll
      for (int i = 0; i < 8; ++i)  // exact in fp16
        asm("mul.f16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(s2));
      store_block<kWide>(dst + (int64_t)h * kKv4Row, x);
    }
  }
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

// Heads are walked by a CTA where there are CTAs enough for the GPU without
// (a thread's next row is then in flight while it packs this one), and spread
// over CTAs otherwise.  16383 tokens of 8 heads, append and read, with at least
// 888, 1776, 3552, 7104 CTAs: 41, 37, 37, 41 us.
dim3 grid_for(int tokens, int heads) {
  dim3 g((unsigned)((tokens + kTokens - 1) / kTokens), 1, 1);
  while ((int)g.y < heads && (long long)g.x * g.y < 148 * 12 && g.y < 65535u) ++g.y;
  return g;
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
  const dim3 grid = da::grid_for(tokens, n_kv_heads);
  const auto kernel = dtype == DA_BF16 ? da::kv4_append_kernel<__nv_bfloat16>
                                       : da::kv4_append_kernel<float>;
  return da::launch_after(kernel, grid, da::kThreads, 0, cs, a) == cudaSuccess ? DA_OK
                                                                               : DA_ERR_CUDA;
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
  const dim3 grid = da::grid_for(tokens, n_kv_heads);
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  const auto kernel = dtype == DA_BF16
                          ? (wide ? da::kv4_read_kernel<__nv_bfloat16, true>
                                  : da::kv4_read_kernel<__nv_bfloat16, false>)
                          : (wide ? da::kv4_read_kernel<float, true>
                                  : da::kv4_read_kernel<float, false>);
  return da::launch_after(kernel, grid, da::kThreads, 0, cs, a) == cudaSuccess ? DA_OK
                                                                               : DA_ERR_CUDA;
}
