// decode_kv4.cu — single-token differential attention over the paged 4-bit
// cache (format and layout: kv4.cuh), V2 and V1.
//
//   S = q k^T / sqrt(d), o = O1 / l1 - lambda O2 / l2 with O = sum p v, l = sum p,
//   p = 2^(s log2(e) - m), m a running reference maximum;  V1 then applies the
//   per-head norm.
//
// Bound by the cache's bytes: 144 per token and KV head, and close behind by
// the instructions that turn codes into operands.  So:
//  - The work is one line of stages (64 tokens of one KV head of one
//    sequence), computed from the lengths on the device and cut into equal
//    runs, one for each warp of the grid: no lengths on the host, no idle
//    warps behind ragged lengths, no synchronisation between warps.
//  - Each warp keeps a ring of stages in shared memory filled by bulk copies
//    (a page is contiguous, so a stage is one copy), which holds enough bytes
//    in flight for the memory's latency.
//  - The matrix instruction is m16n8k16 in fp16 with the cache as its 16-row
//    operand: tokens x channels for the scores, channels x tokens for the
//    values, the (at most 8) query heads as columns.  code * scale is exact in
//    fp16, so the cache's values enter unrounded.  The layout gives every lane
//    its own operand pieces: codes become fp16 pairs in its registers and
//    never pass through shared memory again.  (tcgen05 would want them
//    written back to shared or tensor memory first, and 16 columns at least;
//    its rate is not what is missing here.)
//  - q is scaled by a power of two per head into fp16's range: exact down to
//    2^-17 of the head's largest feature; what is smaller is rounded, by 2^-25
//    of the largest at most.  p is rounded to fp16 (half a step is 2^-11 of a
//    probability), the sums l (of the unrounded p) and O are fp32.  m moves only
//    when a score passes it by more than 2^10, so p reaches 2^15 at most and the
//    common stage needs no maximum across lanes.
// A run leaves (O, l, m) of each sequence and head that it touches in the
// workspace; a second kernel joins them, subtracts, and normalises.
//
// Measured, 64 sequences of 32768 entries, 8 KV heads, 64 query heads (2.4 GB):
// 377 to 387 us in bursts at 1965 MHz, 0.95 to 0.98 of the copy rate (the copies
// alone 363); 450 to 475 us when the board's power limit sets the clock (1550 MHz
// at 995 W).  V1, 16 x 8191 x 32 heads (0.6 GB): 108 to 120 us.
// A tile and head costs 238 instructions: 64 conversions, 64 multiplications
// and 16 matrix instructions, which hold the former two up for 7 of their 8
// clocks, make 285 of about 400 clocks of an SM quarter, where the memory
// allows 405 at 1965 MHz.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "diffattn.h"
#include "kernels.h"
#include "kv4.cuh"
#include "kv4_index.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kD = 128;
constexpr int kTiles = 4;  // of a stage
constexpr int kStageTokens = kTiles * kKv4Tile;
constexpr int kStageBytes = kTiles * kKv4TileBytes;
// Warps of a CTA, one CTA an SM (3 of 4 warps took 104 us for 101: V1, 16 x 8191).
// Two column tiles need 235 registers a thread: 8 warps, where 12 with 168 spill
// (32 sequences of 8192 entries, 80 query heads on 8: 84 us for 91; with one
// tile 8 warps take 66 us for 63).
__host__ __device__ constexpr int warps_of(int tiles) { return tiles == 1 ? 12 : 8; }
constexpr int kRing = 2;
constexpr int kPlanSms = 148;      // fixed: the workspace size is the same on every device
constexpr int kMinStages = 1;      // shortest run of a warp
constexpr int kChunkHeads = 16;    // query heads that share one pass over the cache
constexpr float kNoMax = -3.0e38f;
constexpr float kShift = 5.0f;    // p = 2^(s - m + kShift)
constexpr float kRaise = 10.0f;   // m is raised when a score passes m + kRaise

struct Kv4Args {
  const __nv_bfloat16* q;  // [batch][q_heads][128]
  const uint8_t* cache;
  const int* table;  // [batch][max_pages]
  const int* lens;
  int batch, heads, group, chunks;  // KV heads; query columns of one; passes over one
  int max_pages, page_shift, n_pages, window;
  float scale;  // log2(e) / sqrt(d)
  int runs;     // warps of the grid
  int cols;     // columns kept per slot
  float* part_o;   // [slot][cols][128]
  float* part_ml;  // [slot][cols][2]
  int2* spans;     // [batch][units]: first run and segments of a unit, or null
  int* dev_status;
  // combine
  const float* lambda;
  __nv_bfloat16* out;
  int out_heads, v1, apply_norm;
  const float* gain;
  float eps, post_scale;
};

__host__ __device__ constexpr int smem_of(int tiles) { return warps_of(tiles) * kRing * (kStageBytes + 16); }

__device__ __forceinline__ void span_of(const Kv4Args& a, int b, int& lo, int& len) {
  const long long room = (long long)a.max_pages << a.page_shift;
  len = a.lens[b];
  len = len < 0 ? 0 : (len > room ? (int)room : len);
  lo = a.window > 0 && len > a.window ? len - a.window : 0;
}
__device__ __forceinline__ int stages_of(const Kv4Args& a, int b) {
  int lo, len;
  span_of(a, b, lo, len);
  return len > lo ? (len - 1) / kStageTokens - lo / kStageTokens + 1 : 0;
}

// Stages of one (KV head, pass) of the sequences before b, and of all; the
// whole warp calls it.
__device__ __forceinline__ void stage_sums(const Kv4Args& a, int b, long long& before,
                                           long long& total) {
  before = total = 0;
  for (int i = (int)lane_id(); i < a.batch; i += 32) {
    const int n = stages_of(a, i);
    total += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, off);
    total += __shfl_xor_sync(0xffffffffu, total, off);
  }
}

// x / y for x >= 0, y > 0; nearly always of 32 bits, where it costs a fifth.
__device__ __forceinline__ long long divide(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (long long)((uint32_t)x / (uint32_t)y);
  return x / y;
}

__device__ __forceinline__ long long run_length(const Kv4Args& a, long long total) {
  const long long q = divide(total + a.runs - 1, a.runs);
  return q < kMinStages ? kMinStages : q;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// Both halves of x times the low (high) half of y.
__device__ __forceinline__ uint32_t hmul2_lo(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 d;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 d, {l, l};\n\t"
      "mul.f16x2 %0, %1, d;\n\t}"
      : "=r"(r)
      : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t hmul2_hi(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 d;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 d, {h, h};\n\t"
      "mul.f16x2 %0, %1, d;\n\t}"
      : "=r"(r)
      : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                              uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint4 ldg128(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 P, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\t"
      "mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void bulk_to(uint32_t dst, const void* src, uint32_t bytes,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Scale bytes `i`, `i + 1` of w in the halves.
template <int i>
__device__ __forceinline__ uint32_t scale_pair(uint32_t w) {
  return __byte_perm(w, 0u, 0x0404u | (i << 4) | ((i + 1) << 12)) >> 1;
}

// One warp's state of a segment: NT column tiles of 8 query heads.
template <int NT>
struct WarpState {
  float o[NT][8][4];  // channels 16 * (lane / 4) + 2 * i, + 1; columns 2 * (lane % 4), + 1
  float l[NT][2], m[NT][2];
  float off[NT][2];  // kShift - m
  float top[NT][2];  // the unscaled score above which m is raised
};

// The scores of two tiles: c[t][n] holds tokens g, g + 8 of tile t, columns 2q,
// 2q + 1.  The tiles are taken turn and turn about, so that neither waits for
// its own last product.
template <int NT>
__device__ __forceinline__ void pair_scores(uint32_t at, uint32_t lane,
                                            const uint32_t (&qf)[NT][16], float (&c)[2][NT][4]) {
  uint32_t w0[2][4], w1[2][4], s[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const uint4 k0 = lds128(at + t * kKv4TileBytes + lane * 16),
                k1 = lds128(at + t * kKv4TileBytes + 512 + lane * 16);
    const uint32_t sw = lds32(at + t * kKv4TileBytes + kKv4KScales + lane * 4);
    w0[t][0] = k0.x, w0[t][1] = k0.y, w0[t][2] = k0.z, w0[t][3] = k0.w;
    w1[t][0] = k1.x, w1[t][1] = k1.y, w1[t][2] = k1.z, w1[t][3] = k1.w;
    // Tokens (g, g + 8) of the lane's even and of its odd block.
    s[t][0] = (sw << 7) & 0x7F807F80u;
    s[t][1] = (sw >> 1) & 0x7F807F80u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a[2][4], b[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      e2m1x8_to_f16x2(w0[t][i], a[t][0], a[t][1], a[t][2], a[t][3]);
      e2m1x8_to_f16x2(w1[t][i], b[t][0], b[t][1], b[t][2], b[t][3]);
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t sc = s[t][i / 2];
        const uint32_t x0 = hmul2_lo(a[t][j], sc), x1 = hmul2_hi(b[t][j], sc);
        const uint32_t x2 = hmul2_lo(a[t][j + 1], sc), x3 = hmul2_hi(b[t][j + 1], sc);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (i == 0 && j == 0)
            mma_f16_first(c[t][n], x0, x1, x2, x3, qf[n][0], qf[n][1]);
          else
            mma_f16(c[t][n], x0, x1, x2, x3, qf[n][4 * i + j], qf[n][4 * i + j + 1]);
        }
      }
  }
}

// Adds sixteen tokens' values: p[nt] are the operand's two registers.  `seen`
// masks the scales of tokens that take no part (all ones for a whole tile): a
// row behind the end may hold anything, and 0 * NaN is not 0.
template <int NT>
__device__ __forceinline__ void tile_values(uint32_t at, uint32_t lane, uint32_t seen0,
                                            uint32_t seen1, const uint32_t (&p)[NT][2],
                                            float (&o)[NT][8][4]) {
  const uint4 v0 = lds128(at + kKv4VCodes + lane * 16),
              v1 = lds128(at + kKv4VCodes + 512 + lane * 16);
  const uint32_t sw = lds32(at + kKv4VScales + lane * 4);
  const uint32_t s0 = scale_pair<0>(sw) & seen0, s1 = scale_pair<2>(sw) & seen1;
  constexpr uint32_t kLow = 0x0F0F0F0Fu;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t x0 = half ? v0.y : v0.x, z0 = half ? v0.w : v0.z;
    const uint32_t x1 = half ? v1.y : v1.x, z1 = half ? v1.w : v1.z;
    // Bytes of (channel, channel + 1) of two tokens become bytes of (token,
    // token + 1) of two channels.
    uint32_t e0[4], d0[4], e1[4], d1[4];
    e2m1x8_to_f16x2((x0 & kLow) | ((z0 << 4) & ~kLow), e0[0], e0[1], e0[2], e0[3]);
    e2m1x8_to_f16x2(((x0 >> 4) & kLow) | (z0 & ~kLow), d0[0], d0[1], d0[2], d0[3]);
    e2m1x8_to_f16x2((x1 & kLow) | ((z1 << 4) & ~kLow), e1[0], e1[1], e1[2], e1[3]);
    e2m1x8_to_f16x2(((x1 >> 4) & kLow) | (z1 & ~kLow), d1[0], d1[1], d1[2], d1[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a0 = hmul2(e0[i], s0), a1 = hmul2(d0[i], s0), a2 = hmul2(e1[i], s1),
                     a3 = hmul2(d1[i], s1);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * half + i], a0, a1, a2, a3, p[n][0], p[n][1]);
    }
  }
}

template <int NT, bool kV1>
__global__ void __launch_bounds__(warps_of(NT) * 32, 1) kv4_decode_kernel(const Kv4Args a) {
  constexpr int kWarps = warps_of(NT);
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t lane = threadIdx.x & 31u;
  const int warp = (int)(threadIdx.x >> 5);
  const uint32_t g = lane >> 2, qd = lane & 3u;
  const uint32_t ring_at = smem_u32(smem) + warp * kRing * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * kRing * kStageBytes) + warp * kRing;
  const uint32_t bars_at = smem_u32(bars);
  uint32_t* loaded = reinterpret_cast<uint32_t*>(smem + kWarps * kRing * (kStageBytes + 8)) +
                     warp * kRing;  // which tiles of a ring slot hold tokens
  if (lane == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  after_previous();
  let_next_start();  // not sooner: kv4_combine_kernel reads the lengths before its own wait

  const int units = a.heads * a.chunks;  // of one sequence
  long long before, total;
  stage_sums(a, 0, before, total);
  total *= units;
  const long long run = run_length(a, total);
  // Neighbouring runs lie on different SMs.
  const int me = warp * (int)gridDim.x + (int)blockIdx.x;
  long long pos = run * me;
  const long long end = pos + run < total ? pos + run : total;
  if (pos >= end) return;

  // The sequence that holds `pos`.
  int b = 0, n_b = 0;
  long long base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int mine = b0 + (int)lane < a.batch ? stages_of(a, b0 + (int)lane) : 0;
    long long upto = (long long)mine * units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, off);
      if ((int)lane >= off) upto += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + upto > pos);
    if (past) {
      const int src = __ffs(past) - 1;
      b = b0 + src;
      n_b = __shfl_sync(0xffffffffu, mine, src);
      base += __shfl_sync(0xffffffffu, upto, src) - (long long)n_b * units;
      break;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
  }

  int slot = 0;          // next ring slot
  uint32_t parity = 0;   // of that slot
  while (pos < end) {
    const int unit = (int)divide(pos - base, n_b);
    const int s_first = (int)((pos - base) - (long long)unit * n_b);
    const int count = (int)(end - pos < n_b - s_first ? end - pos : n_b - s_first);
    const int kvh = unit / a.chunks, chunk = unit - kvh * a.chunks;
    int lo, len;
    span_of(a, b, lo, len);
    const int s0 = lo / kStageTokens + s_first;  // absolute stage

    // The segment's queries: column g of column tile n, channels 32 * qd ...  They
    // are asked for before the copies, which would hold them up for 3 us when
    // all warps start at once.
    uint32_t qf[NT][16];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = chunk * kChunkHeads + n * 8 + (int)g;
      bool live = col < a.group;
      const __nv_bfloat16* src;
      if (kV1) {  // column 0 has features 0..63 of the head, column 1 the rest
        src = a.q + ((size_t)b * a.heads + kvh) * kD + 32 * qd;
        live = live && (g == qd / 2);
      } else {
        src = a.q + ((size_t)b * a.heads * a.group + (size_t)kvh * a.group + col) * kD + 32 * qd;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (live) u = ldg128(src + 8 * i);
        qf[n][4 * i] = u.x, qf[n][4 * i + 1] = u.y, qf[n][4 * i + 2] = u.z, qf[n][4 * i + 3] = u.w;
      }
    }
    // The next 32 tiles (8 stages) of the segment, one per lane, and the 32
    // behind them.
    const int* row = a.table + (size_t)b * a.max_pages;
    const int first_tile = lo >> 4, last_tile = min((len - 1) >> 4, kTiles * (s0 + count) - 1);
    const int sh = a.page_shift - 4;
    auto tile_of = [&](int at) -> uint32_t {  // index in the cache of the segment's tile `at`
      const int t = kTiles * s0 + at;
      if (t < first_tile || t > last_tile) return kNoTile;
      const int page = row[t >> sh];
      if ((unsigned)page >= (unsigned)a.n_pages) return kBadTile;
      return (((uint32_t)page * (uint32_t)a.heads + (uint32_t)kvh) << sh) +
             (uint32_t)(t & ((1 << sh) - 1));
    };
    // Bit l: the tiles of lanes l and l + 1 are neighbours in memory.
    auto joined = [&](uint32_t mine) {
      const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
      return __ballot_sync(0xffffffffu, tiles_joined(mine, next));
    };
    uint32_t tile = tile_of((int)lane), ahead = tile_of(32 + (int)lane);
    uint32_t join = joined(tile);
    auto issue = [&](int i, int to) {  // stage i of the segment into ring slot `to`
      const uint32_t lead = (uint32_t)(i & 7) * kTiles;
      const uint32_t dst = ring_at + to * kStageBytes, bar = bars_at + to * 8;
      if (((join >> lead) & 7u) == 7u) {
        if (lane == lead) {
          loaded[to] = 15u;
          expect(bar, kStageBytes);
          bulk_to(dst, a.cache + (uint64_t)tile * kKv4TileBytes, kStageBytes, bar);
        }
      } else {
        const bool mine = lane - lead < (uint32_t)kTiles;
        const bool ok = mine && tile < kBadTile;
        const uint32_t have = __ballot_sync(0xffffffffu, ok) >> lead;
        if (mine && tile == kBadTile) report(a.dev_status, DA_ERR_PAGE);
        if (lane == lead) {
          loaded[to] = have;
          expect(bar, __popc(have) * kKv4TileBytes);
        }
        __syncwarp();
        if (ok)
          bulk_to(dst + (lane - lead) * kKv4TileBytes, a.cache + (uint64_t)tile * kKv4TileBytes,
                  kKv4TileBytes, bar);
      }
    };
    int issued = 0;
    for (int to = slot; issued < kRing && issued < count; ++issued) {
      issue(issued, to);
      if (++to == kRing) to = 0;
    }

    // Query fragments, from what was asked for above.
    float back[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t(&raw)[16] = qf[n];
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        top = max(top, max((raw[i] << 16) & 0x7F800000u, raw[i] & 0x7F800000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // q * 2^-e is in fp16's range with e the largest exponent of the head.
      // An exponent of 0 or of infinities is replaced: the products are 0 or
      // not numbers either way.
      const uint32_t e = min(max(top >> 23, 1u), 253u);
      const float down = __uint_as_float((254u - e) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        raw[i] = pack_f16(bf16lo(raw[i]) * down, bf16hi(raw[i]) * down);
      // A head with an infinity has scores that are infinite or NaN, and no
      // softmax: NaN, where scores of -infinity alone would pass for masked ones.
      if (top >= 0x7F800000u) raw[0] = 0x7FFF7FFFu;
      // Positive, so that it can multiply a masked score's infinity; scores
      // that this floor touches are 0 to any precision here.
      const float up = fmaxf(__uint_as_float(e << 23) * a.scale, 1.0e-30f);
      back[n][0] = __shfl_sync(0xffffffffu, up, 8 * qd);
      back[n][1] = __shfl_sync(0xffffffffu, up, 8 * qd + 4);
    }

    WarpState<NT> w;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) w.o[n][i][j] = 0.f;
      w.l[n][0] = w.l[n][1] = 0.f;
      w.m[n][0] = w.m[n][1] = kNoMax;
      w.off[n][0] = w.off[n][1] = kShift - kNoMax;
      w.top[n][0] = w.top[n][1] = kNoMax;
    }

    for (int i = 0; i < count; ++i) {
      if (!__all_sync(0xffffffffu, try_wait(bars_at + slot * 8, parity))) {
        bool failed = false;
        mbar_wait(&bars[slot], parity, a.dev_status, &failed);
        if (__any_sync(0xffffffffu, failed)) {
          // Leave no copy of ours in flight: wait for the other slots, bounded too.
          for (int k = i + 1; k < issued; ++k) {
            if (++slot == kRing) slot = 0, parity ^= 1u;
            failed = false;
            mbar_wait(&bars[slot], parity, a.dev_status, &failed);
          }
          return;
        }
      }
      const uint32_t have = loaded[slot];
      const int first_tok = (s0 + i) * kStageTokens;
      const bool part = have != 15u || first_tok < lo || len - first_tok < kStageTokens;
#pragma unroll
      for (int pair = 0; pair < kTiles / 2; ++pair) {
        const uint32_t at = ring_at + slot * kStageBytes + pair * 2 * kKv4TileBytes;
        float c[2][NT][4];
        pair_scores<NT>(at, lane, qf, c);
        uint32_t seen[2][2] = {{~0u, ~0u}, {~0u, ~0u}};
        if (part) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const bool there = (have >> (2 * pair + t)) & 1u;
            auto sees = [&](int u) {
              const int tok = first_tok + 32 * pair + 16 * t + u;
              return there && tok >= lo && tok < len;
            };
            const bool r0 = sees((int)g), r1 = sees((int)g + 8);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (!r0) c[t][n][0] = c[t][n][1] = -INFINITY;
              if (!r1) c[t][n][2] = c[t][n][3] = -INFINITY;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
              seen[t][h] = (sees(2 * (int)qd + 8 * h) ? 0xFFFFu : 0u) |
                           (sees(2 * (int)qd + 8 * h + 1) ? 0xFFFF0000u : 0u);
          }
        }
        float mx[NT][2];
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mx[n][j] = fmaxf(max3(c[0][n][j], c[0][n][j + 2], c[1][n][j]), c[1][n][j + 2]);
            raise |= mx[n][j] > w.top[n][j];
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float top = mx[n][j];
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              top = fmaxf(top * back[n][j], w.m[n][j]);
              const float f = ex2(w.m[n][j] - top);
              w.m[n][j] = top;
              w.off[n][j] = kShift - top;
              w.top[n][j] = top > kNoMax ? (top + kRaise) / back[n][j] : kNoMax;
              w.l[n][j] *= f;
#pragma unroll
              for (int k = 0; k < 8; ++k) w.o[n][k][j] *= f, w.o[n][k][j + 2] *= f;
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t p[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float p0 = ex2(fmaf(c[t][n][0], back[n][0], w.off[n][0])),
                        p1 = ex2(fmaf(c[t][n][1], back[n][1], w.off[n][1])),
                        p2 = ex2(fmaf(c[t][n][2], back[n][0], w.off[n][0])),
                        p3 = ex2(fmaf(c[t][n][3], back[n][1], w.off[n][1]));
            w.l[n][0] += p0 + p2;
            w.l[n][1] += p1 + p3;
            p[n][0] = movmatrix_trans(pack_f16(p0, p1));
            p[n][1] = movmatrix_trans(pack_f16(p2, p3));
          }
          tile_values<NT>(at + t * kKv4TileBytes, lane, seen[t][0], seen[t][1], p, w.o);
        }
      }
      __syncwarp();  // every lane has read the slot
      if (issued < count) {
        if ((issued & 7) == 0) {
          tile = ahead;
          join = joined(tile);
          ahead = tile_of(kTiles * (issued + 8) + (int)lane);
        }
        issue(issued, slot);
        ++issued;
      }
      if (++slot == kRing) slot = 0, parity ^= 1u;
    }

    if (a.spans && s_first == 0 && lane == 0) {
      const long long last = pos + n_b - 1;  // of the unit
      a.spans[(size_t)b * units + unit] = make_int2(me, (int)divide(last, run) - me + 1);
    }
    // The segment's sums.  Slots are ordered as the segments are: the next
    // segment has the next unit or the next run.
    const long long part = (long long)b * units + unit + me;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float l = w.l[n][j];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int col = n * 8 + 2 * (int)qd + j;
        if (col < a.cols) {
          float* dst = a.part_o + (part * a.cols + col) * kD + 16 * g;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(dst)[i] =
                make_float4(w.o[n][2 * i][j], w.o[n][2 * i][j + 2], w.o[n][2 * i + 1][j],
                            w.o[n][2 * i + 1][j + 2]);
          if (g == 0) {
            float* ml = a.part_ml + (part * a.cols + col) * 2;
            ml[0] = w.m[n][j];
            ml[1] = l;
          }
        }
      }
    pos += count;
    while (pos < end && pos >= base + (long long)n_b * units) {
      base += (long long)n_b * units;
      n_b = stages_of(a, ++b);
    }
  }
}

// One CTA per output head: its warps take the segments of the two columns in
// turn, four at a time (so that up to 16 segments cost one trip to memory),
// and the first warp joins what they found.
constexpr int kCombineWarps = 4;
constexpr int kAtOnce = 4;

__global__ void __launch_bounds__(kCombineWarps * 32) kv4_combine_kernel(const Kv4Args a) {
  __shared__ float4 sh_o[kCombineWarps][2][32];
  __shared__ float4 sh_ml[kCombineWarps];
  const int lane = (int)(threadIdx.x & 31), warp = (int)(threadIdx.x >> 5);
  const int b = (int)(blockIdx.x / (unsigned)a.out_heads);
  const int p = (int)blockIdx.x - b * a.out_heads;
  int unit, col;
  if (a.v1) {
    unit = p;
    col = 0;
  } else {
    const int kvh = 2 * p / a.group, at = 2 * p - kvh * a.group;
    unit = kvh * a.chunks + at / kChunkHeads;
    col = at % kChunkHeads;
  }
  // The lengths (a.lens) are read before after_previous(), which hides the sums
  // behind the end of the decode.  Whatever wrote them is done: only
  // kv4_decode_kernel is launched before this kernel, it lets this one start
  // behind its own wait, and it does not write them.  It has to stay so.
  const int units = a.heads * a.chunks;
  const int n_b = stages_of(a, b);
  int w0 = 0, n = 0;  // first run, and segments
  if (!a.spans) {
    long long before, total;
    stage_sums(a, b, before, total);
    const long long run = run_length(a, total * units);
    const long long start = before * units + (long long)unit * n_b;
    w0 = (int)divide(start, run);
    n = n_b > 0 ? (int)divide(start + n_b - 1, run) - w0 + 1 : 0;
  }
  after_previous();
  if (a.spans && n_b > 0) {
    const int2 v = a.spans[(size_t)b * units + unit];
    w0 = v.x, n = v.y;
    bound_span(w0, n, a.runs);
  }
  const long long slot0 = (long long)b * units + unit + w0;
  const float* ml = a.part_ml + (slot0 * a.cols + col) * 2;
  const float* po = a.part_o + (slot0 * a.cols + col) * kD + 4 * lane;
  const int64_t ml_step = 2 * a.cols, po_step = (int64_t)a.cols * kD;
  const float lam = a.lambda[p];
  float gain[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) gain[i] = a.gain ? a.gain[4 * lane + i] : 1.f;
  float m[2] = {kNoMax, kNoMax}, l[2] = {0.f, 0.f}, o[2][4] = {};
  for (int s0 = warp; s0 < n; s0 += kCombineWarps * kAtOnce) {
    float4 v[kAtOnce], x[kAtOnce], y[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int s = s0 + k * kCombineWarps;
      v[k] = make_float4(kNoMax, 0.f, kNoMax, 0.f);
      x[k] = y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < n) {
        v[k] = *reinterpret_cast<const float4*>(ml + s * ml_step);
        x[k] = *reinterpret_cast<const float4*>(po + s * po_step);
        y[k] = *reinterpret_cast<const float4*>(po + s * po_step + kD);
      }
    }
    const float old0 = m[0], old1 = m[1];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) m[0] = fmaxf(m[0], v[k].x), m[1] = fmaxf(m[1], v[k].z);
    const float g0 = ex2(old0 - m[0]), g1 = ex2(old1 - m[1]);
    l[0] *= g0, l[1] *= g1;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[0][i] *= g0, o[1][i] *= g1;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const float f0 = ex2(v[k].x - m[0]), f1 = ex2(v[k].z - m[1]);
      l[0] = fmaf(v[k].y, f0, l[0]), l[1] = fmaf(v[k].w, f1, l[1]);
      o[0][0] = fmaf(x[k].x, f0, o[0][0]), o[0][1] = fmaf(x[k].y, f0, o[0][1]);
      o[0][2] = fmaf(x[k].z, f0, o[0][2]), o[0][3] = fmaf(x[k].w, f0, o[0][3]);
      o[1][0] = fmaf(y[k].x, f1, o[1][0]), o[1][1] = fmaf(y[k].y, f1, o[1][1]);
      o[1][2] = fmaf(y[k].z, f1, o[1][2]), o[1][3] = fmaf(y[k].w, f1, o[1][3]);
    }
  }
  const int warps = n < kCombineWarps ? n : kCombineWarps;  // that had a segment
  if (warp > 0 && warp < warps) {
    sh_o[warp][0][lane] = make_float4(o[0][0], o[0][1], o[0][2], o[0][3]);
    sh_o[warp][1][lane] = make_float4(o[1][0], o[1][1], o[1][2], o[1][3]);
    if (lane == 0) sh_ml[warp] = make_float4(m[0], l[0], m[1], l[1]);
  }
  if (n > 1) __syncthreads();
  if (warp > 0) return;
  for (int w = 1; w < warps; ++w) {
    const float4 v = sh_ml[w], x = sh_o[w][0][lane], y = sh_o[w][1][lane];
    const float t0 = fmaxf(m[0], v.x), t1 = fmaxf(m[1], v.z);
    const float g0 = ex2(m[0] - t0), g1 = ex2(m[1] - t1), f0 = ex2(v.x - t0), f1 = ex2(v.z - t1);
    m[0] = t0, m[1] = t1;
    l[0] = l[0] * g0 + v.y * f0, l[1] = l[1] * g1 + v.w * f1;
    o[0][0] = o[0][0] * g0 + x.x * f0, o[0][1] = o[0][1] * g0 + x.y * f0;
    o[0][2] = o[0][2] * g0 + x.z * f0, o[0][3] = o[0][3] * g0 + x.w * f0;
    o[1][0] = o[1][0] * g1 + y.x * f1, o[1][1] = o[1][1] * g1 + y.y * f1;
    o[1][2] = o[1][2] * g1 + y.z * f1, o[1][3] = o[1][3] * g1 + y.w * f1;
  }
  // No token left by the mask: 0.
  const float r0 = l[0] == 0.f ? 0.f : 1.f / l[0], r1 = l[1] == 0.f ? 0.f : lam / l[1];
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = o[0][i] * r0 - o[1][i] * r1;
  if (a.apply_norm && l[0] != 0.f) {  // of 0 it would be a NaN if eps is 0
    float ss = y[0] * y[0] + y[1] * y[1] + y[2] * y[2] + y[3] * y[3];
#pragma unroll
    for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float f = a.post_scale * rsqrtf(ss * (1.f / kD) + a.eps);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= f * gain[i];
  }
  *reinterpret_cast<uint2*>(a.out + (size_t)blockIdx.x * kD + 4 * lane) =
      make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int runs_of(int cols) { return kPlanSms * warps_of(cols > 8 ? 2 : 1); }

// Up to this many sequences the second kernel finds a unit's segments by adding
// up the lengths before it, which costs no trip to what the first kernel wrote
// (one trip, 0.6 us, of 8 for two short requests); above, where every CTA's
// sums would cost the square of the batch, the first kernel writes them down.
constexpr int kSumBatch = 256;

size_t workspace_bytes_of(int batch, int units, int cols) {
  const size_t slots = (size_t)batch * units + runs_of(cols);
  return slots * cols * (kD + 2) * sizeof(float) +
         (batch > kSumBatch ? (size_t)batch * units * sizeof(int2) : 0);
}

int chunks_of(int group) { return (group + kChunkHeads - 1) / kChunkHeads; }

cudaError_t launch(Kv4Args& a, void* workspace, cudaStream_t stream) {
  a.runs = runs_of(a.cols);
  const size_t slots = (size_t)a.batch * a.heads * a.chunks + a.runs;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + slots * a.cols * kD;
  a.spans = a.batch > kSumBatch ? reinterpret_cast<int2*>(a.part_ml + slots * a.cols * 2) : nullptr;
  auto run = [&](auto kernel, int tiles) -> cudaError_t {
    const int smem = smem_of(tiles);
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(kPlanSms), warps_of(tiles) * 32, smem, stream, a);
  };
  cudaError_t e;
  if (a.v1) e = run(kv4_decode_kernel<1, true>, 1);
  else if (a.cols <= 8) e = run(kv4_decode_kernel<1, false>, 1);
  else e = run(kv4_decode_kernel<2, false>, 2);
  if (e != cudaSuccess) return e;
  return launch_after(kv4_combine_kernel, dim3((unsigned)a.batch * (unsigned)a.out_heads),
                      kCombineWarps * 32, 0, stream, a);
}

int check(const void* q, const void* cache, const int* table, const int* lens, const void* out,
          const float* lambda, da_dtype dtype, int batch, int heads, int n_pages, int page_size,
          int max_pages, int window) {
  if (!q || !cache || !table || !lens || !out || !lambda) return DA_ERR_INVALID_ARG;
  if (dtype != DA_BF16 && dtype != DA_FP32) return DA_ERR_INVALID_ARG;
  if (batch < 1 || heads < 1 || n_pages < 1 || max_pages < 1 || page_size < 1 || window < 0)
    return DA_ERR_INVALID_ARG;
  if (dtype != DA_BF16 || !kv4_page_size_ok(page_size)) return DA_ERR_UNSUPPORTED;
  if ((long long)n_pages * page_size >= (1LL << 31) ||
      (long long)max_pages * page_size >= (1LL << 31) ||
      (long long)n_pages * page_size / kKv4Tile * heads >= (long long)kBadTile)
    return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

// Sizes whose indices fit the kernels'.
bool sizes_ok(long long batch, long long q_heads) {
  return batch <= (1 << 20) && q_heads <= (1 << 16) && batch * q_heads < (1LL << 28);
}

}  // namespace
}  // namespace da

using da::Kv4Args;

extern "C" size_t diffattn_v2_decode_kv4_workspace_size(int batch, int n_q_heads,
                                                        int n_kv_heads) {
  if (batch < 1 || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads) return 0;
  const int group = n_q_heads / n_kv_heads;
  if (group % 2 || !da::sizes_ok(batch, n_q_heads)) return 0;
  const int cols = group < da::kChunkHeads ? group : da::kChunkHeads;
  return da::workspace_bytes_of(batch, n_kv_heads * da::chunks_of(group), cols);
}

extern "C" int diffattn_v2_decode_kv4(const void* q, const void* cache, int n_pages,
                                      int page_size, const int* block_table, int max_pages,
                                      const int* cache_lens, int window, void* out,
                                      da_dtype dtype, int batch, int n_q_heads, int n_kv_heads,
                                      int head_dim, const float* lambda, void* workspace,
                                      size_t workspace_bytes, int* dev_status, void* stream) {
  const int st = da::check(q, cache, block_table, cache_lens, out, lambda, dtype, batch,
                           n_kv_heads, n_pages, page_size, max_pages, window);
  if (st != DA_OK) return st;
  if (n_q_heads < 1 || head_dim < 1 || n_q_heads % n_kv_heads || (n_q_heads / n_kv_heads) % 2)
    return DA_ERR_INVALID_ARG;
  if (head_dim != da::kD || !da::sizes_ok(batch, n_q_heads)) return DA_ERR_UNSUPPORTED;
  if (!da::aligned16(q) || !da::aligned16(cache) || !da::aligned16(out)) return DA_ERR_ALIGNMENT;
  if (!workspace ||
      workspace_bytes < diffattn_v2_decode_kv4_workspace_size(batch, n_q_heads, n_kv_heads))
    return DA_ERR_WORKSPACE;
  if (!da::aligned16(workspace)) return DA_ERR_ALIGNMENT;
  Kv4Args a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.cache = static_cast<const uint8_t*>(cache);
  a.table = block_table;
  a.lens = cache_lens;
  a.batch = batch;
  a.heads = n_kv_heads;
  a.group = n_q_heads / n_kv_heads;
  a.chunks = da::chunks_of(a.group);
  a.max_pages = max_pages;
  a.page_shift = da::kv4_shift(page_size);
  a.n_pages = n_pages;
  a.window = window;
  a.scale = (float)(1.4426950408889634 / std::sqrt(128.0));
  a.cols = a.group < da::kChunkHeads ? a.group : da::kChunkHeads;
  a.dev_status = dev_status;
  a.lambda = lambda;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.out_heads = n_q_heads / 2;
  return da::launch(a, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK
                                                                                    : DA_ERR_CUDA;
}

extern "C" size_t diffattn_v1_decode_kv4_workspace_size(int batch, int n_heads) {
  if (batch < 1 || n_heads < 1 || !da::sizes_ok(batch, n_heads)) return 0;
  return da::workspace_bytes_of(batch, n_heads, 2);
}

extern "C" int diffattn_v1_decode_kv4(const void* q, const void* cache, int n_pages,
                                      int page_size, const int* block_table, int max_pages,
                                      const int* cache_lens, int window, void* out,
                                      da_dtype dtype, int batch, int n_heads, int d_qk, int d_v,
                                      const float* lambda, int apply_norm,
                                      const float* norm_weight, float norm_eps,
                                      float lambda_init, void* workspace, size_t workspace_bytes,
                                      int* dev_status, void* stream) {
  const int st = da::check(q, cache, block_table, cache_lens, out, lambda, dtype, batch, n_heads,
                           n_pages, page_size, max_pages, window);
  if (st != DA_OK) return st;
  if (d_qk < 1 || d_v < 1 || (apply_norm && !(norm_eps >= 0.f))) return DA_ERR_INVALID_ARG;
  if (d_qk != 64 || d_v != da::kD || !da::sizes_ok(batch, n_heads)) return DA_ERR_UNSUPPORTED;
  if (!da::aligned16(q) || !da::aligned16(cache) || !da::aligned16(out)) return DA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < diffattn_v1_decode_kv4_workspace_size(batch, n_heads))
    return DA_ERR_WORKSPACE;
  if (!da::aligned16(workspace)) return DA_ERR_ALIGNMENT;
  Kv4Args a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.cache = static_cast<const uint8_t*>(cache);
  a.table = block_table;
  a.lens = cache_lens;
  a.batch = batch;
  a.heads = n_heads;
  a.group = 2;
  a.chunks = 1;
  a.max_pages = max_pages;
  a.page_shift = da::kv4_shift(page_size);
  a.n_pages = n_pages;
  a.window = window;
  a.scale = (float)(1.4426950408889634 / 8.0);
  a.cols = 2;
  a.dev_status = dev_status;
  a.lambda = lambda;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.out_heads = n_heads;
  a.v1 = 1;
  a.apply_norm = apply_norm;
  a.gain = norm_weight;
  a.eps = norm_eps;
  a.post_scale = 1.0f - lambda_init;
  return da::launch(a, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK
                                                                                    : DA_ERR_CUDA;
}
