// Attention over the paged NVFP4 KV cache (sg_kv.cuh):
//
//   O[t, h] = sum_j softmax_j(scale q_t,h . k_j,g) v_j,g       g = h / (H / Hkv)
//
// over the keys of the token's own request, found through its block table.
//
// The streaming kernel: the query rows of a unit (request, kv head, block of 8 NT
// rows; row = token * (H / Hkv) + head of the group) share every cache byte that is
// read.  A decode step does 4 to 16 FLOP per cache byte per row, and 4-bit
// elements must be turned into numbers first, so a unit's work is: bytes from
// memory (bulk copies into a ring that belongs to one warp), codes to fp16 in
// registers (a conversion and a multiply by the block's scale, both exact: 2 + 4
// significant bits), and products on m16n8k16 with the keys (then the head dims)
// on the M side and 8 query rows on the N side.  mma.sync is chosen here over
// tcgen05 because its operands come straight from registers: tcgen05 would take the
// decoded keys and values through shared memory (four times the cache's bytes,
// written and read) to fill 128-row tiles of which 8 rows are used.
//
//   S^T (16 keys x 8 rows)  = K (16 x 128) Q^T      K from codes, Q held as fp16
//   P^T = 2^(S^T - ref)       fp16, turned into the B operand by movmatrix
//   O^T (128 x 8 rows)     += V^T (128 x 16 keys) P^T; row sums by a product with 1
//
// Q is fp16 after a power-of-two shift per row (row maximum at 2^13 .. 2^14), which
// keeps all 8 significant bits of any element within 2^30 of the maximum.
// The reference of a row's weights is its running maximum less 12, moved only when
// a score passes it by 15: weights are at most 2^15, and those down to 2^-14 (2^-26
// of the largest) are normal fp16 numbers, one rounding of 2^-11 each.  Smaller weights
// count where every larger one meets a zero in V: a step that holds some down to 2^-38
// takes a second product of those, times 2^24; with smaller ones still, its value
// product runs on m16n8k8 tf32 (11 bits as well, fp32's exponents).
// The sums use the rounded weights.  Sums and the merges are fp32.
//
// Schedule.  A step is 32 NT keys.  The units' steps laid end to end are cut into
// equal shares, one per CTA and spread evenly over its warps, whatever the requests'
// lengths are: every CTA reads the lengths, scans them and finds its warps' runs, so the
// plan follows lengths on the device and a captured launch stays valid.  A warp walks its run
// alone (its own ring and barriers, no CTA-wide step until the end) and stores a
// unit that lies inside its run itself.  Units cut between warps are merged in
// shared memory once the CTA's runs are done; one cut between CTAs leaves one fp32
// partial (output, maximum, sum) per CTA in the workspace, and the CTA whose piece
// arrives last merges them in order: no CTA waits for another, and results do not
// depend on the order of arrival.  (A CTA-wide merge per unit, with every warp
// taking part in each unit, cost 2 to 5 us per unit and CTA.)
//
// Measured, 32 heads on 8 kv heads: 64 requests of 512 to 8192 keys, one token each,
// 207 MB of cache, 59 us (3.5 TB/s, 0.52 of the copy roof); 131071 and 50001 keys, 209
// MB, 54 us (3.9 TB/s).  The loop itself runs at 5.9 TB/s, bound by issue (ALU pipe 46%,
// issue slots 50% of active cycles: 306 instructions per 2304-byte tile and warp); the
// plan and first loads take 7 us and the merges and the tail of uneven warps up to 10.
// One query against 4096 keys, 32 heads with their own: 19.4 us, most of it plan, first
// loads and merges (runs per CTA instead of per warp took 15 there, but 83 and 66 on the
// two above).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sg_internal.h"
#include "sg_kv.cuh"
#include "sg_ptx.cuh"

namespace sg {
namespace {

constexpr float kNoRef = -1e30f;      // reference of a row that has seen no key
constexpr float kRefShift = 12.f;     // the reference lies this far below the maximum it was set from
constexpr float kMoveAbove = 15.f;    // it moves once a score passes it by more than this
constexpr float kSmallBelow = -14.f;  // weights below 2^-14 are not normal fp16 numbers
constexpr float kTinyBelow = -38.f;   // nor is 2^24 times those below 2^-38
constexpr int kRowPitch = 132;        // floats per merged row in shared memory

// What bounds the kernel is the issue of decode instructions (a conversion and a
// multiply per two elements) and their latency, so warps per SM are traded against
// registers: 12 warps of 168 registers (8 rows).
template <int NT>
struct Cfg {
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NT;
  static constexpr int kTiles = 2 * NT;                  // cache tiles per step
  static constexpr int kStepKeys = kTiles * kKvTile;
  static constexpr int kStageBytes = kTiles * kKvTileBytes;
  static constexpr int kStages = 2;
  static constexpr int kPartBytes = kRows * kRowPitch * 4;  // one warp's fp32 output of all rows
  static constexpr int kWarpBytes = kStages * kStageBytes + kPartBytes;
  static constexpr int kBarOff = kWarps * kWarpBytes;
  static constexpr int kMaxOff = kBarOff + kWarps * kStages * 8;
  static constexpr int kSumOff = kMaxOff + 2 * kWarps * kRows * 4;
  static constexpr int kScanOff = kSumOff + 2 * kWarps * kRows * 4;
  static constexpr int kFoundOff = kScanOff + kWarps * 8 + 16;
  static constexpr int kCutOff = kFoundOff + kWarps * 32;
  static constexpr int kMiscOff = kCutOff + 2 * kWarps * 48;
  static constexpr int kSmem = kMiscOff + 64;
  // the last partial of a run lies in the ring, which has no loads left by then
  static_assert(kPartBytes <= kStages * kStageBytes && kPartBytes % 16 == 0, "partial in the ring");
  static_assert(kSmem <= 232448, "shared memory budget");
};

// Shared-memory loads by 32-bit address (volatile: the bytes are written by copies).
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c += 2^-24 a b
__device__ __forceinline__ void mma_f16_low(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  float d[4] = {0.f, 0.f, 0.f, 0.f};
  mma_f16(d, a0, a1, a2, a3, b0, b1);
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = fmaf(d[e], 0x1p-24f, c[e]);
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t to_tf32(float x) {  // nearest, ties away
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t low_f32(uint32_t h2) {
  return __float_as_uint(__low2float(*reinterpret_cast<const __half2*>(&h2)));
}
__device__ __forceinline__ uint32_t high_f32(uint32_t h2) {
  return __float_as_uint(__high2float(*reinterpret_cast<const __half2*>(&h2)));
}

// Transposes an 8 x 8 matrix of fp16 spread over the warp (lane 4 g + t holds row g,
// columns 2 t and 2 t + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
               : "memory");
}

// One cache tile into shared memory (bulk copy), completing on `bar`.
__device__ __forceinline__ void tile_load(uint32_t dst, const uint8_t* src, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "n"(kKvTileBytes), "r"(bar)
               : "memory");
}

// Scores of two tiles (32 keys) at shared address `st`: s[tile][nt] holds keys g8 (0, 1)
// and g8 + 8 (2, 3) of rows 2 t4 and 2 t4 + 1.
template <int NT>
__device__ __forceinline__ void scores(uint32_t st, int lane, const uint32_t (&qf)[NT][16], float (&s)[2][NT][4]) {
  uint4 k[2][2];
  uint32_t sc[2];
#pragma unroll
  for (int tl = 0; tl < 2; ++tl) {
    k[tl][0] = lds128(st + tl * kKvTileBytes + 16 * lane);
    k[tl][1] = lds128(st + tl * kKvTileBytes + 512 + 16 * lane);
    sc[tl] = lds32(st + tl * kKvTileBytes + kKvKScaleOff + 4 * lane);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[tl][nt][e] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // word i: dims 32 t4 + 8 i .. + 7, two k-steps; the tiles' products alternate
#pragma unroll
    for (int tl = 0; tl < 2; ++tl) {
      const __half2 sa = e4m3x2_half2(sc[tl] & 0xFFFFu), sb = e4m3x2_half2(sc[tl] >> 16);
      const uint32_t wa = i == 0 ? k[tl][0].x : i == 1 ? k[tl][0].y : i == 2 ? k[tl][0].z : k[tl][0].w;
      const uint32_t wb = i == 0 ? k[tl][1].x : i == 1 ? k[tl][1].y : i == 2 ? k[tl][1].z : k[tl][1].w;
      uint32_t a[4], b[4];
      e2m1x8_times(wa, i < 2 ? __low2half2(sa) : __high2half2(sa), a);
      e2m1x8_times(wb, i < 2 ? __low2half2(sb) : __high2half2(sb), b);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_f16(s[tl][nt], a[0], b[0], a[1], b[1], qf[nt][4 * i], qf[nt][4 * i + 1]);
        mma_f16(s[tl][nt], a[2], b[2], a[3], b[3], qf[nt][4 * i + 2], qf[nt][4 * i + 3]);
      }
    }
  }
}

// o += V^T P and l += sums of P for one tile: weights 2^d, V codes at shared address
// `tile`, scale bytes `sc`.
enum class Weights { kNormal, kLow, kWide };
template <int NT, Weights W>
__device__ __forceinline__ void values(uint32_t tile, uint32_t sc, int lane, const float (&d)[NT][4], float (&o)[8][NT][4],
                                       float (&l)[NT][4]) {
  const uint4 va = lds128(tile + kKvVCodeOff + 16 * lane), vb = lds128(tile + kKvVCodeOff + 512 + 16 * lane);
  const __half2 s0 = e4m3x2_half2(sc & 0xFFFFu), s1 = e4m3x2_half2(sc >> 16);
  // weights as the B operand: pb[h] keys 2 t4 + 8 h (low) and 2 t4 + 1 + 8 h (high) of
  // row g8 in fp16; pw[h] the same two in tf32, or (kLow) in pw[h][0] the weights below
  // 2^-14 times 2^24
  uint32_t pb[NT][2], pw[NT][2][2];
  constexpr uint32_t kOne16 = 0x3C003C00u, kOne32 = 0x3F800000u;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float u = exp2_approx(d[nt][2 * h]), v = exp2_approx(d[nt][2 * h + 1]);
      if (W == Weights::kWide) {
        const uint32_t tu = to_tf32(u), tv = to_tf32(v);
        const uint32_t lo = transpose8x8(__byte_perm(tu, tv, 0x5410)), hi = transpose8x8(__byte_perm(tu, tv, 0x7632));
        pw[nt][h][0] = __byte_perm(lo, hi, 0x5410);
        pw[nt][h][1] = __byte_perm(lo, hi, 0x7632);
        mma_tf32(l[nt], kOne32, kOne32, kOne32, kOne32, pw[nt][h][0], pw[nt][h][1]);
      } else {
        if (W == Weights::kLow) {
          const bool lu = u < 0x1p-14f, lv = v < 0x1p-14f;
          pw[nt][h][0] = transpose8x8(half2_bits(__floats2half2_rn(lu ? u * 0x1p24f : 0.f, lv ? v * 0x1p24f : 0.f)));
          u = lu ? 0.f : u;
          v = lv ? 0.f : v;
        }
        pb[nt][h] = transpose8x8(half2_bits(__floats2half2_rn(u, v)));
      }
    }
    if (W != Weights::kWide) mma_f16(l[nt], kOne16, kOne16, kOne16, kOne16, pb[nt][0], pb[nt][1]);
    if (W == Weights::kLow) mma_f16_low(l[nt], kOne16, kOne16, kOne16, kOne16, pw[nt][0][0], pw[nt][1][0]);
  }
  // key pairs side by side in a byte: even dims (row g8) and odd dims (row g8 + 8)
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = h ? va.y : va.x, b = h ? va.w : va.z, c = h ? vb.y : vb.x, e = h ? vb.w : vb.z;
    uint32_t a0[4], a1[4], a2[4], a3[4];
    e2m1x8_times((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), s0, a0);
    e2m1x8_times(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), s0, a1);
    e2m1x8_times((c & 0x0F0F0F0Fu) | ((e << 4) & 0xF0F0F0F0u), s1, a2);
    e2m1x8_times(((c >> 4) & 0x0F0F0F0Fu) | (e & 0xF0F0F0F0u), s1, a3);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (W == Weights::kWide) {
          mma_tf32(o[4 * h + i][nt], low_f32(a0[i]), low_f32(a1[i]), high_f32(a0[i]), high_f32(a1[i]), pw[nt][0][0],
                   pw[nt][0][1]);
          mma_tf32(o[4 * h + i][nt], low_f32(a2[i]), low_f32(a3[i]), high_f32(a2[i]), high_f32(a3[i]), pw[nt][1][0],
                   pw[nt][1][1]);
        } else {
          mma_f16(o[4 * h + i][nt], a0[i], a1[i], a2[i], a3[i], pb[nt][0], pb[nt][1]);
          if (W == Weights::kLow) mma_f16_low(o[4 * h + i][nt], a0[i], a1[i], a2[i], a3[i], pw[nt][0][0], pw[nt][1][0]);
        }
      }
  }
}

// One request as the kernel sees it (row_blocks 0: nothing to compute).
struct Request {
  int32_t q0, nq, n;   // first query row, query tokens, keys
  int32_t steps;       // steps of kStepKeys keys; no keys: one empty step, which gives zeros
  int32_t row_blocks;
  __device__ __forceinline__ int32_t units(const KvAttnParams& p) const { return row_blocks * p.kv_heads; }
};

template <int NT>
__device__ __forceinline__ Request load_request(const KvAttnParams& p, int b) {
  Request r;
  r.q0 = p.cu_q[b];
  const int32_t q1 = p.cu_q[b + 1];
  r.n = p.seq_lens[b];
  const bool bad = r.q0 < 0 || q1 < r.q0 || q1 > p.tokens || q1 - r.q0 > p.max_q || r.n < 0 ||
                   r.n > static_cast<int64_t>(p.max_pages) * p.cache.page_size;
  r.nq = bad ? -1 : q1 - r.q0;
  r.steps = max(1, (r.n - 1) / Cfg<NT>::kStepKeys + 1);
  r.row_blocks = r.nq > 0 ? (r.nq * (p.heads / p.kv_heads) + Cfg<NT>::kRows - 1) / Cfg<NT>::kRows : 0;
  return r;
}

// Where a warp's run begins: its request, and the steps before that request.
struct Found {
  int64_t at;
  int32_t b;
  Request req;
};
static_assert(sizeof(Found) == 32, "shared layout");

// A unit that a run cuts: its partial is in this warp's buffer.
struct Cut {
  int64_t start;        // first step of the unit, over the whole launch
  int32_t unit;
  int32_t valid;        // 1: the run holds part of it
  int32_t past;         // 1: it goes on past the run's end
  Request req;
  int32_t pad[2];
};
static_assert(sizeof(Cut) == 48, "shared layout");

// a / b for a >= 0, in 32 bits where they suffice (a 64-bit division is ~100 instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 31 == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 1) kv_stream_kernel(const KvAttnParams p) {
  using C = Cfg<NT>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int g8 = lane / 4, t4 = lane % 4;
  uint8_t* ring = smem + warp * C::kWarpBytes;
  const uint32_t ring_addr = smem_u32(ring);
  const uint32_t bars_addr = smem_u32(smem + C::kBarOff) + warp * C::kStages * 8;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff) + warp * C::kStages;
  float* sm_max = reinterpret_cast<float*>(smem + C::kMaxOff);  // [2][warp][row]: partials 0 (first) and 1 (last) of a run
  float* sm_sum = reinterpret_cast<float*>(smem + C::kSumOff);
  int64_t* scan = reinterpret_cast<int64_t*>(smem + C::kScanOff);       // [warp], then the total
  Found* found = reinterpret_cast<Found*>(smem + C::kFoundOff);         // [warp]
  Cut* cuts = reinterpret_cast<Cut*>(smem + C::kCutOff);                // [2][warp]
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff);
  volatile int32_t* finish = reinterpret_cast<volatile int32_t*>(smem + C::kMiscOff + 16);  // [2] cut to merge, or -1
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(&bars[s], 1);
    if (warp == 0) {
      *abort_flag = 0;
      finish[0] = finish[1] = -1;
    }
    cuts[warp].valid = cuts[kWarps + warp].valid = 0;
    cuts[warp].past = cuts[kWarps + warp].past = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- the warps' runs
  auto block_scan = [&](int64_t v) -> int64_t {  // inclusive, over the threads; scan[kWarps]: the total
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = v;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += scan[w];
      all += scan[w];
    }
    if (tid == 0) scan[kWarps] = all;
    __syncthreads();
    return v + before;
  };
  Request mine = {};
  auto work_of = [&](int b) -> int64_t {
    if (b >= p.batch) return 0;
    mine = load_request<NT>(p, b);
    if (mine.nq < 0 && blockIdx.x == 0) record_error(p.err, kDevBadRequest, b);
    return static_cast<int64_t>(mine.units(p)) * mine.steps;
  };
  int64_t total = 0, work = 0, upto = 0;
  for (int base = 0; base < p.batch; base += kThreads) {
    work = work_of(base + tid);
    upto = total + block_scan(work);
    total += scan[kWarps];
  }
  // equal shares per CTA, and the share's steps spread evenly over its warps
  // (at least a step per warp: thinner shares only cut units into more pieces)
  const int64_t share = max(quotient(total + gridDim.x - 1, gridDim.x), static_cast<int64_t>(kWarps));
  const int64_t cta0 = share * blockIdx.x, cta1 = min(cta0 + share, total);
  if (cta0 >= cta1) return;
  // first step of warp w (warps without a step come last, so that cut units run through
  // neighbouring warps)
  auto run_of = [&](int w) -> int64_t {
    const int64_t n = cta1 - cta0;
    return cta0 + (n < kWarps ? min(static_cast<int64_t>(w), n) : quotient(n * w, kWarps));
  };
  if (p.batch > kThreads) total = 0;
  for (int base = 0; base < p.batch; base += kThreads) {
    if (p.batch > kThreads) {  // (else the scan above stands)
      work = work_of(base + tid);
      upto = total + block_scan(work);
      total += scan[kWarps];
    }
    if (work > 0 && upto > cta0 && upto - work < cta1) {
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) {
        const int64_t at = run_of(w);
        if (upto - work <= at && at < upto) {
          found[w].at = upto - work;
          found[w].b = base + tid;
          found[w].req = mine;
        }
      }
    }
    if (p.batch > kThreads && total >= cta1) break;
  }
  __syncthreads();
  const int64_t run0 = run_of(warp);
  const int run = static_cast<int>(run_of(warp + 1) - run0);
  int left = run;  // steps to consume
  const int group = p.heads / p.kv_heads;
  bool failed = false;
  int issued = 0;

  if (left > 0) {
    // ---- positions: `use` of the products, `get` of the loads
    int use_b = found[warp].b;
    Request req = found[warp].req;
    int use_unit = static_cast<int>(quotient(run0 - found[warp].at, req.steps));
    int use_step = static_cast<int>(run0 - found[warp].at - static_cast<int64_t>(use_unit) * req.steps);
    int get_b = use_b, get_unit = use_unit, get_step = use_step;
    Request get_req = req;
    int to_issue = left;    // steps not yet in a batch
    uint32_t extra_tx = p.inject_extra_tx;
    const int tiles_per_page = p.cache.page_size / kKvTile;
    auto next_unit = [&](int& b, int& unit, Request& r) {
      if (++unit < r.units(p)) return;
      unit = 0;
      do {
        if (++b >= p.batch) return;
        r = load_request<NT>(p, b);
      } while (r.row_blocks == 0);
    };
    // Loads go by batches of 32 tiles of one unit: lane i looks up tile i of the batch
    // when the batch before it is used up, and turns the page into an address when its
    // first step is issued (a step later).
    int in_batch = 0;       // steps of the batch still to issue
    bool fresh = true;      // the look-up has not been turned into addresses yet
    int32_t page = -1;
    int page_tile = 0, first_lane = 0;
    bool want = false;
    uint32_t batch_ok = 0;
    const uint8_t* src = nullptr;
    auto look_up = [&]() {
      const int tile = get_step * C::kTiles + lane;
      want = static_cast<int64_t>(tile) * kKvTile < get_req.n;
      page_tile = tile % tiles_per_page;
      page = want ? p.table[get_b * p.table_pitch + tile / tiles_per_page] : -1;
      in_batch = min(min(32 / C::kTiles, get_req.steps - get_step), to_issue);
      to_issue -= in_batch;
      get_step += in_batch;
      first_lane = 0;
      fresh = true;
    };
    auto prefetch_q = [&]() {  // the next unit's query rows (256 bytes each), wanted some steps later
      const int row = lane / 2;
      const int rr = (get_unit % get_req.row_blocks) * C::kRows + row;
      if (row < C::kRows && rr < get_req.nq * group)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.Q + static_cast<int64_t>(get_req.q0 + rr / group) * p.ldq +
                                                      static_cast<int64_t>(get_unit / get_req.row_blocks * group + rr % group) * kKvDim +
                                                      64 * (lane & 1)));
    };
    uint32_t tile_ok = 0;  // 4 bits per stage in flight, the next to be used lowest: tiles loaded
    int issue_stage = 0;
    auto issue = [&]() {
      tile_ok >>= 4;
      if (in_batch == 0) return;
      if (fresh) {
        fresh = false;
        const bool ok = want && page >= 0 && page < p.cache.num_pages;
        if (want && !ok) record_error(p.err, kDevBadPage, get_b);
        batch_ok = __ballot_sync(0xFFFFFFFFu, ok);
        src = p.cache.base + page * p.cache.pitch +
              (static_cast<int64_t>(get_unit / get_req.row_blocks) * tiles_per_page + page_tile) * kKvTileBytes;
      }
      const uint32_t mask = (batch_ok >> first_lane) & ((1u << C::kTiles) - 1u);
      tile_ok |= mask << (4 * (C::kStages - 1));
      const uint32_t bar = bars_addr + issue_stage * 8;
      if (lane == 0) expect_tx(bar, __popc(mask) * kKvTileBytes + extra_tx);
      extra_tx = 0;
      __syncwarp();
      const unsigned at = static_cast<unsigned>(lane - first_lane);
      if (at < C::kTiles && (batch_ok >> lane & 1u)) {
        fence_proxy_async_smem();  // this stage's reads (and the barrier above) before the copy's writes
        tile_load(ring_addr + issue_stage * C::kStageBytes + at * kKvTileBytes, src, bar);
      }
      issue_stage = issue_stage + 1 == C::kStages ? 0 : issue_stage + 1;
      ++issued;
      first_lane += C::kTiles;
      if (--in_batch == 0 && to_issue > 0) {
        if (get_step == get_req.steps) {
          get_step = 0;
          next_unit(get_b, get_unit, get_req);
          prefetch_q();
        }
        look_up();
      }
    };
    // Raw query rows of a unit: lane (g8, t4) takes 64 bytes of row g8 (of each 8 rows).
    uint4 q_rows[NT][4];
    auto q_row = [&](const Request& r, int unit, int row) {
      const int rr = (unit % r.row_blocks) * C::kRows + row;
      return p.Q + static_cast<int64_t>(r.q0 + rr / group) * p.ldq +
             static_cast<int64_t>(unit / r.row_blocks * group + rr % group) * kKvDim + 32 * t4;
    };
    auto q_count = [&](const Request& r, int unit) {
      return min(C::kRows, r.nq * group - (unit % r.row_blocks) * C::kRows);
    };
    auto load_q = [&](const Request& r, int unit) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q_rows[nt][i] = 8 * nt + g8 < q_count(r, unit)
                              ? reinterpret_cast<const uint4*>(q_row(r, unit, 8 * nt + g8))[i]
                              : make_uint4(0u, 0u, 0u, 0u);
    };
    // The first unit's rows are asked for before the cache tiles: behind the copies that
    // fill every ring of the GPU they took 3 us.
    load_q(req, use_unit);
    bool q_loaded = true;
    look_up();
#pragma unroll 1
    for (int s = 0; s < C::kStages; ++s) issue();

    int use_stage = 0;
    uint32_t use_phase = 0;
    while (left > 0 && !failed) {
      // ---- one segment: this run's steps of one unit
      const bool before = use_step > 0;  // the unit began in an earlier run
      const int seg = min(left, req.steps - use_step);
      left -= seg;
      const bool past = use_step + seg < req.steps;
      const int kvh = use_unit / req.row_blocks;
      const int row0 = (use_unit % req.row_blocks) * C::kRows;
      const int rows = min(C::kRows, req.nq * group - row0);
      // Q as B fragments: lane (g8, t4) holds row g8, dims 32 t4 .. 32 t4 + 31
      uint32_t qf[NT][16];
      float col_scale[NT][2];
      int lim[NT][2];
      if (!q_loaded) load_q(req, use_unit);
      q_loaded = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 (&v)[4] = q_rows[nt];
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const int e = top == 0 ? 0 : max(-100, min(127, static_cast<int>(top >> 7) - 127));
        // The scale's sign goes into Q; with scale 0 every score is 0.  A row with a NaN or
        // an infinity becomes NaN as a whole: its scores are NaN or infinite whatever the
        // key, and a softmax over any of those is NaN (left as they are, infinities of one
        // sign would all be -inf and pass for masked keys).
        const float shift = top >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                                           : exp2f(static_cast<float>(13 - e)) *
                                                 (p.scale_log2 < 0.f ? -1.f : p.scale_log2 == 0.f ? 0.f : 1.f);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          qf[nt][i] = half2_bits(__floats2half2_rn(__uint_as_float(w[i] << 16) * shift,
                                                   __uint_as_float(w[i] & 0xFFFF0000u) * shift));
        // (at least 2^-126: an underflow to 0 would turn masked scores, -inf, into NaN)
        const float back =
            p.scale_log2 == 0.f ? 1.f : fmaxf(exp2f(static_cast<float>(e - 13)) * fabsf(p.scale_log2), 0x1p-126f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r2 = 8 * nt + 2 * t4 + c;
          col_scale[nt][c] = __shfl_sync(0xFFFFFFFFu, back, (2 * t4 + c) * 4);
          // keys [0, lim) are visible to the row; rows past the block are dead columns
          lim[nt][c] =
              r2 >= rows ? INT32_MAX : (p.causal ? max(0, req.n - req.nq + (row0 + r2) / group + 1) : req.n);
        }
      }
      const int lim_min = p.causal ? max(0, req.n - req.nq + row0 / group + 1) : req.n;
      float o[8][NT][4], l[NT][4], ref[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        ref[nt][0] = ref[nt][1] = kNoRef;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[nt][e] = 0.f;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) o[mt][nt][e] = 0.f;
        }
      }

#pragma unroll 1
      for (const int seg_end = use_step + seg; use_step < seg_end; ++use_step) {
        const int s = use_stage;
        if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(bars_addr + 8 * s, use_phase))) {
          const bool came = mbar_wait(&bars[s], use_phase, p.timeout_ns, abort_flag);
          if (!__all_sync(0xFFFFFFFFu, came)) {
            if (!*abort_flag && lane == 0) record_error(p.err, kDevTimeoutFull, use_step);
            *abort_flag = 1;
            failed = true;
            break;
          }
        }
        const uint32_t ok = tile_ok & 0xFu;
        if (ok != 0) {
          const uint32_t st0 = ring_addr + s * C::kStageBytes;
#pragma unroll 1
          for (int half_step = 0; half_step < NT; ++half_step) {
            const uint32_t st = st0 + half_step * 2 * kKvTileBytes;
            const int key0 = use_step * C::kStepKeys + 32 * half_step;
            const uint32_t ok2 = (ok >> (2 * half_step)) & 3u;
            float x[2][NT][4];
            scores<NT>(st, lane, qf, x);
            const bool tail = ok2 != 3u || key0 > lim_min - 32;  // (key0 + 32 may pass 2^31)
            if (tail) {
#pragma unroll
              for (int tl = 0; tl < 2; ++tl)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (!(ok2 >> tl & 1u) || key0 + 16 * tl + g8 + 8 * (e >> 1) >= lim[nt][e & 1])
                      x[tl][nt][e] = -INFINITY;  // the scale is positive (its sign is in Q)
            }
            // Most steps change nothing: all scores within [-14, 15] of their reference.
            bool odd = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float hi = fmaxf(fmaxf(x[0][nt][c], x[0][nt][c + 2]), fmaxf(x[1][nt][c], x[1][nt][c + 2]));
                const float lo = fminf(fminf(x[0][nt][c], x[0][nt][c + 2]), fminf(x[1][nt][c], x[1][nt][c + 2]));
                odd = odd || fmaf(hi, col_scale[nt][c], -ref[nt][c]) > kMoveAbove ||
                      fmaf(lo, col_scale[nt][c], -ref[nt][c]) < kSmallBelow;
              }
            Weights kind = Weights::kNormal;
            if (__any_sync(0xFFFFFFFFu, odd)) {
              bool small = false, tiny = false;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  float mx = fmaxf(fmaxf(x[0][nt][c], x[0][nt][c + 2]), fmaxf(x[1][nt][c], x[1][nt][c + 2]));
                  mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
                  mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
                  mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16)) * col_scale[nt][c];
                  if (mx - ref[nt][c] > kMoveAbove) {
                    const float next = mx - kRefShift;
                    const float f = exp2_approx(ref[nt][c] - next);
                    ref[nt][c] = next;
                    l[nt][c] *= f;
                    l[nt][c + 2] *= f;
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                      o[mt][nt][c] *= f;
                      o[mt][nt][c + 2] *= f;
                    }
                  }
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float d = fmaf(x[i >> 1][nt][c + 2 * (i & 1)], col_scale[nt][c], -ref[nt][c]);
                    small = small || (d < kSmallBelow && d >= kTinyBelow);
                    tiny = tiny || (d < kTinyBelow && d > -126.f);
                  }
                }
              if (__any_sync(0xFFFFFFFFu, tiny)) kind = Weights::kWide;
              else if (__any_sync(0xFFFFFFFFu, small)) kind = Weights::kLow;
            }
            uint32_t sc[2];
#pragma unroll
            for (int tl = 0; tl < 2; ++tl) {
              sc[tl] = lds32(st + tl * kKvTileBytes + kKvVScaleOff + 4 * lane);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[tl][nt][e] = fmaf(x[tl][nt][e], col_scale[nt][e & 1], -ref[nt][e & 1]);
            }
            if (tail) {
              // Keys past the sequence (their bytes may hold anything) get scale 0.  A NaN
              // scale would reach every row through 0 * NaN, so it is taken out too and
              // the rows that see its key are set to NaN by hand.
#pragma unroll
              for (int tl = 0; tl < 2; ++tl) {
                const int base = key0 + 16 * tl;
                uint32_t nan_keys = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int key = 2 * t4 + (i & 1) + 8 * (i >> 1);
                  const uint32_t byte = (sc[tl] >> (8 * i)) & 0xFFu;
                  const bool dead = !(ok2 >> tl & 1u) || base + key >= req.n;
                  const bool nan = !dead && (byte & 0x7Fu) == 0x7Fu;
                  if (dead || nan) sc[tl] &= ~(0xFFu << (8 * i));
                  nan_keys |= nan ? 1u << key : 0u;
                }
                if (__any_sync(0xFFFFFFFFu, nan_keys != 0)) {
                  nan_keys |= __shfl_xor_sync(0xFFFFFFFFu, nan_keys, 1);
                  nan_keys |= __shfl_xor_sync(0xFFFFFFFFu, nan_keys, 2);
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                      const int seen = max(0, min(16, lim[nt][c] - base));
                      if (nan_keys & ((1u << seen) - 1u)) {
#pragma unroll
                        for (int mt = 0; mt < 8; ++mt) o[mt][nt][c] = o[mt][nt][c + 2] = __uint_as_float(0x7FC00000u);
                      }
                    }
                }
              }
            }
            if (kind == Weights::kNormal) {
#pragma unroll
              for (int tl = 0; tl < 2; ++tl) values<NT, Weights::kNormal>(st + tl * kKvTileBytes, sc[tl], lane, x[tl], o, l);
            } else if (kind == Weights::kLow) {
#pragma unroll 1
              for (int tl = 0; tl < 2; ++tl)
                values<NT, Weights::kLow>(st + tl * kKvTileBytes, tl ? sc[1] : sc[0], lane, tl ? x[1] : x[0], o, l);
            } else {
#pragma unroll 1
              for (int tl = 0; tl < 2; ++tl)
                values<NT, Weights::kWide>(st + tl * kKvTileBytes, tl ? sc[1] : sc[0], lane, tl ? x[1] : x[0], o, l);
            }
          }
        }
        if (++use_stage == C::kStages) {
          use_stage = 0;
          use_phase ^= 1u;
        }
        __syncwarp();
        issue();
      }
      if (failed) break;

      // ---- end of the segment: lane (g8, t4) holds rows 2 t4 + c, dims 16 g8 .. + 15
      if (!before && !past) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = 8 * nt + 2 * t4 + c;
            if (r >= rows) continue;
            const int rr = row0 + r;
            const float inv = l[nt][c] == 0.f ? 0.f : p.v_scale / l[nt][c];
            uint32_t w[8];
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) w[mt] = bf16x2_bits(o[mt][nt][c] * inv, o[mt][nt][c + 2] * inv);
            uint4* to = reinterpret_cast<uint4*>(p.O + static_cast<int64_t>(req.q0 + rr / group) * p.ldo +
                                                 static_cast<int64_t>(kvh * group + rr % group) * kKvDim + 16 * g8);
            to[0] = make_uint4(w[0], w[1], w[2], w[3]);
            to[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
      } else {
        // partial 0 (the unit began before the run) has a buffer of its own, partial 1
        // (it begins here and goes on past the run's end) the ring
        const int which = before ? 0 : 1;
        float* part = reinterpret_cast<float*>(ring + (before ? C::kStages * C::kStageBytes : 0));
        if (g8 == 0) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              sm_max[(which * kWarps + warp) * C::kRows + 8 * nt + 2 * t4 + c] = ref[nt][c];
              sm_sum[(which * kWarps + warp) * C::kRows + 8 * nt + 2 * t4 + c] = l[nt][c];
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(part + (8 * nt + 2 * t4 + c) * kRowPitch + 16 * g8 + 4 * i) =
                  make_float4(o[2 * i][nt][c], o[2 * i][nt][c + 2], o[2 * i + 1][nt][c], o[2 * i + 1][nt][c + 2]);
        if (lane == 0) {
          Cut& cut = cuts[which * kWarps + warp];
          // the steps of this run consumed so far end at use_step of the unit
          cut.start = run0 + (run - left) - use_step;
          cut.req = req;
          cut.unit = use_unit;
          cut.past = past ? 1 : 0;
          cut.valid = 1;
        }
      }
      if (use_step == req.steps && left > 0) {
        use_step = 0;
        next_unit(use_b, use_unit, req);
      }
    }
    if (failed) {  // let the copies already issued land before the CTA exits
      volatile uint32_t never = 0;
      for (int i = max(0, issued - C::kStages); i < issued; ++i)
        mbar_wait(&bars[i % C::kStages], (i / C::kStages) & 1u, p.timeout_ns, &never);
    }
  }
  if (__syncthreads_or(failed)) return;

  // ---- units cut between this CTA's warps.  One begins where warp 0 holds a partial 0
  // or a warp a partial 1, and goes on through the next warps' partials 0; its rows
  // are shared out over the warps.
  auto slot_of = [&](int64_t cta, bool first) {  // workspace partial of one CTA's piece of a unit
    return p.partials + (2 * cta + (first ? 1 : 0)) * (C::kRows * kRowPitch);
  };
  auto store4 = [&](const Request& r, int unit, int row, float4 acc, float sum) {  // lane: dims 4 lane .. + 3
    const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
    const int rr = (unit % r.row_blocks) * C::kRows + row;
    *reinterpret_cast<uint2*>(p.O + static_cast<int64_t>(r.q0 + rr / group) * p.ldo +
                              static_cast<int64_t>(unit / r.row_blocks * group + rr % group) * kKvDim + 4 * lane) =
        make_uint2(bf16x2_bits(acc.x * inv, acc.y * inv), bf16x2_bits(acc.z * inv, acc.w * inv));
  };
  auto rows_of = [&](const Cut& c) { return min(C::kRows, c.req.nq * group - (c.unit % c.req.row_blocks) * C::kRows); };
  // Sum over up to 32 parts held one per lane (maximum m, sum l; kNoRef and 0 in the
  // other lanes): returns the joint maximum, leaves the lane's weight in f.
  auto join = [&](float m, float l, float& f, float& sum) {
    float top = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    f = exp2_approx(m - top);
    sum = l * f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    return top;
  };
  int turn = 0;
  int open[2] = {-1, -1};  // cuts that leave the CTA: the first unit, the last unit
  // bit w: warp w holds a partial 0 (1), and its unit goes on past the warp's run
  const bool here = lane < kWarps;
  const uint32_t has0 = __ballot_sync(0xFFFFFFFFu, here && cuts[here ? lane : 0].valid);
  const uint32_t has1 = __ballot_sync(0xFFFFFFFFu, here && cuts[kWarps + (here ? lane : 0)].valid);
  const uint32_t past0 = __ballot_sync(0xFFFFFFFFu, here && cuts[here ? lane : 0].past) & has0;
  const uint32_t past1 = __ballot_sync(0xFFFFFFFFu, here && cuts[kWarps + (here ? lane : 0)].past) & has1;
#pragma unroll 1
  for (uint32_t todo = (has0 & 1u) | has1 << 1; todo != 0; todo &= todo - 1) {
    const int k = __ffs(todo) - 1;
    const int which = k == 0 ? 0 : 1, w0 = k == 0 ? 0 : k - 1;
    const Cut& cut = cuts[which * kWarps + w0];
    int last = w0;
    bool past = (which ? past1 : past0) >> w0 & 1u;
    while (past && has0 >> (last + 1) & 1u) {
      ++last;
      past = past0 >> last & 1u;
    }
    const bool whole = which == 1 && !past;
    if (!whole) open[which] = which * kWarps + w0;
    // piece 0 of a unit (the one that begins in this CTA) has slot 1 of the CTA, later ones slot 0
    float* slot = slot_of(blockIdx.x, which == 1);
    const int rows = rows_of(cut), parts = last - w0 + 1;
    for (int row = (warp - turn + kWarps) % kWarps; row < rows; row += kWarps) {
      const int from = lane == 0 ? which * kWarps + w0 : w0 + lane;  // lane i: part i
      const bool in = lane < parts;
      float f, sum;
      const float top = join(in ? sm_max[from * C::kRows + row] : kNoRef, in ? sm_sum[from * C::kRows + row] : 0.f, f, sum);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < parts; ++i) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, i);
        const uint8_t* buf = smem + (w0 + i) * C::kWarpBytes + (i == 0 && which == 1 ? 0 : C::kStages * C::kStageBytes);
        const float4 v = *reinterpret_cast<const float4*>(buf + (row * kRowPitch + 4 * lane) * 4);
        acc.x += v.x * w;
        acc.y += v.y * w;
        acc.z += v.z * w;
        acc.w += v.w * w;
      }
      if (whole) {
        store4(cut.req, cut.unit, row, acc, sum);
      } else {
        __stcg(reinterpret_cast<float4*>(slot + row * kRowPitch + 4 * lane), acc);
        if (lane == 0) __stcg(reinterpret_cast<float2*>(slot + row * kRowPitch + kKvDim), make_float2(top, sum));
      }
    }
    turn = (turn + rows) % kWarps;
  }
  if (open[0] < 0 && open[1] < 0) return;
  __threadfence();  // the partials before the count
  __syncthreads();
  if (lane == 0 && warp < 2 && open[warp] >= 0) {
    const Cut& cut = cuts[open[warp]];
    const int64_t piece0 = quotient(cut.start, share), piece1 = quotient(cut.start + cut.req.steps - 1, share);
    uint32_t* counter = p.counters + piece0;
    const uint32_t arrived = atomicAdd(counter, 1u);
    if (arrived == static_cast<uint32_t>(piece1 - piece0)) {
      *counter = 0;  // ready for the next launch
      finish[warp] = open[warp];
    }
    __threadfence();
  }
  __syncthreads();

  // ---- units whose last piece arrived here: their pieces in order, in `groups` runs
  // per row (one per warp), then the runs
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (finish[k] < 0) continue;
    const Cut& cut = cuts[finish[k]];
    const int rows = rows_of(cut);
    const int64_t piece0 = quotient(cut.start, share);
    const int pieces = static_cast<int>(quotient(cut.start + cut.req.steps - 1, share) - piece0 + 1);
    const int groups = max(1, kWarps / rows);
    float* runs = reinterpret_cast<float*>(smem);  // [row][group][kRowPitch]: the ring and the partials are free
#pragma unroll 1
    for (int item = warp; item < rows * groups; item += kWarps) {
      const int row = item / groups, g = item % groups;
      const int i0 = pieces * g / groups, i1 = pieces * (g + 1) / groups;
      float top = kNoRef, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int base = i0; base < i1; base += 32) {
        const int i = base + lane;
        float2 ms = make_float2(kNoRef, 0.f);
        if (i < i1) ms = __ldcg(reinterpret_cast<const float2*>(slot_of(piece0 + i, i == 0) + row * kRowPitch + kKvDim));
        const int n = min(32, i1 - base);
        constexpr int kAhead = 8;  // outputs asked for together with the maxima
        float4 ahead[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          ahead[j] = j < n ? __ldcg(reinterpret_cast<const float4*>(
                                 slot_of(piece0 + base + j, base + j == 0) + row * kRowPitch + 4 * lane))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        float f, part_sum;
        const float part_top = join(ms.x, ms.y, f, part_sum);
        const float now = fmaxf(top, part_top);
        const float keep = exp2_approx(top - now), add = exp2_approx(part_top - now);
        top = now;
        sum = sum * keep + part_sum * add;
        acc.x *= keep;
        acc.y *= keep;
        acc.z *= keep;
        acc.w *= keep;
        f *= add;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const float w = __shfl_sync(0xFFFFFFFFu, f, j);
          if (j < n) {
            acc.x += ahead[j].x * w;
            acc.y += ahead[j].y * w;
            acc.z += ahead[j].z * w;
            acc.w += ahead[j].w * w;
          }
        }
#pragma unroll 8
        for (int j = kAhead; j < n; ++j) {
          const float w = __shfl_sync(0xFFFFFFFFu, f, j);
          const float4 v = __ldcg(reinterpret_cast<const float4*>(
              slot_of(piece0 + base + j, base + j == 0) + row * kRowPitch + 4 * lane));
          acc.x += v.x * w;
          acc.y += v.y * w;
          acc.z += v.z * w;
          acc.w += v.w * w;
        }
      }
      if (groups == 1) {
        store4(cut.req, cut.unit, row, acc, sum);
      } else {
        *reinterpret_cast<float4*>(runs + item * kRowPitch + 4 * lane) = acc;
        if (lane == 0) *reinterpret_cast<float2*>(runs + item * kRowPitch + kKvDim) = make_float2(top, sum);
      }
    }
    if (groups == 1) continue;
    __syncthreads();
    for (int row = warp; row < rows; row += kWarps) {
      float2 ms = make_float2(kNoRef, 0.f);
      if (lane < groups) ms = *reinterpret_cast<const float2*>(runs + (row * groups + lane) * kRowPitch + kKvDim);
      float f, sum;
      join(ms.x, ms.y, f, sum);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int g = 0; g < groups; ++g) {
        const float w = __shfl_sync(0xFFFFFFFFu, f, g);
        const float4 v = *reinterpret_cast<const float4*>(runs + (row * groups + g) * kRowPitch + 4 * lane);
        acc.x += v.x * w;
        acc.y += v.y * w;
        acc.z += v.z * w;
        acc.w += v.w * w;
      }
      store4(cut.req, cut.unit, row, acc, sum);
    }
    __syncthreads();
  }
}

template <int NT>
cudaError_t launch(const KvAttnParams& p, int sms, cudaStream_t stream) {
  using C = Cfg<NT>;
  static DeviceBits allowed{0};
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kv_stream_kernel<NT>), C::kSmem, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(sms, C::kThreads, C::kSmem, stream, attr);
  return cudaLaunchKernelEx(&cfg, kv_stream_kernel<NT>, p);
}

}  // namespace

cudaError_t launch_kv_stream(const KvAttnParams& p, int sms, cudaStream_t stream) {
  return p.max_q * static_cast<int64_t>(p.heads / p.kv_heads) <= 8 ? launch<1>(p, sms, stream) : launch<2>(p, sms, stream);
}

}  // namespace sg
