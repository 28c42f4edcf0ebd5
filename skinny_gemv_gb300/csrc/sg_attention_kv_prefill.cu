// Attention over the paged NVFP4 KV cache (sg_kv.cuh) for many query rows per
// request: prefill chunks against a cached prefix.  The same function as the
// streaming kernel (sg_attention_kv.cu); here the products bound it, so they run
// on tcgen05 and the cache is decoded once per 256 query rows.
//
// A unit is a run of whole query tokens of one request, at most 256 rows (row = token
// * (H / Hkv) + head of the group, so a group's heads share each decoded key and
// value), for one kv head, over the key blocks (128 keys) its last row sees.  TMEM holds
// two score buffers and two outputs of 128 rows.  More than 128 rows make two tiles,
// which share each decoded block; with fewer, the buffers take the blocks in turns and
// their sums are joined at the unit's end.  Either way the tensor core works for one
// buffer while the softmax of the other runs: for one it is a chain of S, softmax, P V.
//
// Schedule.  The units' blocks laid end to end (causal units by their own counts, each
// with a fixed cost for its start and end) are cut into equal runs, one per CTA, from
// the lengths on the device, as in the streaming kernel: with one CTA per unit the last
// of 1.3 waves left most SMs idle.  A CTA walks its run unit by unit; a unit cut between
// CTAs leaves one fp32 partial per CTA; neighbouring pieces are merged two by two by
// whichever CTA of the two arrives last, in a fixed tree.
//
// Measured: 8 kv heads of 4 query heads, chunks of 1536 and 511 tokens against 6000 and
// 511 keys and two decode rows, 163 us (820 TFLOP/s; 229 us with one 128-row tile per
// CTA and no equal shares); a chunk of 4096 tokens against 8192 keys, 64 heads on 8, 762
// us (1083 TFLOP/s of the 1967 that a large cuBLAS product reaches).  What bounds it is
// issue latency: a block of 128 keys x 256 rows keeps the tensor core busy for 2176
// clocks of some 3800; its issuing warp's waits and the softmax (1600 clocks a tile,
// twice per block, overlapped) take the rest, and a unit's start and end some 10 us.
//
//   warp 0        bulk copies of cache tiles into a raw ring (18 KB per block of 128
//                 keys instead of 64 KB decoded), the next keys before the last values
//   warp 1        TMEM allocator and MMA issuer; per block and buffer O += P V (bf16, P
//                 from TMEM), then the buffer's next S = Q K^T (fp16)
//   warp 2        works out the next unit
//   warps 4-19    Q of the unit (fp16, shifted by a power of two per row so that the row
//                 maximum is 2^13 .. 2^14); then softmax, eight warps per buffer, two
//                 threads per row (64 columns each, row maxima swapped through shared
//                 memory; the TMEM load itself gives the maximum of its columns); P
//                 written over S
//   warps 20-27   decode: per block each warp one cache tile, K to fp16 and V to bf16,
//                 exactly, in the 128-byte-swizzled layout the MMA reads (four warps on
//                 K and four on V wait for the slower V: 198 us against 183)
// P is rounded to bf16, half a step 2^-8 of a weight, and the row sums are of the rounded
// weights, so that an average stays one (summing them unrounded: 160 us for the chunks
// above).  The tensor core's fp32 additions truncate: about 2^-25 per 16 keys that a CTA
// adds up, 2.3% low at 14 million keys, below P's rounding up to some 2^21.
// V must be bf16 because P is (weights far below the row maximum count where every
// larger one meets a zero in V; fp16 would flush them).  E2M1 to bf16 is a shift and
// a mask: s eem -> s 000000ee m000000 is the value times 2^-126, and the block's
// scale is multiplied in as scale * 2^110, so V carries 2^-16, undone at the end.
// That extraction pairs elements i and i + 4 of a code word; V's dims stay in that
// order and the output's columns are put back in the last store.
//
// Keys are visible as a prefix [0, lim) of the request's keys.  Masked keys get
// weight 0, their V scales are 0 where the bytes belong to no token, and a NaN scale
// in V is taken out and remembered as the smallest such key per block of dims: a row
// whose prefix reaches it gets NaN there, and no other row does.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sg_internal.h"
#include "sg_kv.cuh"
#include "sg_ptx.cuh"

namespace sg {
namespace {

constexpr int kPfThreads = 896;
constexpr int kPfSoftWarp = 4, kPfDecWarp = 20, kPfDecWarps = 8;
// Registers per thread: 72 at launch (896 threads); then 40 for warps 0-3, 96 for the
// softmax and 40 for the decoders (40 + 4 * 96 + 2 * 40 = 7 * 72).
constexpr int kPfRegsLaunch = 72, kPfRegsIssue = 40, kPfRegsSoft = 96, kPfRegsDec = 40;
static_assert(kPfRegsIssue + 4 * kPfRegsSoft + 2 * kPfRegsDec == 7 * kPfRegsLaunch, "register split");
constexpr int kPfTileRows = 128, kPfRows = 2 * kPfTileRows, kPfKeys = 128, kPfTiles = kPfKeys / kKvTile;
constexpr int kPfBox = 128 * 128;              // 128 rows x 64 elements of 16 bits
constexpr int kPfHalfTile = kKvTileBytes / 2;  // the key or value half of a cache tile
constexpr int kPfRawBytes = kPfTiles * kPfHalfTile;
constexpr int kPfQOff = 0;                     // 2 tiles of 2 boxes
constexpr int kPfKOff = 4 * kPfBox;            // 2 buffers of 2 boxes
constexpr int kPfVOff = kPfKOff + 4 * kPfBox;
constexpr int kPfRawOff = kPfVOff + 4 * kPfBox;  // ring of kPfRaw halves: keys 0, values 0, keys 1, ...
constexpr int kPfRaw = 3;
// Their barriers: keys of even and odd blocks, then values (one per slot would do only
// for readers that take every load in order).
constexpr int kPfRawBars = 4;
constexpr int kPfBarOff = kPfRawOff + kPfRaw * kPfRawBytes;
// q, raw full/empty [kPfRawBars], k_full[2], k_empty[2], v_full[2], v_empty[2],
// s_full[2], p_ready[2], o_done[2], teardown
constexpr int kPfNumBars = 1 + 2 * kPfRawBars + 4 * 2 + 3 * 2 + 1;
constexpr int kPfScaleOff = kPfBarOff + kPfNumBars * 8;  // per row: score scale in log2 units
constexpr int kPfXchgOff = kPfScaleOff + kPfRows * 4;      // [turn & 1][score buffer][half][128 rows]
constexpr int kPfMiscOff = (kPfXchgOff + 2 * 2 * kPfRows * 4 + 15) / 16 * 16;
constexpr int kPfMiscBytes = 768;
constexpr int kPfSmem = kPfMiscOff + kPfMiscBytes + 1024;
static_assert(kKvVCodeOff == kPfHalfTile, "keys then values in a cache tile");
constexpr int kPfTmemCols = 512;
constexpr int kPfPartPitch = 132;         // floats per row of a part
constexpr int kPfUnitCost = 6;  // what starting and ending a unit costs, in blocks (about 10 us)
constexpr int kPfMinShare = kPfUnitCost + 4;  // cost per CTA, at least (above kPfUnitCost)
constexpr uint32_t kPfOCol = 256;  // S / P of tile x at 128 x, O at 256 + 128 x
constexpr float kPfRescaleLog2 = 8.f;
static_assert(kPfSmem <= 232448, "shared memory budget");

// Raw load 2 g + (0: keys, 1: values) of a CTA's block g: its barrier and phase.
__device__ __forceinline__ uint32_t raw_bar(uint32_t load) { return 2 * (load & 1u) + (load >> 1 & 1u); }
__device__ __forceinline__ uint32_t raw_phase(uint32_t load) { return load >> 2 & 1u; }

// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// a + b for two packed floats.
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// a b + c for two packed floats.
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ uint32_t pf_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void pf_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Eight E2M1 codes of a word to bf16 times scale * 2^-16, in the order 0, 4, 1, 5, 2,
// 6, 3, 7; s2 holds scale * 2^110 twice.
__device__ __forceinline__ uint32_t v_pair(uint32_t y, __nv_bfloat162 s2) {  // codes in bits 12-15 and 28-31
  const uint32_t b = (y & 0x80008000u) | ((y >> 6) & 0x01C001C0u);
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), s2);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint4 v_decode(uint32_t w, __nv_bfloat162 s2) {
  return make_uint4(v_pair(w << 12, s2), v_pair(w << 8, s2), v_pair(w << 4, s2), v_pair(w, s2));
}

// One request and its units for one kv head.
struct PfRequest {
  int32_t q0, nq, n;      // first query row, query tokens (-1: bad lengths), keys
  int32_t units;          // per kv head
};

// Query tokens per unit.
__device__ __forceinline__ int pf_tokens(int group) { return kPfRows / group; }

// sum over 0 <= i < n of floor((a i + c) / 128), reduced as in the Euclidean algorithm.
// a n + c stays below 2^32: it counts keys of one request.
__device__ __forceinline__ int64_t sum_of_blocks(uint32_t n, uint32_t a, uint32_t c) {
  uint32_t m = kPfKeys;
  int64_t sum = 0;
  while (n > 0) {
    sum += static_cast<int64_t>(n) * (n - 1) / 2 * (a / m) + static_cast<int64_t>(n) * (c / m);
    a %= m;
    c %= m;
    const uint32_t top = a * n + c;  // what is left: floor(top / m) steps of one, counted by where they fall
    n = top / m;
    c = top % m;
    const uint32_t swap = m;
    m = a;
    a = swap;
  }
  return sum;
}

// Key blocks of unit t (at least 1: a unit that sees no key still writes zeros).
__device__ __forceinline__ int pf_unit_blocks(const KvAttnParams& p, const PfRequest& r, int t, int tau) {
  const int64_t last = min(static_cast<int64_t>(r.nq), (t + 1) * static_cast<int64_t>(tau));
  const int64_t lim = p.causal ? r.n - r.nq + last : r.n;
  return lim <= 0 ? 1 : static_cast<int>((lim + kPfKeys - 1) / kPfKeys);
}

// Cost of the units before unit t, in blocks.
__device__ __forceinline__ int64_t pf_cost_before(const KvAttnParams& p, const PfRequest& r, int64_t t, int tau) {
  if (t <= 0) return 0;
  if (!p.causal) return t * (pf_unit_blocks(p, r, 0, tau) + kPfUnitCost);
  int64_t last = t * kPfUnitCost;  // and the blocks of the last unit, which may be short of tokens
  if (t == r.units) {
    last += pf_unit_blocks(p, r, r.units - 1, tau);
    t = r.units - 1;
  }
  const int64_t a = static_cast<int64_t>(r.n) - r.nq + tau;          // unit i sees a + i tau keys
  const int64_t blind = a >= 1 ? 0 : min(t, (1 - a + tau - 1) / tau);  // units that see none
  const int64_t first = a + blind * tau + kPfKeys - 1;
  return last + blind + sum_of_blocks(static_cast<uint32_t>(t - blind), tau, static_cast<uint32_t>(first));
}

__device__ __forceinline__ PfRequest pf_request(const KvAttnParams& p, int b, int tau) {
  PfRequest r;
  r.q0 = p.cu_q[b];
  const int32_t q1 = p.cu_q[b + 1];
  r.n = p.seq_lens[b];
  const bool bad = r.q0 < 0 || q1 < r.q0 || q1 > p.tokens || q1 - r.q0 > p.max_q || r.n < 0 ||
                   r.n > static_cast<int64_t>(p.max_pages) * p.cache.page_size;
  r.nq = bad ? -1 : q1 - r.q0;
  r.units = r.nq > 0 ? (r.nq + tau - 1) / tau : 0;
  return r;
}

// Where a CTA's run begins.
struct PfStart {
  int64_t at, per_head;  // cost before the request, cost per kv head
  PfRequest r;
  int32_t b;
};

// One segment: a CTA's blocks of one unit.  Kept in shared memory, so that no role
// carries what it does not use in registers.
struct PfSegment {
  int64_t unit_at, end;         // cost before the unit's first block, before the end of the CTA's run
  PfRequest r;
  int32_t b, head, unit, row0;  // row0: first row of the unit within the request
  int32_t rows, unit_blocks;
  int32_t j_begin, nblk;        // this CTA's blocks of the unit (nblk 0: no segment)
  int32_t done, done0, done1;   // before the segment: blocks, and those of the first and second score buffer
  int32_t seg1;                 // segments before that used the second
};

// Fills in what follows from the unit and the run's end.
__device__ __forceinline__ void pf_set_segment(const KvAttnParams& p, PfSegment* s, int tau, int group) {
  s->row0 = s->unit * tau * group;
  s->rows = min(tau, s->r.nq - s->unit * tau) * group;
  s->unit_blocks = pf_unit_blocks(p, s->r, s->unit, tau);
  const int64_t until = min(static_cast<int64_t>(s->unit_blocks), s->end - s->unit_at);
  s->nblk = static_cast<int>(max(int64_t(0), until - s->j_begin));
}

// Blocks of score buffer x: with more rows than a tile each buffer is a tile's, and takes
// every block; otherwise the two take turns.
__device__ __forceinline__ int pf_blocks_of(const PfSegment* s, int x) {
  return s->rows > kPfTileRows ? s->nblk : (s->nblk + 1 - x) / 2;
}

// The segment after `s`.
__device__ __forceinline__ void pf_next_segment(const KvAttnParams& p, const PfSegment* s, PfSegment* next, int tau,
                                                int group) {
  next->end = s->end;
  next->done = s->done + s->nblk;
  next->done0 = s->done0 + pf_blocks_of(s, 0);
  next->done1 = s->done1 + pf_blocks_of(s, 1);
  next->seg1 = s->seg1 + (pf_blocks_of(s, 1) > 0 ? 1 : 0);
  next->nblk = 0;
  next->unit_at = s->unit_at + s->unit_blocks + kPfUnitCost;
  if (next->unit_at >= s->end) return;
  next->j_begin = 0;
  next->r = s->r;
  next->b = s->b;
  next->head = s->head;
  next->unit = s->unit + 1;
  if (next->unit == next->r.units) {
    next->unit = 0;
    if (++next->head == p.kv_heads) {
      next->head = 0;
      do {
        if (++next->b >= p.batch) return;  // (not before the run's end)
        next->r = pf_request(p, next->b, tau);
      } while (next->r.units == 0);
    }
  }
  pf_set_segment(p, next, tau, group);
}

__global__ void __launch_bounds__(kPfThreads, 1) kv_prefill_kernel(const KvAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset, so that it stays a shared-memory address)
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + kPfBarOff);
  uint64_t* raw_full = q_full + 1;
  uint64_t* raw_empty = raw_full + kPfRawBars;
  uint64_t* k_full = raw_empty + kPfRawBars;
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* s_full = v_empty + 2;   // per score buffer
  uint64_t* p_ready = s_full + 2;   // per score buffer
  uint64_t* o_done = p_ready + 2;   // per score buffer: a unit's last product
  uint64_t* teardown = o_done + 2;
  float* row_scale = reinterpret_cast<float*>(smem + kPfScaleOff);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + kPfMiscOff);
  uint32_t* tmem_slot = misc;
  volatile uint32_t* abort_flag = misc + 1;
  volatile uint32_t* last_flag = misc + 2;
  uint32_t* nan_keys = misc + 4;          // [segment & 1][8] smallest key with a NaN V scale, per block
  volatile uint32_t* raw_ok = misc + 20;  // [kPfRaw] tiles loaded
  volatile uint32_t* blk_ok = misc + 24;  // [4] block j's tiles: blk_ok[j & 3]
  int64_t* scan = reinterpret_cast<int64_t*>(misc + 28);  // [warps]
  PfSegment* segments = reinterpret_cast<PfSegment*>(misc + 28 + 2 * (kPfThreads / 32));  // [segment & 3]
  PfStart* start = reinterpret_cast<PfStart*>(segments + 4);
  volatile uint32_t* never = misc + 3;    // 0
  static_assert((28 + 2 * (kPfThreads / 32)) * 4 + 4 * sizeof(PfSegment) + sizeof(PfStart) <= kPfMiscBytes, "misc");

  // workspace part of one CTA's piece of a unit: slot 1 if the unit begins there
  auto slot_of = [&](int64_t cta, bool first) {
    return p.partials + (2 * cta + (first ? 1 : 0)) * (kPfRows * kPfPartPitch);
  };
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int group = p.heads / p.kv_heads;
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- this CTA's run: units laid end to end, each its fixed cost and then its blocks
  const int tau = pf_tokens(group);
  int64_t share = 0, run0 = 0, run1 = 0;
  PfRequest r = {};
  int64_t work = 0, upto = 0, all = 0;  // cost of request `base + tid`, up to its end, of all
  auto count = [&](int base) {
    const int b = base + tid;
    work = 0;
    if (b < p.batch) {
      r = pf_request(p, b, tau);
      work = pf_cost_before(p, r, r.units, tau) * p.kv_heads;
    }
    int64_t v = work;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = v;
    __syncthreads();
    upto = all + v;
    for (int w = 0; w < kPfThreads / 32; ++w) {
      const int64_t part = scan[w];
      if (w < warp) upto += part;
      all += part;
    }
  };
#pragma unroll 1
  for (int base = 0; base < p.batch; base += kPfThreads) {
    count(base);
    if (r.nq < 0 && base + tid < p.batch && blockIdx.x == 0) record_error(p.err, kDevBadRequest, base + tid);
  }
  share = max((all + gridDim.x - 1) / static_cast<int64_t>(gridDim.x), static_cast<int64_t>(kPfMinShare));
  run0 = share * blockIdx.x;
  run1 = min(run0 + share, all);
  if (run0 >= run1) return;
  if (p.batch > kPfThreads) all = 0;
#pragma unroll 1
  for (int base = 0; base < p.batch; base += kPfThreads) {
    if (p.batch > kPfThreads) count(base);
    __syncthreads();  // (the scan is read)
    if (work > 0 && upto - work <= run0 && run0 < upto) {  // one thread of the CTA
      start->at = upto - work;
      start->per_head = work / p.kv_heads;
      start->r = r;
      start->b = base + tid;
    }
  }
  __syncthreads();
  if (warp == 0) {  // the unit inside the request: 32 probes at a time
    const int head = static_cast<int>((run0 - start->at) / start->per_head);
    const int64_t off = run0 - start->at - head * start->per_head;
    int64_t lo = 0, hi = start->r.units, before = 0;  // cost before lo <= off < cost before hi
    while (hi - lo > 1) {
      const int64_t step = (hi - lo + 31) / 32;
      const int64_t t = min(hi, lo + step * lane);
      const int64_t here = pf_cost_before(p, start->r, t, tau);
      const uint32_t below = __ballot_sync(0xFFFFFFFFu, t < hi && here <= off);
      const int k = 31 - __clz(below);  // lane 0 always holds
      before = __shfl_sync(0xFFFFFFFFu, here, k);
      hi = min(hi, lo + step * (k + 1));
      lo += step * k;
    }
    if (lane == 0) {
      PfSegment* s = segments;
      s->unit_at = start->at + head * start->per_head + before + kPfUnitCost;
      s->end = run1;
      s->r = start->r;
      s->b = start->b;
      s->head = head;
      s->unit = static_cast<int>(lo);
      s->j_begin = static_cast<int>(max(int64_t(0), off - before - kPfUnitCost));
      s->done = s->done0 = s->done1 = s->seg1 = 0;
      pf_set_segment(p, s, tau, group);
    }
  }
  if (tid == 0) {
    mbar_init(q_full, kPfDecWarp - kPfSoftWarp);
    for (int u = 0; u < kPfRawBars; ++u) {
      mbar_init(&raw_full[u], 1);
      mbar_init(&raw_empty[u], kPfDecWarps);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&k_full[u], kPfDecWarps);
      mbar_init(&k_empty[u], 1);
      mbar_init(&v_full[u], kPfDecWarps);
      mbar_init(&v_empty[u], 1);
      mbar_init(&s_full[u], 1);
      mbar_init(&p_ready[u], 2 * kPfTileRows);
      mbar_init(&o_done[u], 1);
    }
    mbar_init(teardown, 1);
    *abort_flag = 0;
    *never = 0;
    for (int i = 0; i < 16; ++i) nan_keys[i] = 0x7FFFFFFFu;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kPfTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Every role walks the CTA's segments by itself; all meet at the end of each.  The
  // decision to give up is the barrier's, so that all take it at the same one.
  auto walk = [&](auto&& role, auto&& after) -> bool {
#pragma unroll 1
    for (uint32_t seg = 0;; ++seg) {
      const PfSegment* const cur = segments + (seg & 3);
      if (cur->nblk == 0) return true;
      role(seg, cur);
      tc_fence_before();
      if (__syncthreads_or(static_cast<int>(*abort_flag))) return false;
      tc_fence_after();
      after(seg, cur);
    }
  };
  auto nothing = [](uint32_t, const PfSegment*) {};

  if (warp < kPfSoftWarp) regs_down<kPfRegsIssue>();
  if (warp == 0) {
    // ------------------------------------------------------------ raw tiles
    uint32_t sent = 0;  // loads issued so far
    const bool done_all = walk([&](uint32_t, const PfSegment* cur) {
      // Lanes 0-7 copy the key halves of a block's eight cache tiles, lanes 8-15 the value
      // halves.  Pages are looked up four blocks at a time (lane: block lane / 8, tile
      // lane % 8), a group ahead of the copies, and the tiles asked for into L2: the ring
      // holds too little to cover the latency of DRAM.
      const int b = cur->b, n = cur->r.n, kvh = cur->head, j_begin = cur->j_begin, nblk = cur->nblk, done = cur->done;
      const int tiles_per_page = p.cache.page_size / kKvTile;
      const int32_t* table = p.table + b * p.table_pitch;
      const int tl = lane & 7;
      const bool values = lane >= 8;
      auto look_up = [&](int j) -> const uint8_t* {  // of the group that begins with block j
        const int tile = (j_begin + j) * kPfTiles + lane;
        if (j + lane / kPfTiles >= nblk || static_cast<int64_t>(tile) * kKvTile >= n) return nullptr;
        const int at = tile / tiles_per_page;
        const int32_t page = table[at];
        if (page < 0 || page >= p.cache.num_pages) {
          record_error(p.err, kDevBadPage, b);
          return nullptr;
        }
        return kv_tile(p.cache, page, kvh, (tile - at * tiles_per_page) * kKvTile);
      };
      const uint8_t* group_now = nullptr;
      const uint8_t* group_next = look_up(0);
      if (group_next) bulk_prefetch_l2(group_next, kKvTileBytes);
      for (int j = 0; j < nblk; ++j) {
        if (j % 4 == 0) {
          group_now = group_next;
          group_next = look_up(j + 4);
          if (group_next) bulk_prefetch_l2(group_next, kKvTileBytes);
        }
        const uint8_t* src = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uintptr_t>(group_now), (j % 4) * kPfTiles + tl));
        const bool good = lane < 2 * kPfTiles && src != nullptr;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, good) & 0xFFu;
        bool ok = true;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t load = 2u * (done + j) + half, slot = load % kPfRaw;
          uint64_t* full = &raw_full[raw_bar(load)];
          // the load that used the slot last is decoded
          const uint32_t last = load - kPfRaw;
          ok = ok && (load < kPfRaw || mbar_wait(&raw_empty[raw_bar(last)], raw_phase(last), p.timeout_ns, abort_flag));
          if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
          if (lane == 0) {
            raw_ok[slot] = mask;
            mbar_arrive_expect_tx(full, __popc(mask) * kPfHalfTile + (load == 0 ? p.inject_extra_tx : 0u));
          }
          sent = load + 1;
          __syncwarp();
          if (good && values == (half != 0)) {
            fence_proxy_async_smem();
            bulk_load(smem + kPfRawOff + slot * kPfRawBytes + tl * kPfHalfTile, src + half * kPfHalfTile, kPfHalfTile,
                      full);
          }
        }
        if (!ok) {
          if (!*abort_flag && lane == 0) record_error(p.err, kDevTimeoutEmpty, j);
          *abort_flag = 1;
          break;
        }
      }
    }, nothing);
    if (!done_all)  // let the copies already issued land before the CTA exits
      for (uint32_t load = sent > kPfRaw ? sent - kPfRaw : 0; load < sent; ++load)
        mbar_wait(&raw_full[raw_bar(load)], raw_phase(load), p.timeout_ns, never);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    walk([&](uint32_t seg, const PfSegment* cur) {
      // The whole warp runs the loop and one elected lane issues, so that descriptors stay
      // in uniform registers (issued from a one-lane branch, each product first moves its
      // operands there and the issue, not the tensor core, sets the pace).
      constexpr uint32_t kIdescS = (1u << 4) | ((kPfKeys >> 3) << 17) | ((kPfTileRows >> 4) << 24);  // fp16, fp32 D
      constexpr uint32_t kIdescO = idesc_bf16_f32(kPfTileRows, kKvDim) | (1u << 16);               // B MN-major
      const uint32_t base = smem_u32(smem);
      // (broadcasts, so that what follows from them stays in uniform registers too)
      auto same = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
      const int nblk = same(cur->nblk), done = same(cur->done), done0 = same(cur->done0), done1 = same(cur->done1);
      const int turns = same(cur->rows) > kPfTileRows ? 1 : 2;  // 2: the score buffers take turns, block by block
      // descriptors: only the address field (16-byte units, low bits) changes
      const uint64_t q_desc = smem_desc_sw128(base + kPfQOff);
      const uint64_t k_desc = smem_desc_sw128(base + kPfKOff);
      const uint64_t v_desc = smem_desc_sw128_mn(base + kPfVOff, kPfBox);
      const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code, int where) -> bool {
        const bool came = mbar_wait(bar, parity, p.timeout_ns, abort_flag);
        if (__all_sync(0xFFFFFFFFu, came)) return true;
        if (lane == 0 && !*abort_flag) record_error(p.err, code, where);
        return false;
      };
      bool ok = wait(q_full, seg & 1u, kDevTimeoutFull, 0);
      auto wait_k = [&](int j) { return wait(&k_full[(done + j) & 1], ((done + j) >> 1) & 1u, kDevTimeoutFull, j); };
      // S of block j into buffer x (one lane); the keys are free after the last tile's
      auto issue_s = [&](int j, int x) {
        const uint32_t u = (done + j) & 1;
        const uint64_t qd = q_desc + (turns == 2 ? 0 : x) * (2 * kPfBox >> 4), kd = k_desc + u * (2 * kPfBox >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((kk >> 2) * kPfBox + (kk & 3) * 32) >> 4;
          tc_mma_bf16(tmem + x * kPfKeys, qd + off, kd + off, kIdescS, kk > 0 ? 1u : 0u);  // kind::f16: fp16
        }
        tc_commit(&s_full[x]);
        if (turns == 2 || x == 1) tc_commit(&k_empty[u]);
      };
      for (int x = 0; x < 2 && ok && (turns == 1 || x < nblk); ++x) {
        const int j = turns == 2 ? x : 0;
        ok = (turns == 1 && x == 1) || wait_k(j);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) issue_s(j, x);
        __syncwarp();
      }
      for (int j = 0; j < nblk && ok; ++j) {
        const uint32_t g = done + j, u = g & 1;
        const uint64_t vd = v_desc + u * (2 * kPfBox >> 4);
        for (int x = turns == 2 ? j & 1 : 0; x < 2 && ok; x += turns) {
          const uint32_t ph = ((x ? done1 : done0) + j / turns) & 1u;
          const bool more = j + turns < nblk;
          ok = ((turns == 1 && x == 1) || wait(&v_full[u], (g >> 1) & 1u, kDevTimeoutFull, j)) &&
               (turns == 2 || x == 1 || !more || wait_k(j + 1)) && wait(&p_ready[x], ph, kDevTimeoutTmemEmpty, j);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc_mma_bf16_ts(tmem + kPfOCol + x * kKvDim, tmem + x * kPfKeys + kk * 8, vd + (kk * 2048 >> 4), kIdescO,
                             (j >= turns || kk > 0) ? 1u : 0u);
            if (turns == 2 || x == 1) tc_commit(&v_empty[u]);
            if (!more) tc_commit(&o_done[x]);
            // the product above reads P where the next S goes: the tensor core runs them in order
            if (more && turns == 1) issue_s(j + 1, x);
          }
          __syncwarp();
          if (more && turns == 2) {
            ok = wait_k(j + 2);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) issue_s(j + 2, x);
            __syncwarp();
          }
        }
      }
      if (!ok) *abort_flag = 1;
      if (__any_sync(0xFFFFFFFFu, *abort_flag != 0)) {
        if (elect_one()) tc_commit(teardown);
        __syncwarp();
        if (!mbar_wait(teardown, 0, p.timeout_ns, never) && lane == 0) record_error(p.err, kDevTimeoutTeardown, 0);
        __syncwarp();
      }
    }, nothing);
    tc_fence_after();
    tmem_dealloc(*tmem_slot, kPfTmemCols);
  } else if (warp < kPfSoftWarp) {
    // ------------------------------------------------------------ next segment
    walk([&](uint32_t seg, const PfSegment* cur) {
      if (warp == 2 && lane == 0) pf_next_segment(p, cur, segments + ((seg + 1) & 3), tau, group);
      if (warp == 3 && lane < 8) nan_keys[((seg & 1) ^ 1) * 8 + lane] = 0x7FFFFFFFu;
    }, nothing);
  } else if (warp >= kPfDecWarp) {
    // ------------------------------------------------------------ decode
    regs_down<kPfRegsDec>();
    walk([&](uint32_t seg, const PfSegment* cur) {
      uint32_t* nan_key = nan_keys + (seg & 1) * 8;
      const int dw = warp - kPfDecWarp;
      const int n = cur->r.n, j_begin = cur->j_begin, nblk = cur->nblk, done = cur->done;
      const int g8 = lane / 4, t4 = lane % 4;
      const int tl = dw;  // this warp's tile of a block, keys and values
      static_assert(kPfDecWarps == kPfTiles, "a warp per cache tile");
      for (int j = 0; j < nblk; ++j) {
        const int g = done + j, u = g & 1;
        const uint32_t ph = (g >> 1) & 1u;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t load = 2u * g + half, slot = load % kPfRaw;
          const bool ok = mbar_wait(&raw_full[raw_bar(load)], raw_phase(load), p.timeout_ns, abort_flag) &&
                          mbar_wait(half ? &v_empty[u] : &k_empty[u], ph ^ 1u, p.timeout_ns, abort_flag);
          if (!__all_sync(0xFFFFFFFFu, ok)) {
            if (!*abort_flag && lane == 0) record_error(p.err, kDevTimeoutFull, j);
            *abort_flag = 1;
            j = nblk;
            break;
          }
          const uint8_t* tile = smem + kPfRawOff + slot * kPfRawBytes + tl * kPfHalfTile;
          const uint32_t loaded = raw_ok[slot];
          if (half == 0) {
            if (dw == 0 && lane == 0) blk_ok[g & 3] = loaded;
            {
              uint8_t* box = smem + kPfKOff + u * 2 * kPfBox + (t4 >> 1) * kPfBox;
              const uint32_t sc = *reinterpret_cast<const uint32_t*>(tile + kKvKScaleOff + 4 * lane);
#pragma unroll
              for (int h = 0; h < 2; ++h) {  // keys g8 and g8 + 8: dims 32 t4 .. 32 t4 + 31
                const uint4 c = *reinterpret_cast<const uint4*>(tile + 512 * h + 16 * lane);
                const __half2 s2 = e4m3x2_half2((sc >> (16 * h)) & 0xFFFFu);
                // words in the order 0 1 2 3, or 2 3 0 1 for t4 >= 2: eight lanes of a store
                // then hit eight different 16-byte bank groups
                const bool flip = t4 >= 2;
                const uint32_t w[4] = {flip ? c.z : c.x, flip ? c.w : c.y, flip ? c.x : c.z, flip ? c.y : c.w};
                const __half2 sf = flip ? __lowhigh2highlow(s2) : s2;
                const int r = 16 * tl + 8 * h + g8;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int chunk = 4 * (t4 & 1) + (k ^ (flip ? 2 : 0));
                  uint32_t o[4];
                  e2m1x8_times(w[k], k < 2 ? __low2half2(sf) : __high2half2(sf), o);
                  *reinterpret_cast<uint4*>(box + r * 128 + ((chunk ^ (r & 7)) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
              }
            }
          } else {
            const int key0 = (j_begin + j) * kPfKeys;
            {
              uint32_t sc = *reinterpret_cast<const uint32_t*>(tile + (kKvVScaleOff - kPfHalfTile) + 4 * lane);
              const int live = loaded >> tl & 1u ? n - (key0 + 16 * tl) : 0;  // keys of the tile that hold tokens
              const uint32_t low7 = sc & 0x7F7F7F7Fu;
              // a byte of 0x7f: adding 1 carries into its top bit
              if (live < 16 || ((low7 + 0x01010101u) & 0x80808080u)) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int key = 2 * t4 + (k & 1) + 8 * (k >> 1);
                  const bool nan = key < live && ((sc >> (8 * k)) & 0x7Fu) == 0x7Fu;
                  if (nan) atomicMin(&nan_key[g8], static_cast<uint32_t>(key0 + 16 * tl + key));
                  if (nan || key >= live) sc &= ~(0xFFu << (8 * k));
                }
              }
              uint8_t* box = smem + kPfVOff + u * 2 * kPfBox + (g8 >> 2) * kPfBox;  // lane: dims 16 g8 .. + 15
#pragma unroll
              for (int h = 0; h < 2; ++h) {  // keys 2 t4 + 8 h and the next
                const uint4 c = *reinterpret_cast<const uint4*>(tile + 512 * h + 16 * lane);
                const float2 f = __half22float2(e4m3x2_half2((sc >> (16 * h)) & 0xFFFFu));
                const __nv_bfloat162 sa = __float2bfloat162_rn(f.x * 0x1p110f), sb = __float2bfloat162_rn(f.y * 0x1p110f);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int r = 16 * tl + 8 * h + 2 * t4 + k;
                  const uint32_t w0 = k ? c.z : c.x, w1 = k ? c.w : c.y;
                  const bool flip = g8 & 1;  // odd blocks store their second chunk first (bank groups)
#pragma unroll
                  for (int i2 = 0; i2 < 2; ++i2) {
                    const int chunk = (2 * g8 + (i2 ^ (flip ? 1 : 0))) & 7;
                    *reinterpret_cast<uint4*>(box + r * 128 + ((chunk ^ (r & 7)) * 16)) =
                        v_decode((i2 != 0) == flip ? w0 : w1, k ? sb : sa);
                  }
                }
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(half ? &v_full[u] : &k_full[u]);
            mbar_arrive(&raw_empty[raw_bar(load)]);
          }
        }
      }
    }, nothing);
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    regs_up<kPfRegsSoft>();
    walk([&](uint32_t seg, const PfSegment* cur) {
      const uint32_t* nan_key = nan_keys + (seg & 1) * 8;
      // Q: a warp per row at a time, lane l holds dims 4 l .. 4 l + 3; kRowsAhead rows
      // asked for together, whose places the first lanes work out
      constexpr int kRowsAhead = 8, kSoftWarps = kPfDecWarp - kPfSoftWarp;
      const int tiles = cur->rows > kPfTileRows ? 2 : 1;
#pragma unroll 1
      for (int base = (warp - kPfSoftWarp) * kRowsAhead; base < tiles * kPfTileRows; base += kSoftWarps * kRowsAhead) {
        const int rr = cur->row0 + base + lane % kRowsAhead;
        const int64_t at = static_cast<int64_t>(cur->r.q0 + rr / group) * p.ldq +
                           static_cast<int64_t>(cur->head * group + rr % group) * kKvDim;
        const int live = cur->rows - base;
        uint2 v[kRowsAhead];
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
          const int64_t from = __shfl_sync(0xFFFFFFFFu, at, i);
          v[i] = i < live ? *reinterpret_cast<const uint2*>(p.Q + from + 4 * lane) : make_uint2(0u, 0u);
        }
        const float sign = p.scale_log2 < 0.f ? -1.f : p.scale_log2 == 0.f ? 0.f : 1.f;
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
          const int r = base + i;
          uint32_t top = max(max(v[i].x & 0x7FFFu, (v[i].x >> 16) & 0x7FFFu),
                             max(v[i].y & 0x7FFFu, (v[i].y >> 16) & 0x7FFFu));
          top = __reduce_max_sync(0xFFFFFFFFu, top);
          const int e = top == 0 ? 0 : max(-100, min(127, static_cast<int>(top >> 7) - 127));
          // 2^(13 - e) and the scale's sign (with scale 0 every score is 0); a row with a NaN
          // or an infinity becomes NaN as a whole, as its softmax is (infinite scores of one
          // sign would all be -inf and pass for masked keys)
          const float up = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __int_as_float((127 + 13 - e) << 23) * sign;
          const uint32_t lo = half2_bits(
              __floats2half2_rn(__uint_as_float(v[i].x << 16) * up, __uint_as_float(v[i].x & 0xFFFF0000u) * up));
          const uint32_t hi = half2_bits(
              __floats2half2_rn(__uint_as_float(v[i].y << 16) * up, __uint_as_float(v[i].y & 0xFFFF0000u) * up));
          const int chunk = (lane / 2) & 7;
          uint8_t* box = smem + kPfQOff + (2 * (r / kPfTileRows) + lane / 16) * kPfBox + (r % kPfTileRows) * 128;
          *reinterpret_cast<uint2*>(box + ((chunk ^ (r & 7)) * 16) + (lane & 1) * 8) = make_uint2(lo, hi);
          // (at least 2^-126: an underflow to 0 would turn masked scores, -inf, into NaN)
          if (lane == 0)
            row_scale[r] =
                sign == 0.f ? 1.f : fmaxf(__int_as_float((127 - 13 + e) << 23) * fabsf(p.scale_log2), 0x1p-126f);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      const int x = (warp - kPfSoftWarp) >> 3;           // score buffer
      const int turns = cur->rows > kPfTileRows ? 1 : 2;
      const int half = ((warp - kPfSoftWarp) >> 2) & 1;  // which 64 columns of its rows
      const int q = warp & 3;                            // TMEM lane quarter
      const int r = (turns == 2 ? 0 : x * kPfTileRows) + q * 32 + lane;  // row of the unit
      const uint32_t lanes = *tmem_slot + (static_cast<uint32_t>(q * 32) << 16);
      const uint32_t s_col = lanes + x * kPfKeys, o_col = lanes + kPfOCol + x * kKvDim + half * 64;
      // keys visible to the row: [0, lim_row())
      auto lim_row = [&]() -> int {
        if (r >= cur->rows) return 0;
        const int n = cur->r.n;
        return p.causal ? max(0, min(n, n - cur->r.nq + (cur->row0 + r) / group + 1)) : n;
      };
      const int lim = lim_row() - cur->j_begin * kPfKeys - half * 64;
      const int blocks = pf_blocks_of(cur, x), ahead = x ? cur->done1 : cur->done0, blocks_before = cur->done;
      const int pair_bar = 1 + 4 * x + q;                // the two warps of these 32 rows
      // [turn & 1][score buffer][half][row]: a buffer is written again two blocks later, when the
      // partner has passed the barrier in between and so read it
      float* mine = reinterpret_cast<float*>(smem + kPfXchgOff) + x * 256 + half * 128 + q * 32 + lane;
      float* other = mine + (half ? -128 : 128);
      float m_run = -INFINITY, l_run = 0.f, scale = 0.f;
      bool ok = true;
      auto give_up = [&](int where) {
        if (!*abort_flag && lane == 0) record_error(p.err, kDevTimeoutTmemFull, where);
        __syncwarp();
        *abort_flag = 1;
      };
      for (int i = 0; i < blocks; ++i) {
        const int j = turns * i + (turns == 2 ? x : 0);  // block of the segment

        // After a wait that ran out (`ok` false) a warp goes on with what is there, without
        // waiting again, so that both warps of a row still meet at every barrier; nothing
        // is stored in the end.
        ok = ok && mbar_wait(&s_full[x], (ahead + i) & 1u, p.timeout_ns, abort_flag);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) give_up(j);
        tc_fence_after();
        if (i == 0) scale = row_scale[r];  // written before Q was handed over
        uint32_t sv[2][32];
        float mx2[2];
        tmem_ld_max_32x32b_x32(s_col + half * 64, sv[0], mx2[0]);
        tmem_ld_max_32x32b_x32(s_col + half * 64 + 32, sv[1], mx2[1]);
        const int kv = lim - j * kPfKeys;  // columns of this half visible: [0, kv)
        const uint32_t bad = ~blk_ok[(blocks_before + j) & 3] & 0xFFu;
        tmem_ld_wait(sv[0]);
        tmem_ld_wait(sv[1]);
        asm volatile("" : "+f"(mx2[0]), "+f"(mx2[1]));  // (there after the wait, too)
        float mx = fmaxf(mx2[0], mx2[1]);
        if (kv < 64 || bad != 0) {
          mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (32 * c + e >= kv || (bad >> (half * 4 + 2 * c + e / 16) & 1u)) sv[c][e] = 0xFF800000u;  // -inf
              mx = fmaxf(mx, __uint_as_float(sv[c][e]));
            }
        }
        mine[(i & 1) * 512] = mx;
        pf_bar(pair_bar, 64);  // (so both have S in registers before either writes P over it)
        mx = fmaxf(mx, other[(i & 1) * 512]) * scale;  // log2 units (scale > 0)
        const bool move = mx > m_run + kPfRescaleLog2;
        const float m_new = move ? mx : m_run;
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = move ? exp2_approx(m_run - m_use) : 1.f;  // 0 while nothing was visible yet
        m_run = m_new;
        // (S of this block is there, so the product of the last one is done with O)
        if (i > 0 && __any_sync(0xFFFFFFFFu, move)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t ov[16];
            tmem_ld_32x32b_x16(o_col + 16 * c, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st_32x32b_x16(o_col + 16 * c, ov);
          }
        }
        uint64_t sums[2] = {0, 0};
        const uint64_t scale2 = pack_f32x2(scale, scale), minus2 = pack_f32x2(-m_use, -m_use);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint64_t xs = pack_f32x2(__uint_as_float(sv[c][2 * e]), __uint_as_float(sv[c][2 * e + 1]));
            const uint64_t y = fma_f32x2(xs, scale2, minus2);
            const float p0 = exp2_approx(__uint_as_float(static_cast<uint32_t>(y)));
            const float p1 = exp2_approx(__uint_as_float(static_cast<uint32_t>(y >> 32)));
            pk[e] = pf_pack(p0, p1);
            // (the sum is of the weights that the product takes)
            sums[e & 1] = add_f32x2(sums[e & 1], pack_f32x2(__uint_as_float(pk[e] << 16),
                                                            __uint_as_float(pk[e] & 0xFFFF0000u)));
          }
          tmem_st_32x32b_x16(s_col + 32 * half + 16 * c, pk);
        }
        sums[0] = add_f32x2(sums[0], sums[1]);
        l_run = l_run * alpha + (__uint_as_float(static_cast<uint32_t>(sums[0])) +
                                 __uint_as_float(static_cast<uint32_t>(sums[0] >> 32)));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_ready[x]);
      }
      if (blocks > 0) {  // the row's total weight: both halves' sums
        mine[(blocks & 1) * 512] = l_run;
        pf_bar(pair_bar, 64);
        l_run += other[(blocks & 1) * 512];
      }
      const bool joined = turns == 2 && cur->nblk > 1;  // both buffers hold some of the rows' sums
      bool have_o = ok && blocks > 0;

      if (have_o) have_o = mbar_wait(&o_done[x], (x ? cur->seg1 : seg) & 1u, p.timeout_ns, abort_flag);
      if (have_o && joined && x == 1) have_o = mbar_wait(&o_done[0], seg & 1u, p.timeout_ns, abort_flag);
      have_o = __all_sync(0xFFFFFFFFu, have_o);
      if (blocks > 0 && !have_o) give_up(cur->nblk);
      tc_fence_after();
      // the second buffer's sums go to the first's threads, through the tiles of K and V
      // (no product reads them any more)
      float mine_f = 1.f, other_f = 0.f;
      float* swap = reinterpret_cast<float*>(smem + kPfKOff) + (q * 32 + lane) * kPfPartPitch;
      if (joined) {
        if (x == 1) {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t ov[32];
            tmem_ld_32x32b_x32(o_col + 32 * c, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(swap + half * 64 + 32 * c + 4 * e) =
                  make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
          }
          if (half == 0) *reinterpret_cast<float2*>(swap + kKvDim) = make_float2(m_run, l_run);
        }
        pf_bar(9, 4 * kPfTileRows);
        if (x == 0) {
          const float2 ml = *reinterpret_cast<const float2*>(swap + kKvDim);
          const float top = fmaxf(m_run, ml.x), use = top == -INFINITY ? 0.f : top;
          mine_f = exp2_approx(m_run - use);
          other_f = exp2_approx(ml.x - use);
          l_run = l_run * mine_f + ml.y * other_f;
          m_run = top;
        }
      }
      const bool writes = turns == 1 || x == 0;
      const bool store = r < cur->rows && !*abort_flag;
      const bool cut = cur->nblk < cur->unit_blocks;
      const int seen = lim_row();
      const int rr = cur->row0 + r;
      uint16_t* orow = p.O + static_cast<int64_t>(cur->r.q0 + rr / group) * p.ldo +
                       static_cast<int64_t>(cur->head * group + rr % group) * kKvDim + half * 64;
      // cut unit: this CTA's part, [256 rows][132]: output (times 2^16), maximum, sum
      float* part = slot_of(blockIdx.x, cur->j_begin == 0) + r * kPfPartPitch;
      const float inv = l_run == 0.f ? 0.f : p.v_scale * 0x1p16f / l_run;
#pragma unroll 1
      for (int c = 0; c < 2 && writes; ++c) {
        uint32_t ov[32];
        if (have_o) {
          tmem_ld_32x32b_x32(o_col + 32 * c, ov);
          tmem_ld_wait(ov);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = 0u;
        }
        if (joined) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 o4 = *reinterpret_cast<const float4*>(swap + half * 64 + 32 * c + 4 * e);
            const float f4[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ov[4 * e + k] = __float_as_uint(__uint_as_float(ov[4 * e + k]) * mine_f + f4[k] * other_f);
          }
        }
        if (!store) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 8 dims, held in the order 0 4 1 5 2 6 3 7
          const int blk = (64 * half + 32 * c + 8 * k) / kKvBlock;
          const bool nan = seen > 0 && static_cast<uint32_t>(seen) > nan_key[blk];
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            f[(e >> 1) + 4 * (e & 1)] = nan ? __uint_as_float(0x7FC00000u) : __uint_as_float(ov[8 * k + e]);
          if (!cut) {
            *reinterpret_cast<uint4*>(orow + 32 * c + 8 * k) =
                make_uint4(pf_pack(f[0] * inv, f[1] * inv), pf_pack(f[2] * inv, f[3] * inv),
                           pf_pack(f[4] * inv, f[5] * inv), pf_pack(f[6] * inv, f[7] * inv));
          } else {
            float* dst = part + half * 64 + 32 * c + 8 * k;
            __stcg(reinterpret_cast<float4*>(dst), make_float4(f[0], f[1], f[2], f[3]));
            __stcg(reinterpret_cast<float4*>(dst + 4), make_float4(f[4], f[5], f[6], f[7]));
          }
        }
      }
      if (cut && store && writes && half == 0)
        __stcg(reinterpret_cast<float2*>(part + kKvDim), make_float2(l_run == 0.f ? -1e30f : m_run, l_run));
    }, [&](uint32_t, const PfSegment* cur) {
      if (cur->nblk < cur->unit_blocks) {
        // Cut unit: its pieces' parts are merged two by two, in a tree over the pieces in
        // order; of two neighbours the one that arrives last merges both (64 tokens against
        // 65536 keys, 19 pieces a unit: 118 us; with one CTA merging them all 26 more).
        const int64_t piece0 = cur->unit_at / share;
        const int pieces = static_cast<int>((cur->unit_at + cur->unit_blocks - 1) / share - piece0 + 1);
        int first = static_cast<int>(blockIdx.x - piece0);  // of the pieces merged here so far
        for (int width = 1; width < pieces; width *= 2) {
          const int left = first & ~width, right = first | width;
          if (right >= pieces) continue;
          if (tid == kPfSoftWarp * 32) {
            uint32_t* counter = p.counters + piece0 + right;  // (a piece is the first right one of one pair)
            __threadfence();  // the CTA's part (seen through the barrier) before the count
            const uint32_t arrived = atomicAdd(counter, 1u);
            *last_flag = arrived;
            if (arrived == 1) *counter = 0;  // ready for the next launch
            __threadfence();
          }
          pf_bar(10, 4 * kPfTileRows);
          if (*last_flag == 0) break;
          const bool whole = left == 0 && 2 * width >= pieces;
          float* const into = slot_of(piece0 + left, left == 0);
          const float* const other = slot_of(piece0 + right, false);
          constexpr int kRows = 4;  // asked for together
          constexpr int kWarps = kPfDecWarp - kPfSoftWarp;
          for (int row0 = warp - kPfSoftWarp; row0 < cur->rows; row0 += kWarps * kRows) {
            float2 ma[kRows], mb[kRows];
            float4 va[kRows], vb[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
              const int at = min(row0 + kWarps * k, cur->rows - 1) * kPfPartPitch;
              va[k] = __ldcg(reinterpret_cast<const float4*>(into + at + 4 * lane));
              vb[k] = __ldcg(reinterpret_cast<const float4*>(other + at + 4 * lane));
              ma[k] = __ldcg(reinterpret_cast<const float2*>(into + at + kKvDim));
              mb[k] = __ldcg(reinterpret_cast<const float2*>(other + at + kKvDim));
            }
            __syncwarp();  // (a part is written over below)
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
              const int row = row0 + kWarps * k;
              if (row >= cur->rows) break;
              const float top = fmaxf(ma[k].x, mb[k].x);
              const float fa = exp2_approx(ma[k].x - top), fb = exp2_approx(mb[k].x - top);
              const float sum = ma[k].y * fa + mb[k].y * fb;
              const float4 o = make_float4(va[k].x * fa + vb[k].x * fb, va[k].y * fa + vb[k].y * fb,
                                           va[k].z * fa + vb[k].z * fb, va[k].w * fa + vb[k].w * fb);
              if (!whole) {
                __stcg(reinterpret_cast<float4*>(into + row * kPfPartPitch + 4 * lane), o);
                if (lane == 0) __stcg(reinterpret_cast<float2*>(into + row * kPfPartPitch + kKvDim), make_float2(top, sum));
              } else {
                const float inv = sum == 0.f ? 0.f : p.v_scale * 0x1p16f / sum;
                const int rr = cur->row0 + row;
                *reinterpret_cast<uint2*>(p.O + static_cast<int64_t>(cur->r.q0 + rr / group) * p.ldo +
                                          static_cast<int64_t>(cur->head * group + rr % group) * kKvDim + 4 * lane) =
                    make_uint2(pf_pack(o.x * inv, o.y * inv), pf_pack(o.z * inv, o.w * inv));
              }
            }
          }
          first = left;
          pf_bar(10, 4 * kPfTileRows);
        }
      }
    });
  }
}

}  // namespace

cudaError_t launch_kv_prefill(const KvAttnParams& p, int ctas, cudaStream_t stream) {
  static DeviceBits allowed{0};
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kv_prefill_kernel), kPfSmem, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config(ctas, kPfThreads, kPfSmem, stream, attr);
  return cudaLaunchKernelEx(&cfg, kv_prefill_kernel, p);
}

}  // namespace sg
