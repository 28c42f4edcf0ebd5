// Kernels around the paged NVFP4 KV cache (sg_kv.cuh): page assignment, the
// quantised append and the read-back.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sg_internal.h"
#include "sg_kv.cuh"
#include "sg_ptx.cuh"

namespace sg {
namespace {

// ------------------------------------------------------------ page assignment
// Inclusive block scan (sum) over THREADS threads; `warp_sums` is scratch of 32
// values.  Ends with a barrier, so the scratch may be reused at once.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (THREADS == 1024) {
    if (warp == 0) {
      int64_t s = warp_sums[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
      }
      warp_sums[lane] = s;
    }
    __syncthreads();
    if (warp > 0) v += warp_sums[warp - 1];
  } else {
    for (int w = 0; w < warp; ++w) v += warp_sums[w];
  }
  __syncthreads();
  return v;
}

// Every CTA scans the requests' token and page counts for itself (requests are
// few, and a scan from L2 costs less than a second launch), then the CTAs share
// the token rows, four consecutive rows per thread: row t of request b at position
// p = len + i takes slot page * P + p % P, and the row at a page's first position
// also writes the page into the block table, so every new page is written once.
// A small step (a decode batch) is one CTA of 128 threads: barriers of 32 warps cost
// it 1 us.  All positions fit 31 bits (total_lens is int32), so divisions are 32-bit.
// Bound by latency (two scans, then one dependent read and the stores): measured 5.2 us
// for 64 requests, 10.2 us for 257 requests with a million new tokens (8.5 MB).
template <int THREADS>
__global__ void __launch_bounds__(THREADS) kv_pages_kernel(const KvPagesParams p) {
  extern __shared__ int32_t smem[];
  int32_t* end = smem;                // [requests] token rows up to and with request b
  int32_t* first = smem + p.requests; // [requests] free-list index of b's first new page; -1: not served
  __shared__ int64_t sums[32];
  __shared__ int64_t bcast[2];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t head = *p.free_head;
  const uint32_t P = static_cast<uint32_t>(p.page_size);
  auto pages_of = [&](int64_t n) -> int64_t { return (static_cast<uint32_t>(n) + P - 1) / P; };  // n in [0, 2^31)
  int64_t tokens_done = 0, pages_done = 0, taken = 0;
  int32_t refused = 0;
  for (int base = 0; base < p.requests; base += THREADS) {
    const int b = base + threadIdx.x;
    const bool in = b < p.requests;
    const int64_t len = in ? p.seq_lens[b] : 0, fresh = in ? p.new_lens[b] : 0;
    const int64_t upto = tokens_done + block_scan<THREADS>(fresh > 0 ? fresh : 0, sums);
    const bool sane = in && len >= 0 && fresh >= 0 && len + fresh <= INT32_MAX;
    const int64_t want = sane ? pages_of(len + fresh) : 0;
    bool fits = sane && want <= p.max_pages && upto <= p.tokens;
    const int64_t need = fits ? want - pages_of(len) : 0;
    const int64_t pages = pages_done + block_scan<THREADS>(need, sums);
    // a request that needs no page is served whatever the free list holds
    fits = fits && (need == 0 || (head >= 0 && head + pages <= p.num_free));
    if (in) {
      end[b] = static_cast<int32_t>(min(upto, static_cast<int64_t>(INT32_MAX)));
      first[b] = fits ? static_cast<int32_t>(need ? head + pages - need : 0) : -1;
      refused += fits ? 0 : 1;
      taken += fits ? need : 0;
    }
    if (threadIdx.x == THREADS - 1) {
      bcast[0] = upto;
      bcast[1] = pages;
    }
    __syncthreads();
    tokens_done = bcast[0];
    pages_done = bcast[1];
    __syncthreads();
  }
  // every input has been read: outputs may now replace seq_lens and free_head (a
  // launch of one CTA)
  if (blockIdx.x == 0) {
    taken = block_scan<THREADS>(taken + (static_cast<int64_t>(refused) << 40), sums);  // both sums at once
    if (threadIdx.x == THREADS - 1) {
      *p.free_head_out = static_cast<int32_t>(head + (taken & ((int64_t(1) << 40) - 1)));
      *p.unserved = static_cast<int32_t>(taken >> 40);
    }
  }
  const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x) * 4; t0 < p.tokens;
       t0 += static_cast<int64_t>(gridDim.x) * THREADS * 4) {
    int32_t slot[4] = {-1, -1, -1, -1}, pos[4] = {0, 0, 0, 0};
    if (t0 < tokens_done) {
      int b = 0;
      for (int hi = p.requests - 1; b < hi;) {  // the first request whose end exceeds t0
        const int mid = (b + hi) / 2;
        if (end[mid] > t0) hi = mid; else b = mid + 1;
      }
      int at = -1;          // request the state below belongs to
      uint32_t len = 0, have = 0, start = 0, held = 0xFFFFFFFFu;
      int32_t page = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + i;
        if (t >= tokens_done || t >= p.tokens) break;
        while (end[b] <= t) ++b;
        if (first[b] < 0) continue;
        if (b != at) {
          at = b;
          len = static_cast<uint32_t>(p.seq_lens[b]);
          have = static_cast<uint32_t>(pages_of(len));
          start = b > 0 ? static_cast<uint32_t>(end[b - 1]) : 0u;
          held = 0xFFFFFFFFu;
        }
        const uint32_t where = len + static_cast<uint32_t>(t) - start, k = where / P, off = where - k * P;
        int32_t* entry = p.table + b * p.table_pitch + k;
        if (k != held) {
          held = k;
          page = k < have ? *entry : p.free_pages[first[b] + (k - have)];
        }
        if (k >= have && off == 0) *entry = page;
        const int64_t s = static_cast<int64_t>(page) * P + off;
        if (page >= 0 && s <= INT32_MAX) {
          slot[i] = static_cast<int32_t>(s);
          pos[i] = static_cast<int32_t>(where);
        } else {
          record_error(p.err, kDevBadPage, b);
        }
      }
    }
    if (wide && t0 + 4 <= p.tokens) {
      *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int i = 0; i < 4 && t0 + i < p.tokens; ++i) {
        p.slots[t0 + i] = slot[i];
        p.positions[t0 + i] = pos[i];
      }
    }
  }
  __syncthreads();  // a launch of one CTA may write over seq_lens
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; b < p.requests;
       b += static_cast<int64_t>(gridDim.x) * THREADS) {
    const int32_t len = p.seq_lens[b];
    p.total_lens[b] = first[b] >= 0 ? len + p.new_lens[b] : len;
    p.cu_new[b + 1] = end[b];
    if (b == 0) p.cu_new[0] = 0;
  }
  if (p.requests == 0 && blockIdx.x == 0 && threadIdx.x == 0) p.cu_new[0] = 0;
}

// ------------------------------------------------------------ append and read
constexpr int kRowThreads = 256;

// The cache place of (token, kv head): false if the token is
// skipped or its slot lies past the cache.
__device__ __forceinline__ bool kv_place(const KvRowsParams& p, uint32_t t, uint32_t h, uint8_t** tile, int* r) {
  const int32_t slot = p.slots[t];
  if (slot < 0) return false;
  const uint32_t P = static_cast<uint32_t>(p.cache.page_size);
  const uint32_t page = static_cast<uint32_t>(slot) / P, off = static_cast<uint32_t>(slot) - page * P;
  if (page >= static_cast<uint32_t>(p.cache.num_pages)) {
    record_error(p.err, kDevBadSlot, t);
    return false;
  }
  *tile = kv_tile(p.cache, static_cast<int32_t>(page), static_cast<int>(h), static_cast<int>(off));
  *r = static_cast<int>(off % kKvTile);
  return true;
}

// 16 lanes per (token, kv head), 8 elements of the key row and of the value row each
// (16-byte accesses, consecutive over the lanes; with 16 elements per lane the two
// halves of a row's sectors took separate passes through L1).
// Bound by memory; a token's 144 bytes per head lie in four places of its tile, two of
// them single bytes for the scales.  Measured: 8191 tokens x 8 heads appended and read
// back, 77 MB in two launches, 22.1 us (3.5 TB/s); 64 tokens 3.5 us for the two.  Apart,
// 38 MB each: append 11.8 us with slots consecutive inside pages and 12.7 scattered, read
// 10.9 and 11.3; a plain device copy of 38 MB took 14.3.
constexpr int kRowLanes = kKvDim / 8;

// Splits a thread index into (token, kv head, lane of the row); false past the end.
__device__ __forceinline__ bool kv_row(const KvRowsParams& p, uint32_t* t, uint32_t* h, int* j) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const uint64_t row = static_cast<uint64_t>(i) / kRowLanes;
  *j = static_cast<int>(i % kRowLanes);
  *t = static_cast<uint32_t>(row >> 32 ? row / static_cast<uint32_t>(p.kv_heads)
                                       : static_cast<uint32_t>(row) / static_cast<uint32_t>(p.kv_heads));
  *h = static_cast<uint32_t>(row - static_cast<uint64_t>(*t) * p.kv_heads);
  return row < static_cast<uint64_t>(p.tokens) * p.kv_heads;
}

__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(const KvRowsParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  uint32_t t, h;
  int j;
  const bool in = kv_row(p, &t, &h, &j);
  uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
  if (in) {
    k = *reinterpret_cast<const uint4*>(p.K + t * p.ldk + h * kKvDim + 8 * j);
    v = *reinterpret_cast<const uint4*>(p.V + t * p.ldv + h * kKvDim + 8 * j);
  }
  uint8_t* tile = nullptr;
  int r = 0;
  const bool place = in && kv_place(p, t, h, &tile, &r);
  uint32_t kc, vc;
  const uint32_t ks = kv_quantise(k, p.k_inv, &kc), vs = kv_quantise(v, p.v_inv, &vc);  // pairs of lanes: no early exit
  if (!place) return;
  const int q = j / 2;
  *reinterpret_cast<uint32_t*>(tile + kv_k_code(r, q) + 4 * (j & 1)) = kc;
  *reinterpret_cast<uint32_t*>(tile + kv_v_code(r, q) + 4 * (j & 1)) = vc;
  // the even lane stores the key scale, the odd one the value scale
  tile[j & 1 ? kv_v_scale(r, q) : kv_k_scale(r, q)] = static_cast<uint8_t>(j & 1 ? vs : ks);
}

// Eight codes to bf16 times `s` (at most 6 significant bits: exact).
__device__ __forceinline__ uint4 kv_values(uint32_t codes, float s) {
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(e2m1x2_half2((codes >> (8 * e)) & 0xFFu));
    const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * s, f.y * s);
    out[e] = *reinterpret_cast<const uint32_t*>(&o);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const KvRowsParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  uint32_t t, h;
  int j;
  if (!kv_row(p, &t, &h, &j)) return;
  uint32_t kc = 0, vc = 0, scales = 0;
  uint8_t* tile;
  int r;
  if (kv_place(p, t, h, &tile, &r)) {
    const int q = j / 2;
    kc = *reinterpret_cast<const uint32_t*>(tile + kv_k_code(r, q) + 4 * (j & 1));
    vc = *reinterpret_cast<const uint32_t*>(tile + kv_v_code(r, q) + 4 * (j & 1));
    scales = tile[kv_k_scale(r, q)] | static_cast<uint32_t>(tile[kv_v_scale(r, q)]) << 8;
  }
  const float2 s = __half22float2(e4m3x2_half2(scales));
  *reinterpret_cast<uint4*>(p.K + t * p.ldk + h * kKvDim + 8 * j) = kv_values(kc, s.x * p.k_scale);
  *reinterpret_cast<uint4*>(p.V + t * p.ldv + h * kKvDim + 8 * j) = kv_values(vc, s.y * p.v_scale);
}

template <int THREADS>
cudaError_t launch_pages(const KvPagesParams& p, int grid, cudaStream_t stream) {
  static DeviceBits allowed{0};
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kv_pages_kernel<THREADS>),
                                           2 * sizeof(int32_t) * kKvMaxRequests, &allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(grid, THREADS, 2 * sizeof(int32_t) * static_cast<size_t>(p.requests), stream, attr);
  return cudaLaunchKernelEx(&cfg, kv_pages_kernel<THREADS>, p);
}

}  // namespace

cudaError_t launch_kv_pages(const KvPagesParams& p, int grid, cudaStream_t stream) {
  return p.requests <= 128 && p.tokens <= 512 ? launch_pages<128>(p, 1, stream) : launch_pages<1024>(p, grid, stream);
}

cudaError_t launch_kv_append(const KvRowsParams& p, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(p.tokens) * p.kv_heads * kRowLanes;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config((n + kRowThreads - 1) / kRowThreads, kRowThreads, 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, kv_append_kernel, p);
}

cudaError_t launch_kv_read(const KvRowsParams& p, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(p.tokens) * p.kv_heads * kRowLanes;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config((n + kRowThreads - 1) / kRowThreads, kRowThreads, 0, stream, attr);
  return cudaLaunchKernelEx(&cfg, kv_read_kernel, p);
}

}  // namespace sg
