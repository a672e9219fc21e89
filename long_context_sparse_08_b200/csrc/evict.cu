// Page eviction by accumulated attention weight (attn_mass.cu): which pages of a request's
// cache stay when it may keep `budget` of them.
//
// 【论文解读】DeepSeek-V4, 二、基础设施 (六) 推理框架: finished entries live in pages through a page
// table. A page's score is the largest accumulated weight of its entries (a maximum: exact,
// and a page is worth as much as its most attended entry). The first `keep_first` and the
// last `keep_last` pages stay; the best scored others fill the budget, the lower page first
// among equals.
//
//   k_evict_keys    an order-preserving 32-bit key per page (0: no page; ~0: always kept)
//   k_evict_select  a CTA per request: the budget-th largest key by four 8-bit radix passes
//                   over keys held in registers, then one scan places kept and evicted pages
//   k_evict_entries the kept pages' entries as an index list
// All of it is a few passes over 4 bytes per entry and page: the launches bound it.
#include "common.cuh"
#include "internal.h"

namespace csa {

namespace {

constexpr int kSelThreads = 1024;
constexpr uint32_t kAlways = 0xffffffffu;

// entries finished by the tokens up to pos, and the pages that hold them
__device__ __forceinline__ int used_entries(const EvictArgs& a, int b) {
  const int64_t pos = a.pos[b];
  const int64_t n = pos < 0 ? 0 : (pos + 1) / a.m;
  const int64_t cap = (int64_t)a.page_rows * a.max_pages;
  return (int)(n < cap ? n : cap);
}
__device__ __forceinline__ int used_pages(const EvictArgs& a, int entries) {
  return entries / a.page_rows + (entries % a.page_rows != 0 ? 1 : 0);
}

// order-preserving key of a weight, never 0 or ~0; a NaN is the lowest
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 1u : float_key(w); }

// kWarp: a warp per page (its lanes over the entries), else a thread per page
template <bool kWarp>
__global__ void __launch_bounds__(256) k_evict_keys(EvictArgs a, uint32_t* keys) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if ((kWarp ? i >> 5 : i) >= a.max_pages) return;
  const int page = (int)(kWarp ? i >> 5 : i);
  const int n = used_entries(a, b), used = used_pages(a, n);
  uint32_t key = 0;
  if (page < used && a.page_table[(size_t)b * a.max_pages + page] >= 0) {
    if (page < a.keep_first || page >= used - a.keep_last) {
      key = kAlways;
    } else {
      const float* w = a.acc + ((size_t)b * a.max_pages + page) * (size_t)a.page_rows;
      const int rows = min(a.page_rows, n - page * a.page_rows);
      for (int r = kWarp ? lane : 0; r < rows; r += kWarp ? 32 : 1) {
        const uint32_t k = weight_key(w[r]);
        key = k > key ? k : key;
      }
      if (kWarp) key = __reduce_max_sync(0xffffffffu, key);
    }
  }
  if (!kWarp || lane == 0) keys[(size_t)b * a.max_pages + page] = key;
}

// Exclusive scan over the block of two counts packed in one word; *total: the sums.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* red, uint64_t* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();
  if (lane == 31) red[wid] = s;
  __syncthreads();
  if (wid == 0) {
    uint64_t w = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    red[lane] = w;
  }
  __syncthreads();
  *total = red[31];
  return s - v + (wid > 0 ? red[wid - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads) k_evict_select(EvictArgs a, const uint32_t* keys_all) {
  __shared__ int hist[256];
  __shared__ uint64_t red[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_want;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int n = used_entries(a, b), used = used_pages(a, n);
  pdl_wait();
  pdl_trigger();
  const uint32_t* keys = keys_all + (size_t)b * a.max_pages;

  // present pages
  int mine = 0;
  for (int k = tid; k < used; k += kSelThreads) mine += keys[k] != 0;
  uint64_t present = 0;
  block_scan((uint64_t)mine, red, &present);

  // tau: the budget-th largest key; `want` of the pages equal to it stay
  uint32_t tau = 0;
  int want = 0;
  if ((int64_t)present > a.budget) {
    if (tid == 0) {
      s_prefix = 0;
      s_want = a.budget;
    }
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : ~0u << (shift + 8);
      for (int k = tid; k < used; k += kSelThreads) {
        const uint32_t key = keys[k];
        if (key != 0 && (key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
      }
      __syncthreads();
      // the digit where the count from above reaches s_want
      if (tid < 32) {
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = hist[255 - (8 * tid + i)];
          sum += c[i];
        }
        int above = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, above, o);
          if (tid >= o) above += u;
        }
        above -= sum;
        const int w = s_want;
        __syncwarp();
        if (above < w && above + sum >= w) {
          int run = above;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (run < w && run + c[i] >= w) {
              s_prefix = prefix | ((uint32_t)(255 - (8 * tid + i)) << shift);
              s_want = w - run;
            }
            run += c[i];
          }
        }
      }
      __syncthreads();
    }
    tau = s_prefix;
    want = s_want;
  }

  // in page order: ties before a page, then kept and evicted pages
  int ties = 0, kept = 0, gone = 0;
  for (int k0 = 0; k0 < a.max_pages; k0 += kSelThreads) {
    const int k = k0 + tid;
    const size_t at = (size_t)b * a.max_pages + k;
    const uint32_t key = k < used ? keys[k] : 0u;
    const bool tie = key != 0 && tau != 0 && key == tau;
    uint64_t total;
    const int before = ties + (int)block_scan(tie ? 1 : 0, red, &total);
    ties += (int)total;
    const bool keep = key != 0 && (key > tau || (tie && before < want));
    const bool out = key != 0 && !keep;
    const uint64_t pos = block_scan((keep ? 1ull : 0ull) | (out ? 1ull << 32 : 0ull), red, &total);
    if (k < a.max_pages) a.new_table[at] = out ? kEvicted : a.page_table[at];
    if (keep) a.kept[(size_t)b * a.budget + kept + (int)(uint32_t)pos] = k;
    if (out) a.evicted[(size_t)b * a.max_pages + gone + (int)(pos >> 32)] = k;
    kept += (int)(uint32_t)total;
    gone += (int)(total >> 32);
  }
  for (int i = kept + tid; i < a.budget; i += kSelThreads) a.kept[(size_t)b * a.budget + i] = -1;
  for (int i = gone + tid; i < a.max_pages; i += kSelThreads)
    a.evicted[(size_t)b * a.max_pages + i] = -1;
  if (tid == 0) {
    a.counts[3 * b] = kept;
    a.counts[3 * b + 2] = gone;
    // the last page may be open: it is the last kept one if it stays
    const int open = n % a.page_rows;
    const bool last = open != 0 && keys[used - 1] != 0 &&
                      (keys[used - 1] > tau || (keys[used - 1] == tau && ties <= want));
    a.counts[3 * b + 1] = kept * a.page_rows - (last ? a.page_rows - open : 0);
  }
}

// entries of the kept pages in order; -1 behind them
__global__ void __launch_bounds__(256) k_evict_entries(EvictArgs a) {
  const int b = blockIdx.y;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n_out = (int64_t)a.budget * a.page_rows;
  const int n = used_entries(a, b);
  pdl_wait();
  if (i >= n_out) return;
  const int page = a.kept[(size_t)b * a.budget + i / a.page_rows];
  const int64_t e = page < 0 ? -1 : (int64_t)page * a.page_rows + i % a.page_rows;
  a.entries[(size_t)b * n_out + i] = e < n ? (int32_t)e : -1;
}

}  // namespace

size_t evict_workspace_bytes(int B, int max_pages) {
  return ((size_t)B * max_pages * sizeof(uint32_t) + 255) / 256 * 256;
}

cudaError_t launch_evict(const EvictArgs& a, void* ws, cudaStream_t st) {
  uint32_t* keys = static_cast<uint32_t*>(ws);
  const bool warp = a.page_rows >= 32;
  const int64_t threads = (int64_t)a.max_pages * (warp ? 32 : 1);
  const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)a.B);
  cudaError_t e = warp ? launch(false, k_evict_keys<true>, grid, dim3(256), 0, st, a, keys)
                       : launch(false, k_evict_keys<false>, grid, dim3(256), 0, st, a, keys);
  if (e != cudaSuccess) return e;
  e = launch(true, k_evict_select, dim3((unsigned)a.B), dim3(kSelThreads), 0, st, a,
             (const uint32_t*)keys);
  if (e != cudaSuccess || a.entries == nullptr) return e;
  const int64_t n_out = (int64_t)a.budget * a.page_rows;
  return launch(true, k_evict_entries, dim3((unsigned)((n_out + 255) / 256), (unsigned)a.B),
                dim3(256), 0, st, a);
}

}  // namespace csa
