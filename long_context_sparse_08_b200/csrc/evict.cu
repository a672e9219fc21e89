// Page eviction by accumulated attention weight (attn_mass.cu): which pages of a request's
// cache stay when it may keep `budget` of them.
//
// 【论文解读】DeepSeek-V4, 二、基础设施 (六) 推理框架: finished entries live in pages through a page
// table. A page's score is the largest accumulated weight of its entries (a maximum: exact,
// and a page is worth as much as its most attended entry). The first `keep_first` and the
// last `keep_last` pages stay; the best scored others fill the budget, the lower page first
// among equals.
//
//   k_evict_keys    (pages of several entries) an order-preserving 32-bit key per page, 0 for
//                   a page without entries, over the whole device;
//   k_evict_select  a CTA per request: the keys in shared memory, the budget-th largest by
//                   radix passes of 11, 11 and 10 bits (a pass that leaves nothing to decide is
//                   the last), one scan per 8192 pages to place them, and the lists;
//   k_evict_entries (long lists of entries) writes those over the whole device.
// 4 bytes are read per entry and a few per page, so latencies bound it. One CTA with the keys at
// hand beat a cluster of eight per request (18 to 40 us: seven cluster barriers and sums
// through distributed shared memory) and a CTA that read the keys from L2 in every pass (26 us).
// Measured, calls one after another: 16 requests of 8192 one-entry pages 12.6 to 13.6 us, 4 of 8192
// pages of 32 entries (lists of 64000 entries written) 17.6 us, one of 600 pages 6.8 us (replayed
// from a graph 12.7, 17.6 and 5.2 us).
#include "common.cuh"
#include "host_util.cuh"
#include "internal.h"

namespace csa {

namespace {

constexpr int kThreads = 1024;
constexpr int kPer = 8;                      // pages of a lane in a round
constexpr int kRound = kThreads * kPer;
constexpr int kSmemKeys = 5 * kRound;        // 160 KB; a longer table leaves its keys in L2
constexpr int kBins = 2048;
constexpr uint32_t kAlways = 0xffffffffu;

// entries finished by the tokens up to pos, and the pages that hold them
__device__ __forceinline__ int used_entries(const EvictArgs& a, int b) {
  const int64_t pos = a.pos[b];
  if (pos < 0) return 0;
  const int64_t n = pos < 0x7fffffff ? (int64_t)((uint32_t)(pos + 1) / (uint32_t)a.m) : (pos + 1) / a.m;
  const int64_t cap = (int64_t)a.page_rows * a.max_pages;
  return (int)(n < cap ? n : cap);
}
__device__ __forceinline__ int pages_of(const EvictArgs& a, int entries) {
  return (int)((uint32_t)entries / (uint32_t)a.page_rows) + ((uint32_t)entries % (uint32_t)a.page_rows != 0);
}

// order-preserving key of a weight, never 0 or ~0; a NaN is the lowest
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 1u : float_key(w); }

// `lanes` neighbouring lanes (a power of two) per page; kVec: four entries a load
template <bool kVec>
__global__ void __launch_bounds__(256) k_evict_keys(EvictArgs a, uint32_t* keys, int lanes) {
  const int b = blockIdx.y;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t p64 = i / lanes;
  const int sub = (int)(i % lanes);
  pdl_wait();
  pdl_trigger();
  const int n = used_entries(a, b);
  const int page = p64 < a.max_pages ? (int)p64 : a.max_pages;  // whole warps stay for the exchange
  uint32_t key = 0;
  if (page < a.max_pages) {
    const int64_t e0 = (int64_t)page * a.page_rows;
    const int rows = (int)(n - e0 < a.page_rows ? n - e0 : a.page_rows);  // <= 0: none
    const float* w = a.acc + (size_t)b * a.max_pages * a.page_rows + e0;
    if (kVec) {
      for (int r = 4 * sub; r < rows; r += 4 * lanes) {
        const float4 v = *reinterpret_cast<const float4*>(w + r);
        key = max(key, weight_key(v.x));
        if (r + 1 < rows) key = max(key, weight_key(v.y));
        if (r + 2 < rows) key = max(key, weight_key(v.z));
        if (r + 3 < rows) key = max(key, weight_key(v.w));
      }
    } else {
      for (int r = sub; r < rows; r += lanes) key = max(key, weight_key(w[r]));
    }
  }
  for (int o = 1; o < lanes; o <<= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  if (sub == 0 && page < a.max_pages) keys[(size_t)b * a.max_pages + page] = key;
}

// Exclusive scan over the block; *total: the sum. The caller separates two uses of `red` by a
// barrier (there is one inside, before the sums are read).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* red, uint32_t* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) red[wid] = s;
  __syncthreads();
  uint32_t w = red[lane];  // every warp scans the 32 sums for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, w, (wid + 31) & 31);
  return s - v + (wid > 0 ? before : 0);
}

// Entries [first, end) of a list: those of the kept pages page_at(0), page_at(1), .. (-1: none),
// below n. `first` and the list are aligned to four entries.
template <class PageAt>
__device__ __forceinline__ void write_entries(int32_t* out, uint32_t end, uint32_t pr, int n,
                                              uint32_t thread, uint32_t threads, PageAt page_at,
                                              uint32_t first = 0) {
  const bool pow2 = (pr & (pr - 1)) == 0;
  const int log2 = 31 - __clz(pr);
  auto div = [&](uint32_t i) { return pow2 ? i >> log2 : i / pr; };
  if (pr % 4 == 0) {  // four entries of a page a thread (the list is then 16-byte aligned)
#pragma unroll 1
    for (uint32_t i = first + 4 * thread; i < end; i += 4 * threads) {
      const uint32_t q = div(i);
      const int page = page_at(q), e = page * (int)pr + (int)(i - q * pr);
      int4 v = make_int4(e, e + 1, e + 2, e + 3);
      if (page < 0) v = make_int4(-1, -1, -1, -1);
      else if (e + 3 >= n) v = make_int4(e < n ? e : -1, e + 1 < n ? e + 1 : -1, e + 2 < n ? e + 2 : -1, -1);
      *reinterpret_cast<int4*>(out + i) = v;
    }
  } else {
#pragma unroll 1
    for (uint32_t i = first + thread; i < end; i += threads) {
      const uint32_t q = div(i);
      const int page = page_at(q), e = page * (int)pr + (int)(i - q * pr);
      out[i] = page >= 0 && e < n ? e : -1;
    }
  }
}

// kKeys: the keys come from k_evict_keys (in `ws`), else from acc (pages of one entry). kSmem:
// they fit shared memory, else `ws` holds them throughout.
template <bool kKeys, bool kSmem>
__global__ void __launch_bounds__(kThreads, 1) k_evict_select(EvictArgs a, uint32_t* ws) {
  extern __shared__ uint32_t smem_keys[];
  __shared__ uint32_t hist[kBins];
  // block_scan's sums: two arrays in turn, and one of the first scan's own: a request within its
  // budget goes from that scan straight to the placement's, with no barrier between
  __shared__ uint32_t red[3][32];
  __shared__ uint2 votes[kThreads / 32][kPer];  // of a round: kept, present
  __shared__ int pick[3], s_last;  // digit, keys above it, keys at it
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, pr = a.page_rows;
  for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
  if (!kKeys) pdl_wait();  // (with keys, the kernel that made them has waited)
  const int n = used_entries(a, b), used = pages_of(a, n);
  uint32_t* wk = ws + (size_t)b * a.max_pages;
  uint32_t* keys = kSmem ? smem_keys : wk;
  const int32_t* table = a.page_table + (size_t)b * a.max_pages;
  const float* acc = a.acc + (size_t)b * a.max_pages * pr;
  if (kKeys) pdl_wait();
  pdl_trigger();

  // ---- keys: pages that are mapped, those always kept above all; the table goes over as it is
  //      (evicted pages are marked below) ----
  int32_t* nt = a.new_table + (size_t)b * a.max_pages;
  int mine = 0;
  // (unrolled by two here and rolled below: every line of code is fetched cold, and eight-fold
  // unrolling took 1.2 us more)
#pragma unroll 2
  for (int k = tid; k < used; k += kThreads) {
    uint32_t key = kKeys ? wk[k] : weight_key(acc[k]);
    const int32_t page = table[k];
    nt[k] = page;
    if (page < 0) key = 0;
    else if (k < a.keep_first || k >= used - a.keep_last) key = kAlways;
    keys[k] = key;
    mine += key != 0;
  }
  uint32_t total;
  block_scan((uint32_t)mine, red[2], &total);  // (its barrier also publishes keys and bins)
  const int present = (int)total;

  // ---- which stay: those with key >> shift >= least, the budget-th largest key or its decided
  //      high bits ----
  uint32_t least = 0;
  int shift = 0;
  if (present > a.budget) {
    int want = a.budget, top = 32;  // want: how many of the keys with the digits so far stay
    uint32_t tau = 0;
    bool decided = false;
    for (int pass = 0; pass < 3 && !decided; ++pass) {
      const int bits = pass < 2 ? 11 : 10;
      shift = top - bits;
#pragma unroll 4
      for (int k = tid; k - lane < used; k += kThreads) {
        const uint32_t key = k < used ? keys[k] : 0u;
        const bool in = key != 0 && (pass == 0 || (key >> top) == (tau >> top));
        if (!__any_sync(0xffffffffu, in)) continue;
        const uint32_t digit = in ? (key >> shift) & ((1u << bits) - 1u) : kBins;
        // equal weights: one addition for the warp (32 to one bin would go one after another)
        int same;
        __match_all_sync(0xffffffffu, digit, &same);
        if (same) {
          if (lane == 0) atomicAdd(&hist[digit], 32u);
        } else if (in) {
          atomicAdd(&hist[digit], 1u);
        }
      }
      __syncthreads();
      // thread t: bins 2047 - 2 t and 2046 - 2 t, the highest first
      const uint32_t c0 = hist[kBins - 1 - 2 * tid], c1 = hist[kBins - 2 - 2 * tid];
      hist[kBins - 1 - 2 * tid] = 0;
      hist[kBins - 2 - 2 * tid] = 0;
      const int above = (int)block_scan(c0 + c1, red[(pass + 1) & 1], &total);
      if (above < want && above + (int)(c0 + c1) >= want) {
        const bool second = above + (int)c0 < want;
        pick[0] = kBins - 1 - 2 * tid - (second ? 1 : 0);
        pick[1] = above + (second ? (int)c0 : 0);
        pick[2] = (int)(second ? c1 : c0);
      }
      __syncthreads();
      tau |= (uint32_t)pick[0] << shift;
      want -= pick[1];
      top = shift;
      decided = want == pick[2];  // all of the digit's keys stay
    }
    least = tau >> shift;
    if (!decided) {
      // more keys equal tau than stay: the first `want` in page order are raised above all
      ++least;
      int before = 0;
      for (int k0 = 0, round = 0; k0 < used; k0 += kThreads, ++round) {
        const bool tie = k0 + tid < used && keys[k0 + tid] == tau;
        const uint32_t ties = __ballot_sync(0xffffffffu, tie);
        uint32_t at = block_scan(lane == 0 ? (uint32_t)__popc(ties) : 0u, red[round & 1], &total);
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(ties & ((1u << lane) - 1u));
        if (tie && before + (int)at < want) keys[k0 + tid] = kAlways;
        before += (int)total;
      }
      __syncthreads();
    }
  }

  // ---- placement in page order: a warp has up to 256 consecutive pages of a round, 32 at a
  //      time; ballots count the kept and the present pages before each ----
  const int64_t n_out = (int64_t)a.budget * pr;
  int32_t* out_entries = a.entries != nullptr ? a.entries + (size_t)b * n_out : nullptr;
  int32_t* out_kept = a.kept + (size_t)b * a.budget;
  int32_t* out_gone = a.evicted + (size_t)b * a.max_pages;
  const uint32_t below = (1u << lane) - 1u;
  int n_kept = 0, seen = 0;
  bool last_stays = false;
  for (int k0 = 0, round = 0; k0 < used; k0 += kRound, ++round) {
    const int steps = min(kPer, (used - k0 + kThreads - 1) / kThreads);
    const int first = k0 + (tid >> 5) * (32 * steps) + lane;
    uint2* mine_of = votes[tid >> 5];
    uint32_t mine2 = 0;  // kept and present pages of the warp, 16 bits each
#pragma unroll 2
    for (int i = 0; i < steps; ++i) {
      const uint32_t key = first + 32 * i < used ? keys[first + 32 * i] : 0u;
      const uint32_t here = __ballot_sync(0xffffffffu, key != 0);
      const uint32_t keep = __ballot_sync(0xffffffffu, key != 0 && (key >> shift) >= least);
      if (lane == 0) mine_of[i] = make_uint2(keep, here);
      mine2 += (uint32_t)__popc(keep) + ((uint32_t)__popc(here) << 16);
    }
    uint32_t all2;  // lane 0 speaks for its warp
    uint32_t pos = block_scan(lane == 0 ? mine2 : 0u, red[round & 1], &all2);
    pos = __shfl_sync(0xffffffffu, pos, 0);
    int kept0 = n_kept + (int)(pos & 0xffff), here0 = seen + (int)(pos >> 16);
#pragma unroll 2
    for (int i = 0; i < steps; ++i) {
      const int page = first + 32 * i;
      const uint2 v = mine_of[i];
      const bool here = (v.y >> lane) & 1u, keep = (v.x >> lane) & 1u;
      const int kept = kept0 + __popc(v.x & below);
      if (keep) {
        out_kept[kept] = page;
        if (kSmem) keys[kept] = (uint32_t)page;  // every key up to here has been read
      } else if (here) {
        nt[page] = kEvicted;
        out_gone[here0 + __popc(v.y & below) - kept] = page;
      }
      if (page == used - 1) last_stays = keep;
      kept0 += __popc(v.x);
      here0 += __popc(v.y);
    }
    n_kept += (int)(all2 & 0xffff);
    seen += (int)(all2 >> 16);
  }
  const int n_gone = present - n_kept;
  for (int k = used + tid; k < a.max_pages; k += kThreads) nt[k] = table[k];
  for (int i = n_kept + tid; i < a.budget; i += kThreads) out_kept[i] = -1;
  for (int i = n_gone + tid; i < a.max_pages; i += kThreads) out_gone[i] = -1;
  if (tid == 0) {
    a.counts[3 * b] = n_kept;
    a.counts[3 * b + 2] = n_gone;
  }
  // whoever had the last used page knows whether it, perhaps open, stays
  const int open = n % pr;
  if (last_stays) a.counts[3 * b + 1] = n_kept * pr - (open != 0 ? pr - open : 0);
  if (tid == 0) s_last = 0;
  __syncthreads();
  if (last_stays) s_last = 1;
  __syncthreads();
  if (tid == 0 && !s_last) a.counts[3 * b + 1] = n_kept * pr;
  if (out_entries != nullptr) {
    __syncthreads();  // the kept pages, written by this CTA
    write_entries(out_entries, (uint32_t)n_out, (uint32_t)pr, n, (uint32_t)tid, kThreads,
                  [&](uint32_t q) { return (int)q < n_kept ? (kSmem ? (int)keys[q] : out_kept[q]) : -1; });
  }
}

// The same for long lists: one SM stores 64 bytes a cycle, so that 4 requests' lists of 64000
// entries took 4.6 us of 19.7 in the CTAs above, and 18.0 in all with this launch. A list of 16384
// takes one SM as long as the launch does.
constexpr int64_t kLongList = 16384;
constexpr int kListBlock = 4096;  // entries of a block

__global__ void __launch_bounds__(256) k_evict_entries(EvictArgs a) {
  const int b = blockIdx.y;
  const int64_t n_out = (int64_t)a.budget * a.page_rows;
  const int n = used_entries(a, b);
  const int32_t* kept = a.kept + (size_t)b * a.budget;
  pdl_wait();
  const int n_kept = a.counts[3 * b];
  const int64_t first = (int64_t)blockIdx.x * kListBlock;
  write_entries(a.entries + (size_t)b * n_out,
                (uint32_t)(n_out - first < kListBlock ? n_out : first + kListBlock), (uint32_t)a.page_rows, n, (uint32_t)threadIdx.x, 256,
                [&](uint32_t q) { return (int)q < n_kept ? kept[q] : -1; }, (uint32_t)first);
}

}  // namespace

size_t evict_workspace_bytes(int B, int max_pages) {
  return ((size_t)B * max_pages * sizeof(uint32_t) + 255) / 256 * 256;
}

cudaError_t launch_evict(const EvictArgs& a, void* ws, cudaStream_t st) {
  uint32_t* keys = static_cast<uint32_t*>(ws);
  const bool own = a.page_rows > 1, fits = a.max_pages <= kSmemKeys;
  cudaError_t e;
  if (own) {
    const bool vec = a.page_rows % 4 == 0;
    const int units = vec ? a.page_rows / 4 : a.page_rows;
    int lanes = 1;
    while (lanes < 32 && 2 * lanes <= units) lanes *= 2;
    const int64_t threads = (int64_t)a.max_pages * lanes;
    const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)a.B);
    e = launch(true, vec ? k_evict_keys<true> : k_evict_keys<false>, grid, dim3(256), 0, st, a, keys,
               lanes);
    if (e != cudaSuccess) return e;
  }
  auto kern = own ? (fits ? k_evict_select<true, true> : k_evict_select<true, false>)
                  : (fits ? k_evict_select<false, true> : k_evict_select<false, false>);
  const size_t smem = fits ? (size_t)a.max_pages * sizeof(uint32_t) : 0;
  static std::atomic<uint64_t> allowed[4];
  e = allow_smem(kern, kSmemKeys * (int)sizeof(uint32_t), allowed[2 * own + fits]);
  if (e != cudaSuccess) return e;
  const int64_t n_out = a.entries != nullptr ? (int64_t)a.budget * a.page_rows : 0;
  EvictArgs sel = a;
  if (n_out > kLongList) sel.entries = nullptr;
  e = launch(true, kern, dim3((unsigned)a.B), dim3(kThreads), smem, st, sel, keys);
  if (e != cudaSuccess || n_out <= kLongList) return e;
  const dim3 grid((unsigned)((n_out + kListBlock - 1) / kListBlock), (unsigned)a.B);
  return launch(true, k_evict_entries, grid, dim3(256), 0, st, a);
}

}  // namespace csa
