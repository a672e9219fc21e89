// Accumulated attention weight per cache entry:
//   acc[b, e] = decay * acc[b, e] + sum over the queries t and heads h of request b of
//               p[t, h, e],   p = e^z / (sum over the query's rows of e^z + e^sink_h),
// z and the rows (selected or visible entries, then the window) as in the attention of
// 【论文解读】DeepSeek-V4 一(三)1(3) / 2(2), 3(1)-(4). What the cache is asked for is thereby
// known per entry, and the pages with the least of it can be given back (evict.cu).
//
// The sums are meant to be compared over thousands of steps, so the weights are formed to
// fp32: q_hat is split into two 16-bit operands, hi + lo (f16 over 4-bit rows: 22 bits; bf16
// over bf16 rows: 16 bits), stacked as the 128 rows of one M = 128 product, so that both parts
// cost one read of the KV tile:
//   [hi; lo][128 x 512] . K^T[512 x 64 rows] -> TMEM, z = (hi + lo) * scale * log2(e)
// Head 16 w + i has hi in row 32 w + i and lo in row 32 w + 16 + i, so that both lie in the
// TMEM lanes of one warp and one exchange adds them.
//   q_tiles.cu      prepares the [hi; lo] tiles;
//   k_mass_logits   (a CTA per (query, 64 heads, split)) writes z as fp32 and, per split and
//                   head, the running maximum and sum;
//   k_mass_dense    adds 2^(z - L) over queries and heads for one entry per thread;
//   k_mass_sparse   does so for one list slot per thread and adds the result to a 64-bit
//                   fixed-point array (2^-40), whose order of additions changes nothing;
//   k_mass_finish   acc = decay * acc + that array.
// The KV tile is single-buffered, but each 64-value atom is given back as soon as its
// products are done, so the gather warps refill atom 0 while atoms 1-7 are multiplied.
#include <cmath>

#include "common.cuh"
#include "host_util.cuh"
#include "internal.h"
#include "kv_rows.cuh"
#include "tc.cuh"

namespace csa {

namespace {

using namespace tc;
using namespace rows;

constexpr int kThreads = (6 + kGatherWarps) * 32;
constexpr int kMaxSplit = 32;
constexpr int kQRows = 128;                       // hi and lo of 64 heads
constexpr int kOffKV = 0;
constexpr int kOffQ = kAtoms * kAtomBytes;        // [atom][row][128 B]
constexpr int kQAtom = kQRows * 128;
constexpr int kOffEnd = kOffQ + kAtoms * kQAtom;
constexpr uint32_t kTmemCols = 128;               // two S tiles of 64 columns
constexpr float kFixed = 1099511627776.f;         // 2^40
constexpr unsigned long long kNotFinite = 1ull << 63;

// 221 ring free, 222 ring full / 223 atom free, 224 q_hat / KV full / S free, 225 S full;
// 226 = 221 + 5: a page id outside the pool
enum { kErrRing = 221, kErrGather = 222, kErrMma = 224, kErrRead = 225 };

struct Smem {
  AddrRing ring;
  uint64_t kv_full[kAtoms], kv_free[kAtoms], s_full[2], s_free[2], q_full, done;
  uint32_t tmem_slot;
};

struct Params {
  MqaArgs a;
  int G, nsplit;
  int64_t z_rows;            // rows of a head's z (a multiple of 64)
  float* z;                  // [stream][64][z_rows]
  float* part;               // [stream][split][m 64 | l 64]
  unsigned long long* fixed; // [B][n_cap] (sparse)
  float* acc;
  const uint8_t* tiles;      // q_hat tiles, 128 KB per stream
  float scale2, decay;
};

template <int kFmt>
__global__ void __launch_bounds__(kThreads, 1) k_mass_logits(const __grid_constant__ Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_align1024(smem_raw);
  Smem& S = *reinterpret_cast<Smem*>(base + kOffEnd);
  const MqaArgs& a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == 4) {
    if (lane == 0) {
      for (int i = 0; i < kRing; ++i) {
        mbar_init(&S.ring.full[i], 1);
        mbar_init(&S.ring.free[i], kGatherWarps + 4);
      }
      for (int i = 0; i < kAtoms; ++i) {
        mbar_init(&S.kv_full[i], i == kAtoms - 1 ? 2 : 1);
        mbar_init(&S.kv_free[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&S.s_full[i], 1);
        mbar_init(&S.s_free[i], 4);
      }
      mbar_init(&S.q_full, 1);
      mbar_init(&S.done, 1);
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(&S.tmem_slot, kTmemCols);
  }
  Item x;
  x.set(a, blockIdx.x, P.G, P.nsplit, item_pos(a, blockIdx.x, P.G, P.nsplit));
  const int n = x.c1 - x.c0;
  RowBatch rows0;
  if (warp == 5) rows0.lookup(a, x, x.c0);
  if (P.fixed != nullptr) {  // the sparse sums start at zero
    const size_t n = (size_t)a.B * a.n_cap, step = (size_t)gridDim.x * kThreads;
    for (size_t i = (size_t)blockIdx.x * kThreads + tid; i < n; i += step) P.fixed[i] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = S.tmem_slot;

  if (warp >= 6) {
    gather_loop<kFmt, 1, kAtoms, kAtoms>(base + kOffKV, warp - 6, S.ring, S.kv_full, S.kv_free, kErrGather);
  } else if (warp == 5) {
    uint32_t it = 0;
    if (resolve_rows<kFmt>(rows0, a, x, it, S.ring, kErrRing)) resolve_end(it, S.ring, kErrRing);
  } else if (warp == 4) {
    const uint32_t idS = idesc_f16(kFmt == kFp4 ? 0 : 1, kQRows, kRows);
    const uint64_t dq = smem_desc(smem_u32(base + kOffQ), 16, 1024, kLayoutSw128);
    const uint64_t dk = smem_desc(smem_u32(base + kOffKV), 16, 1024, kLayoutSw128);
    bool ok = n > 0;
    if (ok) {
      pdl_wait();  // the q_hat tiles of the launch before
      if (elect_one()) {
        mbar_arrive_expect_tx(&S.q_full, kAtoms * kQAtom);
        bulk_load(base + kOffQ, P.tiles + (size_t)x.stream * (kAtoms * kQAtom), kAtoms * kQAtom, &S.q_full);
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, mbar_wait(&S.q_full, 0, kErrMma));
    }
    for (int it = 0; it < n && ok; ++it) {
      const int slot = it & 1;
      ok = __all_sync(0xffffffffu,
                      mbar_wait(&S.s_free[slot], ((uint32_t)(it >> 1) & 1) ^ 1, kErrMma));
      if (!ok) break;
#pragma unroll
      for (int atom = 0; atom < kAtoms; ++atom) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&S.kv_full[atom], (uint32_t)it & 1, kErrMma));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kq = 0; kq < 4; ++kq)
            mma_f16(tmem + 64 * slot, dq + ((atom * kQAtom + kq * 32) >> 4),
                    dk + ((atom * kAtomBytes + kq * 32) >> 4), idS, (atom | kq) != 0 ? 1u : 0u);
          mma_commit(&S.kv_free[atom]);
        }
      }
      if (!ok) break;
      if (elect_one()) mma_commit(&S.s_full[slot]);
      __syncwarp();
    }
    __syncwarp();
    if (elect_one()) mma_commit(&S.done);  // fires when nothing issued here is in flight
    __syncwarp();
    mbar_wait(&S.done, 0, kErrMma);
  } else {
    // ---- logits: lane i and i + 16 hold hi and lo of head 16 w + i % 16; after the exchange
    //      lane i has the head's rows 0-31 of the chunk and lane i + 16 its rows 32-63 ----
    const uint32_t lane_base = tmem + ((uint32_t)(32 * warp) << 16);
    const int hi_half = lane >> 4, head = 16 * warp + (lane & 15);
    float* zrow = P.z + ((size_t)x.stream * kHg + head) * P.z_rows + 32 * hi_half;
    float m = -INFINITY, sum = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int it = 0; it < n && ok; ++it) {
      const int j = x.c0 + it, slot = it & 1, rs = it % kRing;
      ok = __all_sync(0xffffffffu, mbar_wait(&S.s_full[slot], (uint32_t)(it >> 1) & 1, kErrRead));
      if (!ok) break;
      tc_fence_after();
      uint32_t v[64];
      tmem_ld_32x32b_x64(lane_base + 64 * slot, v);
      tmem_ld_wait();
      const uint32_t live = S.ring.mask[rs][hi_half];
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.ring.free[rs]);
        mbar_arrive(&S.s_free[slot]);
      }
      float z[32], cm = -INFINITY;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float give = __uint_as_float(hi_half ? v[c] : v[32 + c]);
        const float keep = __uint_as_float(hi_half ? v[32 + c] : v[c]);
        const float got = __shfl_xor_sync(0xffffffffu, give, 16);
        z[c] = (live >> c) & 1u ? (keep + got) * P.scale2 : -INFINITY;
        cm = fmaxf(cm, z[c]);
      }
      if (j < x.l.nc) {
        float4* dst = reinterpret_cast<float4*>(zrow + (size_t)kRows * j);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          dst[c] = make_float4(z[4 * c], z[4 * c + 1], z[4 * c + 2], z[4 * c + 3]);
      }
      const float mn = fmaxf(m, cm);
      if (mn != -INFINITY) {
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 32; ++c) s4[c & 3] += exp2f(z[c] - mn);
        sum = sum * exp2f(m - mn) + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
        m = mn;
      }
    }
    // the two halves of the head
    const float om = __shfl_xor_sync(0xffffffffu, m, 16), os = __shfl_xor_sync(0xffffffffu, sum, 16);
    const float M = fmaxf(m, om);
    float t = 0.f;
    if (M != -INFINITY) t = sum * exp2f(m - M) + os * exp2f(om - M);
    if (hi_half == 0) {
      float* pp = P.part + ((size_t)x.stream * P.nsplit + x.split) * (2 * kHg);
      pp[head] = M;
      pp[kHg + head] = t;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// log2 of the softmax denominator of head h (of all H) of query bt
__device__ __forceinline__ float denominator(const Params& P, int bt, int h) {
  const int g = h / kHg, hh = h % kHg;
  const float* pp = P.part + (size_t)(bt * P.G + g) * P.nsplit * (2 * kHg) + hh;
  const float zs = P.a.sink ? P.a.sink[h] * 1.44269504088896341f : -INFINITY;
  float M = zs;
  for (int s = 0; s < P.nsplit; ++s) M = fmaxf(M, pp[s * 2 * kHg]);
  if (M == -INFINITY) return INFINITY;  // no row: every weight is 0
  float t = zs == -INFINITY ? 0.f : exp2f(zs - M);
  for (int s = 0; s < P.nsplit; ++s) {
    const float m = pp[s * 2 * kHg];
    if (m != -INFINITY) t = fmaf(pp[s * 2 * kHg + kHg], exp2f(m - M), t);
  }
  return M + log2f(t);
}

// sum over the heads of 2^(z - L) for row `row` of query bt; L in shared memory
__device__ __forceinline__ float weight_of(const Params& P, int bt, int64_t row, const float* L) {
  float s = 0.f;
  for (int g = 0; g < P.G; ++g) {
    const float* z = P.z + (size_t)(bt * P.G + g) * kHg * P.z_rows + row;
#pragma unroll 16
    for (int h = 0; h < kHg; ++h) s += exp2f(z[(size_t)h * P.z_rows] - L[g * kHg + h]);
  }
  return s;
}

constexpr int kRedThreads = 256;

__global__ void __launch_bounds__(kRedThreads) k_mass_dense(const __grid_constant__ Params P) {
  extern __shared__ float L[];  // [H]
  const int b = blockIdx.y;
  const int64_t e = (int64_t)blockIdx.x * kRedThreads + threadIdx.x;
  const bool in = e < P.a.n_cap;
  const float old = in ? P.acc[(size_t)b * P.a.n_cap + e] : 0.f;
  pdl_wait();
  float sum = 0.f;
  for (int t = 0; t < P.a.T; ++t) {
    const int bt = b * P.a.T + t;
    const int64_t n_vis = make_list(P.a, P.a.q_pos[bt]).n_vis;
    if ((int64_t)blockIdx.x * kRedThreads >= n_vis) continue;  // the same for the whole CTA
    __syncthreads();
    for (int h = threadIdx.x; h < P.a.H; h += kRedThreads) L[h] = denominator(P, bt, h);
    __syncthreads();
    if (e < n_vis) sum += weight_of(P, bt, e, L);
  }
  if (in) P.acc[(size_t)b * P.a.n_cap + e] = fmaf(P.decay, old, sum);
}

__global__ void __launch_bounds__(kRedThreads) k_mass_sparse(const __grid_constant__ Params P) {
  extern __shared__ float L[];
  const int bt = blockIdx.y, b = bt / P.a.T;
  const int j = blockIdx.x * kRedThreads + threadIdx.x;
  const int e = j < P.a.k ? P.a.idx[(size_t)bt * P.a.k + j] : -1;
  pdl_wait();
  for (int h = threadIdx.x; h < P.a.H; h += kRedThreads) L[h] = denominator(P, bt, h);
  __syncthreads();
  if (e < 0 || e >= P.a.n_cap) return;
  const float w = weight_of(P, bt, j, L);
  unsigned long long* at = P.fixed + (size_t)b * P.a.n_cap + e;
  if (w <= 16777216.f) atomicAdd(at, (unsigned long long)__float2ll_rn(w * kFixed));
  else atomicOr(at, kNotFinite);
}

__global__ void __launch_bounds__(kRedThreads) k_mass_finish(const __grid_constant__ Params P) {
  pdl_wait();
  const size_t n = (size_t)P.a.B * P.a.n_cap, i = (size_t)blockIdx.x * kRedThreads + threadIdx.x;
  if (i >= n) return;
  const unsigned long long f = P.fixed[i];
  const float add = f & kNotFinite ? __uint_as_float(0x7fc00000u)
                                   : (float)((double)f * 9.094947017729282e-13);  // 2^-40
  P.acc[i] = fmaf(P.decay, P.acc[i], add);
}

int choose_split(const MqaArgs& a) {
  const int64_t streams = (int64_t)a.B * a.T * (a.H / kHg);
  const int64_t rows = a.k > 0 ? a.k : a.n_cap;
  const int64_t chunks = (rows + kRows - 1) / kRows + ((int64_t)a.n_win + kRows - 1) / kRows;
  int64_t ns = device_sm_count() / (streams > 0 ? streams : 1);
  ns = ns < chunks ? ns : chunks;
  return (int)(ns < 1 ? 1 : (ns > kMaxSplit ? kMaxSplit : ns));
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
  int nsplit;
  int64_t z_rows;
  size_t z_bytes, part_bytes, fixed_bytes, tile_bytes, rope_bytes;
};

Plan make_plan(const MqaArgs& a) {
  Plan p;
  const size_t streams = (size_t)a.B * a.T * (a.H / kHg);
  p.nsplit = choose_split(a);
  p.z_rows = ((a.k > 0 ? a.k : a.n_cap) + kRows - 1) / kRows * kRows;
  p.z_bytes = up256(streams * kHg * (size_t)p.z_rows * sizeof(float));
  p.part_bytes = up256(streams * p.nsplit * 2 * kHg * sizeof(float));
  p.tile_bytes = q_tiles_bytes(a, true);
  p.rope_bytes = q_rope_bytes(a);
  p.fixed_bytes = a.k > 0 ? up256((size_t)a.B * a.n_cap * 8) : 0;
  return p;
}

}  // namespace

size_t attn_mass_workspace_bytes(const MqaArgs& a) {
  const Plan p = make_plan(a);
  return p.z_bytes + p.part_bytes + p.fixed_bytes + p.tile_bytes + p.rope_bytes;
}

cudaError_t launch_attn_mass(const MqaArgs& a, float decay, float* acc, void* ws,
                             cudaStream_t st) {
  const Plan pl = make_plan(a);
  char* w = static_cast<char*>(ws);
  Params P;
  P.a = a;
  P.G = a.H / kHg;
  P.nsplit = pl.nsplit;
  P.z_rows = pl.z_rows;
  P.z = reinterpret_cast<float*>(w);
  P.part = reinterpret_cast<float*>(w + pl.z_bytes);
  P.fixed = a.k > 0 ? reinterpret_cast<unsigned long long*>(w + pl.z_bytes + pl.part_bytes) : nullptr;
  P.acc = acc;
  P.scale2 = a.scale * 1.44269504088896341f;
  P.decay = decay;
  char* tiles = w + pl.z_bytes + pl.part_bytes + pl.fixed_bytes;
  P.tiles = reinterpret_cast<const uint8_t*>(tiles);
  const int64_t streams = (int64_t)a.B * a.T * P.G;
  auto kern = a.fp4 ? k_mass_logits<kFp4> : k_mass_logits<kBf16>;
  const size_t smem = 1024 + kOffEnd + sizeof(Smem);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_q_tiles(a, true, tiles, tiles + pl.tile_bytes, st);
  if (e != cudaSuccess) return e;
  e = launch(true, kern, dim3((unsigned)(streams * P.nsplit)), dim3(kThreads), smem, st, P);
  if (e != cudaSuccess) return e;
  const size_t lsm = (size_t)a.H * sizeof(float);
  if (a.k == 0)
    return launch(true, k_mass_dense,
                  dim3((unsigned)((a.n_cap + kRedThreads - 1) / kRedThreads), (unsigned)a.B),
                  dim3(kRedThreads), lsm, st, P);
  e = launch(true, k_mass_sparse,
             dim3((unsigned)((a.k + kRedThreads - 1) / kRedThreads), (unsigned)(a.B * a.T)),
             dim3(kRedThreads), lsm, st, P);
  if (e != cudaSuccess) return e;
  const size_t n = (size_t)a.B * a.n_cap;
  return launch(true, k_mass_finish, dim3((unsigned)((n + kRedThreads - 1) / kRedThreads)),
                dim3(kRedThreads), 0, st, P);
}

cudaError_t attn_mass_device_error(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, tc::g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(tc::g_device_error, &zero, sizeof(int));
}

}  // namespace csa
