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
// TMEM lanes of one warp, and two loads of 16 lanes bring a thread hi and lo of the same logit.
//   q_tiles.cu      prepares the [hi; lo] tiles;
//   k_mass_logits   (a CTA per (query, 64 heads, split)) writes z as fp32 and, per split and
//                   head, the running maximum and sum;
//   k_mass_dense    adds 2^(z - L) over queries and heads, four threads to an entry;
//   k_mass_sparse   does so for a list slot and adds the result to a 64-bit fixed-point array,
//                   whose order of additions changes nothing. An entry's sum is T * H at most (a
//                   query's rows share a weight of 1 per head), so its steps are 2^-62 of that,
//                   rounded up to a power of two: 2^-56 for a query of 64 heads, 2^-40 at the
//                   largest T * H (2^22) that a call takes;
//   k_mass_finish   acc = decay * acc + that array.
// The KV tile is single-buffered, but each pair of 64-value atoms is given back as soon as its
// products are done, so the gather warps refill the first while the others are multiplied. A
// chunk's logits leave as one bulk copy of 16 KB from a staged tile.
//
// What bounds it: the chain gather -> product -> read over the one KV buffer (the products' operands
// from shared memory, 6 KB and 48 cycles for each 16 of K, and the gather's stores are half of a
// chunk's time), then the logits, 4 bytes per (query, head, row) written and read once more (28 MB
// each way for 16 queries x 64 heads over 5350 to 8191 entries: mostly L2). Measured, calls one after
// another: that case 46.1 us, 3 queries over 600 bf16 entries 11.2 us, 4 x 4 queries x 128 heads
// with lists of 1024 26.0 us. Keeping the logits beats a second product over the rows once the maxima
// are known, which would cost another 28 us in the first case where they cost 10.
//
// Roundings: q_hat to the two parts; the tensor cores' sums of 512 products are fp32 and cut off, about
// 1e-6 of a weight at logits of 5 to 9 (the weights of a row beside larger ones come out that much
// high); exponents, maxima and sums are fp32.
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
constexpr int kOffZ = kOffQ + kAtoms * kQAtom;    // one staged tile of logits
constexpr int kTile = kHg * kRows;
constexpr int kOffEnd = kOffZ + kTile * 4;
constexpr int kPairs = kAtoms / 2;                // pairs of atoms, given back one by one
constexpr uint32_t kTmemCols = 128;               // two S tiles of 64 columns
constexpr unsigned long long kNotFinite = 1ull << 63;  // in the fixed-point array

// 221 ring free, 222 ring full / 223 atom free, 224 q_hat / KV full / S free, 225 S full;
// 226 = 221 + 5: a page id outside the pool
enum { kErrRing = 221, kErrGather = 222, kErrMma = 224, kErrRead = 225 };

struct Smem {
  AddrRing ring;
  uint64_t kv_full[kPairs], kv_free[kPairs], s_full[2], s_free[2], q_full, done;
  uint32_t tmem_slot;
};

struct Params {
  MqaArgs a;
  int G, nsplit;
  int64_t z_tiles;           // chunks of a stream's z
  float* z;                  // [stream][chunk][64 heads][64 rows], segments permuted
  float* part;               // [stream][split][m 64 | l 64]
  unsigned long long* fixed; // [B][n_cap] (sparse), in steps of `step` = 1 / fixed_one
  float fixed_one, slot_max; // slot_max: a little above H, the most that one slot can weigh
  double step;
  float* acc;
  const uint8_t* tiles;      // q_hat tiles, 128 KB per stream
  float scale2, decay;
};

__device__ __forceinline__ void bar_readers() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool all_ok(bool ok) {
  uint32_t res;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, 1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(res)
      : "r"((uint32_t)ok)
      : "memory");
  return res != 0;
}

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
      for (int i = 0; i < kPairs; ++i) {
        mbar_init(&S.kv_full[i], i == kPairs - 1 ? 3 : 2);
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
    gather_loop<kFmt, 1, kPairs, kPairs>(base + kOffKV, warp - 6, S.ring, S.kv_full, S.kv_free,
                                         kErrGather);
  } else if (warp == 5) {
    uint32_t it = 0;
    if (resolve_rows<kFmt>(rows0, a, x, it, S.ring, kErrRing, [] {}))
      resolve_end(it, S.ring, kErrRing, [] {});
  } else if (warp == 4) {
    // A CTA without chunks waits for the launch before as well: this grid is not to be over while
    // that launch still runs, since the next call on the stream writes the tiles anew.
    if (n == 0) pdl_wait();
    if (n > 0 && elect_one()) {  // one thread issues everything (see attn_fp4.cu)
      const uint32_t idS = idesc_f16(kFmt == kFp4 ? 0 : 1, kQRows, kRows);
      const uint64_t dq = smem_desc(smem_u32(base + kOffQ), 16, 1024, kLayoutSw128);
      const uint64_t dk = smem_desc(smem_u32(base + kOffKV), 16, 1024, kLayoutSw128);
      pdl_wait();  // the q_hat tiles of the launch before
      mbar_arrive_expect_tx(&S.q_full, kAtoms * kQAtom);
      bulk_load(base + kOffQ, P.tiles + (size_t)x.stream * (kAtoms * kQAtom), kAtoms * kQAtom, &S.q_full);
      bool ok = mbar_wait(&S.q_full, 0, kErrMma);
      for (int it = 0; it < n && ok; ++it) {
        const int slot = it & 1;
        ok = mbar_wait(&S.s_free[slot], ((uint32_t)(it >> 1) & 1) ^ 1, kErrMma);
#pragma unroll 1
        for (int p = 0; p < kPairs && ok; ++p) {
          ok = mbar_wait(&S.kv_full[p], (uint32_t)it & 1, kErrMma);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kq = 0; kq < 8; ++kq) {  // two atoms of four steps
            const int atom = kq >> 2;
            mma_f16(tmem + 64 * slot, dq + (((2 * p + atom) * kQAtom + (kq & 3) * 32) >> 4),
                    dk + (((2 * p + atom) * kAtomBytes + (kq & 3) * 32) >> 4), idS,
                    (p | kq) != 0 ? 1u : 0u);
          }
          mma_commit(&S.kv_free[p]);
        }
        if (ok) mma_commit(&S.s_full[slot]);
      }
      mma_commit(&S.done);  // fires when nothing issued here is in flight
      mbar_wait(&S.done, 0, kErrMma);
    }
    __syncwarp();
  } else {
    // ---- logits: thread t of warp w has rows 8 i + 2 (t % 4), + 1 of the chunk for heads
    //      16 w + t / 4 and that + 8, hi and lo from the two halves of the warp's lanes ----
    const uint32_t lane_base = tmem + ((uint32_t)(32 * warp) << 16);
    const int quad = lane & 3, hq = 16 * warp + (lane >> 2);
    float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    float* const zt = P.z + ((size_t)x.stream * P.z_tiles) * kTile;
    uint8_t* const stage = base + kOffZ;
    bool ok = true;
#pragma unroll 1
    for (int it = 0; it < n; ++it) {
      const int j = x.c0 + it, slot = it & 1, rs = it % kRing;
      ok = mbar_wait(&S.s_full[slot], (uint32_t)(it >> 1) & 1, kErrRead);
      if (tid == 0) bulk_store_wait_read();  // the staged tile of the chunk before has left
      ok = all_ok(ok);  // the four warps leave together
      if (!ok) break;
      tc_fence_after();
      uint32_t hi[32], lo[32];
      tmem_ld_16x256b_x8(lane_base + 64 * slot, hi);
      tmem_ld_16x256b_x8(lane_base + (16u << 16) + 64 * slot, lo);
      tmem_ld_wait();
      const uint32_t live[2] = {S.ring.mask[rs][0], S.ring.mask[rs][1]};
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.ring.free[rs]);
        mbar_arrive(&S.s_free[slot]);
      }
      float cm[2] = {-INFINITY, -INFINITY};
      float* const z = reinterpret_cast<float*>(hi);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int row = 8 * (i >> 2) + 2 * quad + (i & 1), h = (i >> 1) & 1;
        z[i] = (live[row >> 5] >> (row & 31)) & 1u
                   ? (__uint_as_float(hi[i]) + __uint_as_float(lo[i])) * P.scale2
                   : -INFINITY;
        cm[h] = fmaxf(cm[h], z[i]);
      }
      if (j < x.l.nc) {
        // tile [head][64 rows]; the 32-byte segments of a head are permuted by head % 8, so that
        // eight heads' stores fall into distinct banks
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int head = hq + 8 * (i & 1), seg = (i >> 1) ^ (head & 7);
          *reinterpret_cast<float2*>(stage + head * 256 + seg * 32 + quad * 8) =
              make_float2(z[2 * i], z[2 * i + 1]);
        }
        fence_proxy_async_smem();
      }
      bar_readers();
      if (tid == 0 && j < x.l.nc) bulk_store(zt + (size_t)j * kTile, stage, kTile * 4);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (fmaxf passes over a NaN, the sum does not: rows that are all NaN or masked are summed
        // against 0)
        const float mn = fmaxf(m[h], cm[h]), ref = mn == -INFINITY ? 0.f : mn;
        float s2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; ++i) s2[i & 1] += ex2(z[4 * (i >> 1) + 2 * h + (i & 1)] - ref);
        sum[h] = sum[h] * ex2(m[h] - ref) + (s2[0] + s2[1]);
        m[h] = mn;
      }
    }
    // the four threads of a head
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float M = m[h];
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 1));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 2));
      float t = m[h] == -INFINITY ? 0.f : sum[h] * ex2(m[h] - M);
      if (sum[h] != sum[h]) t = sum[h];  // a NaN stays one
      t += __shfl_xor_sync(0xffffffffu, t, 1);
      t += __shfl_xor_sync(0xffffffffu, t, 2);
      if (quad == 0) {
        float* pp = P.part + ((size_t)x.stream * P.nsplit + x.split) * (2 * kHg);
        pp[hq + 8 * h] = M;
        pp[kHg + hq + 8 * h] = t;
      }
    }
    if (tid == 0) bulk_store_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

constexpr int kRedThreads = 256;
constexpr int kParts = 4;                      // threads per row, each a quarter of the heads
constexpr int kRedRows = kRedThreads / kParts;  // 64: one tile of z

// L[h] = log2 of the softmax denominator of head h of query bt, by four threads with every
// fourth split each (one round trip, where a thread a head took two of many loads).
__device__ __forceinline__ void denominators(const Params& P, int bt, float* L) {
  const int q = threadIdx.x & 3;
#pragma unroll 2
  for (int h = threadIdx.x >> 2; h < P.a.H; h += kRedThreads / 4) {  // H: a multiple of 64
    const float* pp = P.part + (size_t)(bt * P.G + h / kHg) * P.nsplit * (2 * kHg) + h % kHg;
    const float zs = P.a.sink ? P.a.sink[h] * 1.44269504088896341f : -INFINITY;
    float m[kMaxSplit / 4], l[kMaxSplit / 4], M = zs;
#pragma unroll
    for (int i = 0; i < kMaxSplit / 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      if (q + 4 * i < P.nsplit) {
        m[i] = pp[(q + 4 * i) * 2 * kHg];
        l[i] = pp[(q + 4 * i) * 2 * kHg + kHg];
      }
    }
#pragma unroll
    for (int i = 0; i < kMaxSplit / 4; ++i) M = fmaxf(M, m[i]);
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 1));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 2));
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxSplit / 4; ++i)  // a split of no row has l = 0, one of NaN alone l = NaN
      t = fmaf(l[i], m[i] == -INFINITY ? 0.f : exp2f(m[i] - M), t);
    t += __shfl_xor_sync(0xffffffffu, t, 1);
    t += __shfl_xor_sync(0xffffffffu, t, 2);
    if (zs != -INFINITY) t += exp2f(zs - M);
    if (q == 0) L[h] = M == -INFINITY && t == 0.f ? INFINITY : M + log2f(t);  // no row: weights of 0
  }
}

// The sum over all heads of 2^(z - L) for row `row` of query bt, by four threads with a
// quarter of each group's heads each; all four get it (summed in a fixed order). L and `part`
// are shared arrays of H and kRedThreads floats; the whole block calls. The first group's z are
// requested before L is worked out.
__device__ __forceinline__ float weight_of(const Params& P, int bt, int64_t row, bool in, float* L,
                                           float* part) {
  constexpr int kMine = kHg / kParts;
  const int p = threadIdx.x / kRedRows, r = threadIdx.x % kRedRows, c = (int)(row % kRows);
  float zv[kMine];
  auto load = [&](int g) {
    const float* z = P.z + ((size_t)(bt * P.G + g) * P.z_tiles + row / kRows) * kTile;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int h = p * kMine + i;
      zv[i] = z[h * kRows + (((c >> 3) ^ (h & 7)) << 3) + (c & 7)];
    }
  };
  if (in) load(0);
  denominators(P, bt, L);
  __syncthreads();
  float s = 0.f;
  if (in) {
    for (int g = 0; g < P.G; ++g) {
      if (g > 0) load(g);
#pragma unroll
      for (int i = 0; i < kMine; ++i) s += ex2(zv[i] - L[g * kHg + p * kMine + i]);
    }
  }
  part[threadIdx.x] = s;
  __syncthreads();
  const float sum = (part[r] + part[kRedRows + r]) + (part[2 * kRedRows + r] + part[3 * kRedRows + r]);
  __syncthreads();
  return sum;
}

__global__ void __launch_bounds__(kRedThreads) k_mass_dense(const __grid_constant__ Params P) {
  extern __shared__ float sm[];
  float *part = sm, *L = sm + kRedThreads;  // [H]
  const int b = blockIdx.y;
  const int64_t e0 = (int64_t)blockIdx.x * kRedRows, e = e0 + threadIdx.x % kRedRows;
  const bool writer = threadIdx.x < kRedRows && e < P.a.n_cap;
  const float old = writer ? P.acc[(size_t)b * P.a.n_cap + e] : 0.f;
  pdl_wait();
  float sum = 0.f;
  for (int t = 0; t < P.a.T; ++t) {
    const int bt = b * P.a.T + t;
    const int64_t n_vis = make_list(P.a, P.a.q_pos[bt]).n_vis;
    if (e0 >= n_vis) continue;  // the same for the whole block
    sum += weight_of(P, bt, e, e < n_vis, L, part);  // ends with a barrier: L may be rewritten
  }
  if (writer) P.acc[(size_t)b * P.a.n_cap + e] = fmaf(P.decay, old, sum);
}

__global__ void __launch_bounds__(kRedThreads) k_mass_sparse(const __grid_constant__ Params P) {
  extern __shared__ float sm[];
  float *part = sm, *L = sm + kRedThreads;
  const int bt = blockIdx.y, b = bt / P.a.T;
  const int j = blockIdx.x * kRedRows + threadIdx.x % kRedRows;
  const int e = j < P.a.k ? P.a.idx[(size_t)bt * P.a.k + j] : -1;
  pdl_wait();
  const bool in = e >= 0 && e < P.a.n_cap;
  const float w = weight_of(P, bt, j, in, L, part);
  if (!in || threadIdx.x >= kRedRows) return;
  unsigned long long* at = P.fixed + (size_t)b * P.a.n_cap + e;
  if (w <= P.slot_max) atomicAdd(at, (unsigned long long)__float2ll_rn(w * P.fixed_one));
  else atomicOr(at, kNotFinite);  // a NaN
}

__global__ void __launch_bounds__(kRedThreads) k_mass_finish(const __grid_constant__ Params P) {
  pdl_wait();
  const size_t n = (size_t)P.a.B * P.a.n_cap, i = (size_t)blockIdx.x * kRedThreads + threadIdx.x;
  if (i >= n) return;
  const unsigned long long f = P.fixed[i];
  const float add = f & kNotFinite ? __uint_as_float(0x7fc00000u)
                                   : (float)((double)f * P.step);
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
  int64_t z_tiles;
  size_t z_bytes, part_bytes, fixed_bytes, tile_bytes, rope_bytes;
};

Plan make_plan(const MqaArgs& a) {
  Plan p;
  const size_t streams = (size_t)a.B * a.T * (a.H / kHg);
  p.nsplit = choose_split(a);
  p.z_tiles = ((a.k > 0 ? a.k : a.n_cap) + kRows - 1) / kRows;
  p.z_bytes = streams * (size_t)p.z_tiles * kTile * sizeof(float);
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
  P.z_tiles = pl.z_tiles;
  P.z = reinterpret_cast<float*>(w);
  P.part = reinterpret_cast<float*>(w + pl.z_bytes);
  P.fixed = a.k > 0 ? reinterpret_cast<unsigned long long*>(w + pl.z_bytes + pl.part_bytes) : nullptr;
  P.acc = acc;
  P.scale2 = a.scale * 1.44269504088896341f;
  P.decay = decay;
  int bits = 62;
  for (int64_t most = 1; most < (int64_t)a.T * a.H; most *= 2) --bits;
  P.fixed_one = std::ldexp(1.f, bits);
  P.step = std::ldexp(1.0, -bits);
  P.slot_max = 1.25f * (float)a.H;  // T slots of it stay below 2^63 steps
  char* tiles = w + pl.z_bytes + pl.part_bytes + pl.fixed_bytes;
  P.tiles = reinterpret_cast<const uint8_t*>(tiles);
  const int64_t streams = (int64_t)a.B * a.T * P.G;
  auto kern = a.fp4 ? k_mass_logits<kFp4> : k_mass_logits<kBf16>;
  const size_t smem = 1024 + kOffEnd + sizeof(Smem);
  static std::atomic<uint64_t> allowed[2];
  cudaError_t e = allow_smem(kern, (int)smem, allowed[a.fp4]);
  if (e != cudaSuccess) return e;
  e = launch_q_tiles(a, true, tiles, tiles + pl.tile_bytes, st);
  if (e != cudaSuccess) return e;
  e = launch(true, kern, dim3((unsigned)(streams * P.nsplit)), dim3(kThreads), smem, st, P);
  if (e != cudaSuccess) return e;
  const size_t lsm = (size_t)(kRedThreads + a.H) * sizeof(float);
  if (a.k == 0)
    return launch(true, k_mass_dense,
                  dim3((unsigned)((a.n_cap + kRedRows - 1) / kRedRows), (unsigned)a.B),
                  dim3(kRedThreads), lsm, st, P);
  e = launch(true, k_mass_sparse,
             dim3((unsigned)((a.k + kRedRows - 1) / kRedRows), (unsigned)(a.B * a.T)),
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
