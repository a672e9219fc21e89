// Stage 4 over 4-bit cache rows (CSA_MIXED_MXFP4_BF16 pages): shared-KV MQA, sparse CSA rows or
// dense HCA rows, plus the sliding window, with query RMSNorm / RoPE, sink and output
// un-rotation.
//
// 【论文解读】DeepSeek-V4 一(三)1(3) / 2(2): every KV row is key and value for all heads; 3(1)
// RMSNorm of each query head; 3(2) RoPE(t) on the last r dims of q, RoPE(-t) on the output;
// 3(3) window rows attended with the compressed rows; 3(4) exp(z'_h) in the denominator. The
// row format is MXFP4 (OCP MX v1.0) for the values without RoPE, as 二(四) keeps the indexer's
// keys, and bf16 for the RoPE values.
//
// Work: a stream is (query, group of 64 heads); its row list is cut into chunks of 64 rows
// and split over `nsplit` CTAs. Per chunk, with f16 operands in 128B-swizzled shared memory
// and fp32 accumulators in TMEM:
//   S[64 heads x 64 rows] = q_hat . K^T          (M = 64; A = q_hat, B = the KV tile)
//   P = 2^(S * scale * log2(e) - m_h) in f16     (four threads a head)
//   O^T[4 x 128 dims x 64 heads] += V^T . P^T    (A = the same KV tile read MN-major)
// q_hat comes as a prepared tile (q_tiles.cu). Warps: 0-3 softmax and epilogue; 4 issues the
// MMAs; 5 resolves addresses; 6-13 each widen one 64-value atom of every row (kv_rows.cuh). Two
// KV buffers: S of chunk j + 1 may be issued before O^T of chunk j, so the tensor cores work
// during the softmax, and the gather warps fill the buffer that O^T released.
// The running max m_h is raised only when a chunk's max exceeds it by more than 2^11.5 (then
// O^T and l are rescaled); P stays below 2^11.5, inside f16, and sums are fp32.
// One split: the CTA finalises. Several: it writes (m, l, O) partials and k_attn_fp4_combine
// merges them in a fixed order.
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

constexpr int kThreads = 14 * 32;
constexpr int kBuf = 2;
constexpr float kLazy = 11.5f;  // rescale threshold (log2 units)
constexpr int kMaxSplit = 32;

constexpr int kSlotKV = kAtoms * kAtomBytes;  // 64 KB
constexpr int kOffKV = 0;
constexpr int kOffQ = kBuf * kSlotKV;         // [atom][head][128 B]
constexpr int kOffP = kOffQ + kAtoms * kHg * 128;
constexpr int kSlotP = kHg * 128;             // [head][64 rows]
constexpr int kOffEnd = kOffP + kBuf * kSlotP;

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;    // S: two tiles of 64 columns (M = 64 layout)
constexpr uint32_t kColO = 256;  // O^T slice s: 256 + 64 s

// 211 ring free, 212 ring full / 213 buffer free, 214 KV / q_hat / P full, 215 S / O^T done;
// 216 = 211 + 5: a page id outside the pool
enum { kErrRing = 211, kErrGather = 212, kErrMma = 214, kErrSoftmax = 215 };

struct Smem {
  AddrRing ring;
  uint64_t kv_full[kBuf], kv_free[kBuf], s_full[kBuf], p_full[kBuf], q_full, done;
  uint32_t tmem_slot;
  uint64_t vote[2];
  uint32_t need[4][4];  // [chunk % 4][softmax warp]: a head of the warp raised its maximum
  float m_used[kHg], l_sum[kHg], alpha[2][kHg], fin[kHg];
  float2 rope[kR / 2];  // cos, sin of the query's position
};

struct Params {
  MqaArgs a;
  int G, nsplit;
  float* part;  // [stream][split][64 m | 64 l | 64 x 512 O], or nullptr
  const uint8_t* tiles;  // q_hat tiles, 64 KB per stream
  const float2* rope;    // [B * T][32]
  float scale2;          // scale * log2(e)
};

constexpr size_t kPartFloats = (size_t)kHg * (kC + 2);

__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// A wait of one softmax warp. No barrier of the four warps follows it inside the chunk loop,
// so a warp whose wait gives up leaves the others to their own limits.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, kErrSoftmax));
}

// 16 TMEM lanes x 64 columns of 32-bit as eight 16 x 8 pieces: thread t gets, in registers 4 i
// .. 4 i + 3, columns 8 i + 2 (t % 4), + 1 of lane t / 4 and of lane t / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31},"
      " [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads, 1) k_attn_fp4(const __grid_constant__ Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_align1024(smem_raw);
  Smem& S = *reinterpret_cast<Smem*>(base + kOffEnd);
  const MqaArgs& a = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stream = blockIdx.x / P.nsplit, split = blockIdx.x % P.nsplit;
  const int bt = stream / P.G, g = stream % P.G, b = bt / a.T, h0 = g * kHg;

  if (warp == 4) {
    if (lane == 0) {
      for (int i = 0; i < kRing; ++i) {
        mbar_init(&S.ring.full[i], 1);
        mbar_init(&S.ring.free[i], 8 + 4);  // gather warps; softmax warps (the mask)
      }
      for (int i = 0; i < kBuf; ++i) {
        mbar_init(&S.kv_full[i], 8);  // the gather warps
        mbar_init(&S.kv_free[i], 1);
        mbar_init(&S.s_full[i], 1);
        mbar_init(&S.p_full[i], 4);
        mbar_init(&S.vote[i], 4);
      }
      mbar_init(&S.q_full, 1);
      mbar_init(&S.done, 1);
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(&S.tmem_slot, kTmemCols);
  }
  // The q_tiles launch before this one waited for everything earlier on the stream, and this
  // kernel starts after that: only the tiles themselves are waited for, below.
  const List l = make_list(a, bt);
  const int c0 = (int)(((int64_t)l.n_chunks * split) / P.nsplit);
  const int c1 = (int)(((int64_t)l.n_chunks * (split + 1)) / P.nsplit);
  RowBatch rows0;
  if (warp == 5) rows0.lookup(a, l, bt, b, c0, c1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = S.tmem_slot;

  if (warp >= 6) {
    gather_loop<kFp4, kBuf, false>(base + kOffKV, c0, c1, l.nc, warp - 6, S.ring, S.kv_full,
                                   S.kv_free, kErrGather);
  } else if (warp == 5) {
    resolve_rows<kFp4>(rows0, a, l, bt, b, c0, c1, S.ring, kErrRing);
  } else if (warp == 4) {
    // ------------------------------ MMA issuer ------------------------------
    // One thread runs the whole loop: a step of it (votes, branches) costs as much as its MMAs
    // when the warp runs it together.
    if (elect_one()) {
      const uint32_t idS = idesc_f16(0, kHg, kRows);             // M = 64, N = 64, both K-major
      const uint32_t idO = idesc_f16(0, 128, kHg) | (1u << 15);  // M = 128 dims; A MN-major
      const uint32_t sb = smem_u32(base);
      const uint64_t dq = smem_desc(sb + kOffQ, 16, 1024, kLayoutSw128);
      const uint64_t dk0 = smem_desc(sb + kOffKV, 16, 1024, kLayoutSw128);
      const uint64_t dv0 = smem_desc(sb + kOffKV, kAtomBytes, 1024, kLayoutSw128);
      const uint64_t dp0 = smem_desc(sb + kOffP, 16, 1024, kLayoutSw128);
      // S runs at most one chunk ahead of O^T. Where both could be issued, whichever has its
      // operands goes first, O^T before S (it frees a buffer). S tile slot i % 2 was read by the
      // softmax of chunk i - 2 before it published P(i - 2), which this thread has waited for.
      const int n = c1 - c0;
      int is = 0, iv = 0;
      bool ok = n > 0;
      if (ok) {
        pdl_wait();  // the tiles
        mbar_arrive_expect_tx(&S.q_full, kAtoms * kHg * 128);
        bulk_load(base + kOffQ, P.tiles + (size_t)stream * (kAtoms * kHg * 128), kAtoms * kHg * 128,
                  &S.q_full);
        ok = mbar_wait(&S.q_full, 0, kErrMma);
      }
      while (ok && iv < n) {
        const int ss = is & 1, sv = iv & 1;
        const uint32_t kp = (uint32_t)(is >> 1) & 1, pp = (uint32_t)(iv >> 1) & 1;
        bool do_v;
        if (iv < is && is < n && is - iv < kBuf) {
          const long long t0 = clock64();
          while (true) {
            do_v = mbar_test(&S.p_full[sv], pp);
            if (do_v || mbar_test(&S.kv_full[ss], kp)) break;
            if (clock64() - t0 > kSpinCycles) {
              set_error(kErrMma);
              ok = false;
              break;
            }
          }
        } else {
          do_v = iv < is;
          ok = mbar_wait(do_v ? &S.p_full[sv] : &S.kv_full[ss], do_v ? pp : kp, kErrMma);
        }
        if (!ok) break;
        tc_fence_after();
        if (do_v) {
          const uint64_t dv = dv0 + (uint64_t)(sv * (kSlotKV >> 4)), dp = dp0 + (uint64_t)(sv * (kSlotP >> 4));
#pragma unroll
          for (int kk = 0; kk < kRows / 16; ++kk)
#pragma unroll
            for (int sl = 0; sl < 4; ++sl)
              mma_f16(tmem + kColO + 64 * sl, dv + ((sl * 2 * kAtomBytes + kk * 2048) >> 4),
                      dp + ((kk * 32) >> 4), idO, (iv > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&S.kv_free[sv]);
          ++iv;
        } else {
          const uint64_t dk = dk0 + (uint64_t)(ss * (kSlotKV >> 4));
#pragma unroll
          for (int atom = 0; atom < kAtoms; ++atom)
#pragma unroll
            for (int kq = 0; kq < 4; ++kq)
              mma_f16(tmem + kColS + 64 * ss, dq + ((atom * (kHg * 128) + kq * 32) >> 4),
                      dk + ((atom * kAtomBytes + kq * 32) >> 4), idS, (atom | kq) != 0 ? 1u : 0u);
          mma_commit(&S.s_full[ss]);
          ++is;
        }
      }
      mma_commit(&S.done);  // fires when nothing issued here is in flight
      mbar_wait(&S.done, 0, kErrMma);
    }
    __syncwarp();
  } else {
    // ------------------------------ softmax ------------------------------
    const uint32_t lane_base = tmem + ((uint32_t)(32 * warp) << 16);
    // The M = 64 accumulator puts head 16w + i in TMEM lane 32w + i (i < 16). Four threads (a
    // quad) share heads h and h + 8: thread t has columns (rows of the chunk) 8 i + 2 (t % 4),
    // + 1 of head 16w + t / 4 in s[4i], s[4i + 1] and of that head + 8 in s[4i + 2], s[4i + 3]:
    // neighbouring rows pair up into one f16x2 of P without an exchange.
    const int quad = lane & 3, hq = 16 * warp + (lane >> 2);
    float mu[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
    bool ok = true;
#pragma unroll 1
    for (int j = c0; j < c1 && ok; ++j) {
      const int it = j - c0, slot = it % kBuf, rs = it % kRing;
      ok = wait_warp(&S.s_full[slot], (uint32_t)(it / kBuf) & 1);
      if (!ok) break;
      tc_fence_after();
      uint32_t sv[32];
      tmem_ld_16x256b_x8(lane_base + kColS + 64 * slot, sv);
      const uint32_t vm[2] = {S.ring.mask[rs][0], S.ring.mask[rs][1]};
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.ring.free[rs]);
      tmem_ld_wait();
      if ((vm[0] & vm[1]) != 0xffffffffu) {  // some row is masked
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int row = 8 * (i >> 2) + 2 * quad + (i & 1);
          if (!((vm[row >> 5] >> (row & 31)) & 1u)) sv[i] = 0xff800000u;  // -inf
        }
      }
      float cm[2], al[2], mref[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 16; ++i)
          m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(sv[4 * (i >> 1) + 2 * x + (i & 1)]));
        cm[x] = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) cm[x] = fmaxf(cm[x], __shfl_xor_sync(0xffffffffu, cm[x], 1));
#pragma unroll
      for (int x = 0; x < 2; ++x) cm[x] = fmaxf(cm[x], __shfl_xor_sync(0xffffffffu, cm[x], 2));
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        cm[x] *= P.scale2;
        al[x] = 1.f;
        if (cm[x] > mu[x] + kLazy || (mu[x] == -INFINITY && cm[x] != -INFINITY)) {
          al[x] = mu[x] == -INFINITY ? 0.f : ex2(mu[x] - cm[x]);
          mu[x] = cm[x];
        }
        lsum[x] *= al[x];
        mref[x] = mu[x] == -INFINITY ? 0.f : mu[x];
      }
      // the warps tell one another whether a maximum was raised, and look once P is computed
      const bool raised = __any_sync(0xffffffffu, (al[0] != 1.f || al[1] != 1.f) && j > c0);
      if (quad == 0) {
        S.alpha[it & 1][hq] = al[0];
        S.alpha[it & 1][hq + 8] = al[1];
      }
      if (lane == 0) S.need[it & 3][warp] = raised ? 1u : 0u;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.vote[it & 1]);
      // p = 2^(s * scale2 - m), paired into f16x2
      float l4[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int i = 0; i < 16; ++i) {  // i = 2 * (column group) + head
        const int x = i & 1;
        const float p0 = ex2(fmaf(__uint_as_float(sv[2 * i]), P.scale2, -mref[x]));
        const float p1 = ex2(fmaf(__uint_as_float(sv[2 * i + 1]), P.scale2, -mref[x]));
        l4[x][0] += p0;
        l4[x][1] += p1;
        sv[i] = pack2<kFp4>(p0, p1);
      }
      lsum[0] += l4[0][0] + l4[0][1];
      lsum[1] += l4[1][0] + l4[1][1];
      ok = wait_warp(&S.vote[it & 1], (uint32_t)(it >> 1) & 1);
      if (!ok) break;
      if ((S.need[it & 3][0] | S.need[it & 3][1] | S.need[it & 3][2] | S.need[it & 3][3]) != 0) {
        // rare: scale this warp's dims of O^T by alpha once the previous chunk's products are
        // done (a chunk's alpha is rewritten two chunks later, after all warps published P)
        const int pi = it - 1;
        ok = wait_warp(&S.kv_free[pi % kBuf], (uint32_t)(pi / kBuf) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int cg = 0; cg < 16; ++cg) {  // 4 slices x 4 groups of 16 heads
          uint32_t o[16];
          const uint32_t ta = lane_base + kColO + 16 * cg;
          tmem_ld_x16(ta, o);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 16; ++h)
            o[h] = __float_as_uint(__uint_as_float(o[h]) * S.alpha[it & 1][16 * (cg & 3) + h]);
          tmem_st_x16(ta, o);
        }
        tmem_st_wait();
      }
      if (it >= kBuf) {  // the P buffer was read by the products of chunk j - 2
        ok = wait_warp(&S.kv_free[slot], (uint32_t)((it - kBuf) / kBuf) & 1);
        if (!ok) break;
      }
      // K-major tile [head][64 rows]: 8 x 8 pieces of 16-bit values, four a store: column groups
      // 2 c and 2 c + 1 of heads 16w .. 16w + 7 and 16w + 8 .. 16w + 15. Lane l gives the address
      // of row l % 8 of piece l / 8 (heads + 8 in odd pieces).
      {
        const uint32_t pt = smem_u32(base + kOffP + slot * kSlotP);
        const int head = 16 * warp + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          stmatrix_x4(pt + sw128(head, 2 * c + (lane >> 4)), sv[4 * c], sv[4 * c + 1], sv[4 * c + 2],
                      sv[4 * c + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.p_full[slot]);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      lsum[x] += __shfl_xor_sync(0xffffffffu, lsum[x], 1);
      lsum[x] += __shfl_xor_sync(0xffffffffu, lsum[x], 2);
    }
    if (quad == 0) {
      S.m_used[hq] = mu[0];
      S.m_used[hq + 8] = mu[1];
      S.l_sum[hq] = lsum[0];
      S.l_sum[hq + 8] = lsum[1];
    }
    // ---- epilogue ----
    pdl_wait();  // the rotation, written beside the tiles
    if (tid < kR / 2) S.rope[tid] = P.rope[(size_t)bt * 32 + tid];
    if (ok && c1 > c0) {
      const int last = c1 - c0 - 1;
      ok = wait_warp(&S.kv_free[last % kBuf], (uint32_t)(last / kBuf) & 1);
    }
    bar_softmax();
    const bool single = P.nsplit == 1;
    float* pp = single ? nullptr : P.part + ((size_t)stream * P.nsplit + split) * kPartFloats;
    if (tid < kHg) {
      const float m = S.m_used[tid], lv = S.l_sum[tid];
      if (single) {
        const float zs = a.sink ? a.sink[h0 + tid] * 1.44269504088896341f : -INFINITY;
        float f = 0.f;
        if (lv != 0.f) {  // a NaN stays one
          const float M = fmaxf(m, zs);
          const float e = exp2f(m - M);
          f = e / (lv * e + (zs == -INFINITY ? 0.f : exp2f(zs - M)));
        }
        S.fin[tid] = f;
      } else {
        pp[tid] = m;
        pp[kHg + tid] = lv;
      }
    }
    bar_softmax();
    tc_fence_after();
    const bool have = ok && c1 > c0;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((size_t)bt * a.H + h0) * kC;
    // O^T slice by slice: thread = dim 128 sl + tid, 64 heads
#pragma unroll 1
    for (int sl = 0; sl < 4; ++sl) {
      uint32_t o[64];
      if (have) {
        tmem_ld_32x32b_x64(lane_base + kColO + 64 * sl, o);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int h = 0; h < 64; ++h) o[h] = 0u;
      }
      const int d = 128 * sl + tid;
      if (single) {
        float cs = 1.f, sn = 0.f;
        const bool rot = d >= kNope;
        if (rot) {
          cs = S.rope[(d - kNope) >> 1].x;
          sn = -S.rope[(d - kNope) >> 1].y;  // rotation by -t
        }
#pragma unroll
        for (int h = 0; h < 64; ++h) {
          const float y = __uint_as_float(o[h]) * S.fin[h];
          const float yp = __shfl_xor_sync(0xffffffffu, y, 1);
          float z = y;
          if (rot) z = (d & 1) == 0 ? y * cs - yp * sn : yp * sn + y * cs;
          out[(size_t)h * kC + d] = __float2bfloat16_rn(z);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 64; ++h) pp[2 * kHg + (size_t)h * kC + d] = __uint_as_float(o[h]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge the partials of one head (fixed split order), add the sink, rotate by -t. kBatch splits
// are loaded before any is used.
template <int kBatch>
__global__ void __launch_bounds__(256) k_attn_fp4_combine(const __grid_constant__ Params P) {
  const MqaArgs& a = P.a;
  const int stream = blockIdx.x, h = blockIdx.y;
  const int bt = stream / P.G, g = stream % P.G;
  const int d = 2 * threadIdx.x, ns = P.nsplit;
  const float* base = P.part + (size_t)stream * ns * kPartFloats;
  pdl_wait();
  pdl_trigger();
  const float zs = a.sink ? a.sink[g * kHg + h] * 1.44269504088896341f : -INFINITY;
  float2 cs_sn = make_float2(1.f, 0.f);  // of +t
  float M = zs, l = 0.f, o0 = 0.f, o1 = 0.f;
  for (int s0 = 0; s0 < ns; s0 += kBatch) {
    float ms[kBatch], ls[kBatch];
    float2 os[kBatch];
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const float* pp = base + (size_t)min(s0 + s, ns - 1) * kPartFloats;
      ms[s] = pp[h];
      ls[s] = pp[kHg + h];
      os[s] = *reinterpret_cast<const float2*>(pp + 2 * kHg + (size_t)h * kC + d);
    }
    if (s0 == 0 && d >= kNope) cs_sn = P.rope[(size_t)bt * 32 + ((d - kNope) >> 1)];
    float Mn = M;
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (s0 + s < ns) Mn = fmaxf(Mn, ms[s]);
    if (Mn == -INFINITY) continue;  // no row and no sink so far
    const float f0 = exp2f(M - Mn);
    l *= f0;
    o0 *= f0;
    o1 *= f0;
    M = Mn;
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      if (s0 + s < ns && ms[s] != -INFINITY) {
        const float f = exp2f(ms[s] - M);
        l = fmaf(ls[s], f, l);
        o0 = fmaf(os[s].x, f, o0);
        o1 = fmaf(os[s].y, f, o1);
      }
    }
  }
  float y0 = 0.f, y1 = 0.f;
  if (l != 0.f) {  // a NaN stays one
    const float den = l + (zs == -INFINITY ? 0.f : exp2f(zs - M));
    y0 = o0 / den;
    y1 = o1 / den;
  }
  if (d >= kNope) {
    const float u0 = y0 * cs_sn.x + y1 * cs_sn.y, u1 = y1 * cs_sn.x - y0 * cs_sn.y;
    y0 = u0;
    y1 = u1;
  }
  __nv_bfloat16* out =
      static_cast<__nv_bfloat16*>(a.out) + ((size_t)bt * a.H + g * kHg + h) * kC + d;
  *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(y0, y1);
}

// CTAs per stream: as many as fill the SMs, at most one per chunk of the longest list, at
// most kMaxSplit.
int choose_split(const MqaArgs& a) {
  const int64_t streams = (int64_t)a.B * a.T * (a.H / kHg);
  const int64_t rows = a.k > 0 ? a.k : a.n_cap;
  const int64_t chunks = (rows + kRows - 1) / kRows + ((int64_t)a.n_win + kRows - 1) / kRows;
  int64_t ns = device_sm_count() / (streams > 0 ? streams : 1);
  ns = ns < chunks ? ns : chunks;
  return (int)(ns < 1 ? 1 : (ns > kMaxSplit ? kMaxSplit : ns));
}

}  // namespace

bool attn_fp4_supported(const MqaArgs& a) {
  return a.c == kC && a.rope_dims == kR && a.H >= kHg && a.H % kHg == 0;
}

size_t attn_fp4_workspace_bytes(const MqaArgs& a) {
  const int ns = choose_split(a);
  const size_t part = ns <= 1 ? 0 : (size_t)a.B * a.T * (a.H / kHg) * ns * kPartFloats * sizeof(float);
  return q_tiles_bytes(a, false) + q_rope_bytes(a) + part;
}

cudaError_t launch_attn_fp4(const MqaArgs& a, void* ws, size_t ws_bytes, cudaStream_t st) {
  Params P;
  P.a = a;
  P.G = a.H / kHg;
  P.nsplit = choose_split(a);
  if (ws_bytes < attn_fp4_workspace_bytes(a)) return cudaErrorInvalidValue;
  uint8_t* w = static_cast<uint8_t*>(ws);
  P.tiles = w;
  P.rope = reinterpret_cast<float2*>(w + q_tiles_bytes(a, false));
  P.part = P.nsplit > 1
               ? reinterpret_cast<float*>(w + q_tiles_bytes(a, false) + q_rope_bytes(a))
               : nullptr;
  P.scale2 = a.scale * 1.44269504088896341f;
  const int64_t streams = (int64_t)a.B * a.T * P.G;
  const size_t smem = 1024 + kOffEnd + sizeof(Smem);
  cudaError_t e = cudaFuncSetAttribute(k_attn_fp4, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_q_tiles(a, false, w, w + q_tiles_bytes(a, false), st);
  if (e != cudaSuccess) return e;
  e = launch(true, k_attn_fp4, dim3((unsigned)(streams * P.nsplit)), dim3(kThreads), smem, st, P);
  if (e != cudaSuccess || P.nsplit == 1) return e;
  return launch(true, P.nsplit <= 8 ? k_attn_fp4_combine<8> : k_attn_fp4_combine<16>,
                dim3((unsigned)streams, kHg), dim3(256), 0, st, P);
}

cudaError_t attn_fp4_device_error(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, tc::g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(tc::g_device_error, &zero, sizeof(int));
}

}  // namespace csa
