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
// q_hat comes as a prepared tile (q_tiles.cu). Warps: 0-3 softmax and epilogue; 4 issues S and 6
// O^T; 5 resolves addresses; 7-15 each widen one 64-value atom of every row (kv_rows.cuh). Two
// KV buffers: S of chunk j + 1 may be issued before O^T of chunk j, so the tensor cores work
// during the softmax, and the gather warps fill the buffer that O^T released.
// The exponent's reference m_h is set 8.5 below a chunk's largest logit (log2 units), and anew only
// when a later chunk's passes it by more than 15 (then O^T and l are rescaled): a head's largest P
// lies between 2^8.5 and 2^15, inside f16, and sums are fp32. f16 has steps of 2^-24 below 2^-14, so
// a row's weight is off by 2^-11 of itself or 2^-33.5 of the head's largest, whichever is more: over
// n rows by n 2^-33.5 of the output, 2^-13.5 at a million. (With P near 1 for the largest, rows below
// 2^-25 of it would be lost from O and kept in l: 2^-8.5 of the output over 262144 rows.) Set 9.5
// below and anew above 14.5, dense decode took 42.8 instead of 42.1 us, for more rescaling.
// One split: the CTA finalises. Several: it writes (m, l, O) partials and k_attn_fp4_combine
// merges them in a fixed order.
//
// Roundings: q_hat and P to f16 (11 bits; bf16 operands would keep 8), the output to bf16; the
// cache rows are exact f16, logits, maxima, sums and O are fp32. The f16 roundings are 2^-11 each beside
// the output's 2^-8: against 64 bits the output is off by 1.7e-3 rms, as one computed in fp32 and rounded
// once, and from that it differs by 3e-4 to 7e-4.
//
// What bounds it: operands come from shared memory at 128 bytes a cycle, and an M = 64 product
// of 64 heads has few operations per byte: 4 KB and 32 cycles for each 16 of K in S, 6 KB and 48
// in a slice of O^T, 512 cycles for the gathered rows' stores. Together 2300 of the 3050 cycles
// a chunk takes; the rest is the chain gather -> S -> softmax -> O^T over two buffers. A CTA
// starts with four dependent reads (position, list, page, row; 3.5 us to the first S) and a
// split one ends with 128 KB of partials and their merge (4.5 us), which is most of a call that
// gives a CTA one chunk. Measured, calls one after another: 16 queries x 64 heads over
// 8192 entries 42.3 us (342 TFLOP/s), 8 x 64 heads over lists of 512 14.3 us, 2048 queries with lists
// of 512 346 us (497 TFLOP/s).
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

constexpr int kThreads = (7 + kGatherWarps) * 32;
constexpr int kBuf = 2;
constexpr int kFree = 4;  // a buffer is given back in four pairs of atoms, one per slice of O^T
constexpr float kUp = 8.5f;     // log2 of P where the reference is set, at a chunk's maximum
constexpr float kTop = 15.f;    // the reference is set anew above this (f16 ends at 2^16; a logit's
                                // rounding to fp32 may add to the difference)
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

// What the other roles have to know of an item; n = 0 ends the list.
struct alignas(16) ItemInfo {
  int stream, bt, w;
  uint32_t n;  // chunks, at least one (an empty share has one whose rows are all masked)
};
constexpr int kItems = 8;  // see the address warp

struct Smem {
  AddrRing ring;
  ItemInfo info[kItems];
  uint64_t item_full[kItems];
  uint64_t kv_full[kBuf], kv_free[kBuf * kFree], s_full[kBuf], p_full[kBuf], q_full, done[2];
  uint32_t tmem_slot;
  alignas(16) float alpha[kHg], fin[kHg];
};

struct Params {
  MqaArgs a;
  int G, nsplit, items;  // items: streams * nsplit
  float* part;  // [stream][split][64 m | 64 l | 4 slices x 64 heads x 128 dims of O], or nullptr
  const uint8_t* tiles;  // q_hat tiles, 64 KB per stream
  const float2* rope;    // [B * T][32]
  float scale2;          // scale * log2(e)
};

constexpr size_t kPartFloats = (size_t)kHg * (kC + 2);

__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool all_softmax(bool ok) {
  uint32_t res;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, 1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(res)
      : "r"((uint32_t)ok)
      : "memory");
  return res != 0;
}
// Barrier of the four warps; the number of threads that vote.
__device__ __forceinline__ uint32_t count_softmax(bool vote) {
  uint32_t n;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.popc.u32 %0, 1, 128, q;\n\t}"
      : "=r"(n)
      : "r"((uint32_t)vote)
      : "memory");
  return n;
}
// A wait of one softmax warp. One that gives up is told to the others by the next vote.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, kErrSoftmax));
}

__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
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
  const int step = gridDim.x;

  if (warp == 4) {
    if (lane == 0) {
      for (int i = 0; i < kRing; ++i) {
        mbar_init(&S.ring.full[i], 1);
        mbar_init(&S.ring.free[i], kGatherWarps + 4);  // and the softmax warps (the mask)
      }
      for (int i = 0; i < kBuf; ++i) {
        mbar_init(&S.kv_full[i], kGatherWarps);
        for (int k = 0; k < kFree; ++k) mbar_init(&S.kv_free[i * kFree + k], 1);
        mbar_init(&S.s_full[i], 1);
        mbar_init(&S.p_full[i], 4);
      }
      for (int i = 0; i < kItems; ++i) mbar_init(&S.item_full[i], 1);
      mbar_init(&S.q_full, 1);
      for (int i = 0; i < 2; ++i) mbar_init(&S.done[i], 1);
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(&S.tmem_slot, kTmemCols);
  }
  // The q_tiles launch before this one waited for everything earlier on the stream, and this
  // kernel starts after that: only the tiles themselves are waited for, below.
  int w = blockIdx.x;
  Item x;
  RowBatch rows0;
  // a share without rows becomes one chunk without rows
  auto set_item = [&](int64_t t) {
    x.set(a, w, P.G, P.nsplit, t);
    if (x.c1 == x.c0) x.c1 = x.c0 + 1;
  };
  if (warp == 5) {
    set_item(item_pos(a, w, P.G, P.nsplit));
    rows0.lookup(a, x, x.c0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = S.tmem_slot;
  // Each role walks the CTA's items (one, where streams are split; several for many queries)
  // with its own count of chunks, so the next item's rows are gathered and multiplied while the
  // last one is finalised. The address warp works the items out and passes them on: with every
  // role doing so for itself, the change of item took 1800 cycles.
  uint32_t it = 0;
  bool ok = true;
  if (warp >= 7) {
    gather_loop<kFp4, kBuf, 1, kFree>(base + kOffKV, warp - 7, S.ring, S.kv_full, S.kv_free,
                                      kErrGather);
  } else if (warp == 5) {
    // An item is passed on where its first chunk `it` has its place in the ring: chunk it - 4 has
    // left the softmax, so S of it is done, its buffer was given back by chunk it - 6, and every
    // role is at most seven items (of a chunk at least) behind.
    uint32_t item = 0;
    auto pass = [&](uint32_t n) {
      if (lane == 0) {
        S.info[item % kItems] = ItemInfo{x.stream, x.bt, w, n};
        mbar_arrive(&S.item_full[item % kItems]);
      }
      ++item;
    };
    while (true) {
      const bool more = w + step < P.items;
      int64_t t_next = 0;
      if (more) t_next = item_pos(a, w + step, P.G, P.nsplit);
      ok = resolve_rows<kFp4>(rows0, a, x, it, S.ring, kErrRing,
                              [&] { pass((uint32_t)(x.c1 - x.c0)); });
      if (!ok || !more) break;
      w += step;
      set_item(t_next);
      rows0.lookup(a, x, x.c0);
    }
    if (ok) resolve_end(it, S.ring, kErrRing, [&] { pass(0); });
  } else if (warp == 4) {
    // ------------------------------ S ------------------------------
    // One thread runs the whole loop (the votes and branches of a converged warp cost as much as
    // the MMAs), and another warp issues O^T: a thread that issued both spent its time asking
    // which of the two had its operands.
    if (elect_one()) {
      const uint32_t idS = idesc_f16(0, kHg, kRows);  // M = 64, N = 64, both K-major
      const uint32_t sb = smem_u32(base);
      const uint64_t dq = smem_desc(sb + kOffQ, 16, 1024, kLayoutSw128);
      const uint64_t dk0 = smem_desc(sb + kOffKV, 16, 1024, kLayoutSw128);
      constexpr uint32_t kQBytes = kAtoms * kHg * 128;
      pdl_wait();  // the tiles
      for (uint32_t item = 0;; ++item) {
        ok = mbar_wait(&S.item_full[item % kItems], (item / kItems) & 1, kErrMma);
        const ItemInfo info = S.info[item % kItems];
        if (!ok || info.n == 0) break;
        mbar_arrive_expect_tx(&S.q_full, kQBytes);
        bulk_load(base + kOffQ, P.tiles + (size_t)info.stream * kQBytes, kQBytes, &S.q_full);
        if (info.w + step < P.items)  // the next tile towards L2 (an item a stream here)
          bulk_prefetch_l2(P.tiles + (size_t)(info.stream + step) * kQBytes, kQBytes);
        ok = mbar_wait(&S.q_full, item & 1, kErrMma);
        const uint32_t end = it + info.n;
        for (; ok && it != end; ++it) {
          const uint32_t slot = it & 1, ph = (it >> 1) & 1;
          // The buffer was given back by the products of chunk it - 2, so the softmax has read
          // this S tile, too.
          ok = mbar_wait(&S.kv_full[slot], ph, kErrMma);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dk = dk0 + (uint64_t)(slot * (kSlotKV >> 4));
#pragma unroll 1
          for (int atom = 0; atom < kAtoms; ++atom)
#pragma unroll
            for (int kq = 0; kq < 4; ++kq)
              mma_f16(tmem + kColS + 64 * slot, dq + ((atom * (kHg * 128) + kq * 32) >> 4),
                      dk + ((atom * kAtomBytes + kq * 32) >> 4), idS, (atom | kq) != 0 ? 1u : 0u);
          mma_commit(&S.s_full[slot]);
        }
        // the item's last S has read q_hat before the next one replaces it
        ok = ok && mbar_wait(&S.s_full[(it - 1) & 1], ((it - 1) >> 1) & 1, kErrMma);
        if (!ok) break;
      }
      mma_commit(&S.done[0]);  // fires when nothing issued here is in flight
      mbar_wait(&S.done[0], 0, kErrMma);
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------ O^T ------------------------------
    if (elect_one()) {
      const uint32_t idO = idesc_f16(0, 128, kHg) | (1u << 15);  // M = 128 dims; A MN-major
      const uint32_t sb = smem_u32(base);
      const uint64_t dv0 = smem_desc(sb + kOffKV, kAtomBytes, 1024, kLayoutSw128);
      const uint64_t dp0 = smem_desc(sb + kOffP, 16, 1024, kLayoutSw128);
      for (uint32_t item = 0; ok; ++item) {
        ok = mbar_wait(&S.item_full[item % kItems], (item / kItems) & 1, kErrMma);
        const uint32_t first = it, n = S.info[item % kItems].n, end = it + n;
        if (!ok || n == 0) break;
        for (; it != end; ++it) {
          const uint32_t slot = it & 1;
          // P says that S is done, that O^T was rescaled where needed, and, of an item's first
          // chunk, that O^T of the item before has been read
          ok = mbar_wait(&S.p_full[slot], (it >> 1) & 1, kErrMma);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = dv0 + (uint64_t)(slot * (kSlotKV >> 4)),
                         dp = dp0 + (uint64_t)(slot * (kSlotP >> 4));
#pragma unroll 1
          for (int sl = 0; sl < 4; ++sl) {  // a slice's two atoms are given back by themselves
#pragma unroll
            for (int kk = 0; kk < kRows / 16; ++kk)
              mma_f16(tmem + kColO + 64 * sl, dv + ((sl * 2 * kAtomBytes + kk * 2048) >> 4),
                      dp + ((kk * 32) >> 4), idO, (it != first || kk > 0) ? 1u : 0u);
            mma_commit(&S.kv_free[slot * kFree + sl]);
          }
        }
      }
      mma_commit(&S.done[1]);
      mbar_wait(&S.done[1], 0, kErrMma);
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
    // fires when every product of chunk i is done (its last slice's)
    auto chunk_done = [&](uint32_t i) { return &S.kv_free[(i % kBuf) * kFree + kFree - 1]; };
    for (uint32_t item = 0;; ++item) {
      ok = wait_warp(&S.item_full[item % kItems], (item / kItems) & 1) && ok;
      // the four warps leave together; S.fin has been read before this item writes it
      ok = all_softmax(ok);
      const ItemInfo x = S.info[item % kItems];
      if (!ok || x.n == 0) break;
      const uint32_t it0 = it, n = x.n;
      float mu[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
#pragma unroll 1
      for (; it - it0 < n; ++it) {  // (left by the vote alone, so by all four warps)
        const uint32_t slot = it % kBuf, rs = it % kRing;
        ok = wait_warp(&S.s_full[slot], (it / kBuf) & 1) && ok;
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
        for (int h = 0; h < 2; ++h) {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 16; ++i)
            m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(sv[4 * (i >> 1) + 2 * h + (i & 1)]));
          cm[h] = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) cm[h] = fmaxf(cm[h], __shfl_xor_sync(0xffffffffu, cm[h], 1));
#pragma unroll
        for (int h = 0; h < 2; ++h) cm[h] = fmaxf(cm[h], __shfl_xor_sync(0xffffffffu, cm[h], 2));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cm[h] *= P.scale2;
          al[h] = 1.f;
          if (cm[h] > mu[h] + kTop || (mu[h] == -INFINITY && cm[h] != -INFINITY)) {
            const float to = cm[h] - kUp;
            al[h] = mu[h] == -INFINITY ? 0.f : ex2(mu[h] - to);
            mu[h] = to;
          }
          lsum[h] *= al[h];
          mref[h] = mu[h] == -INFINITY ? 0.f : mu[h];
        }
        // One barrier of the four warps per chunk: the whole warp votes where a maximum was
        // raised, a single lane where the warp's wait gave up, and all leave together then.
        const bool raised = __any_sync(0xffffffffu, (al[0] != 1.f || al[1] != 1.f) && it != it0);
        if (raised && quad == 0) {
          S.alpha[hq] = al[0];
          S.alpha[hq + 8] = al[1];
        }
        if (!raised && quad == 0 && it != it0) S.alpha[hq] = S.alpha[hq + 8] = 1.f;
        const uint32_t votes = count_softmax(ok ? raised : lane == 0);
        if (votes & 31u) {
          ok = false;
          break;
        }
        // p = 2^(s * scale2 - m), paired into f16x2
        float l4[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < 16; ++i) {  // i = 2 * (column group) + head
          const int h = i & 1;
          const float p0 = ex2(fmaf(__uint_as_float(sv[2 * i]), P.scale2, -mref[h]));
          const float p1 = ex2(fmaf(__uint_as_float(sv[2 * i + 1]), P.scale2, -mref[h]));
          l4[h][0] += p0;
          l4[h][1] += p1;
          sv[i] = pack2<kFp4>(p0, p1);
        }
        lsum[0] += l4[0][0] + l4[0][1];
        lsum[1] += l4[1][0] + l4[1][1];
        if (votes != 0) {
          // rare: scale this warp's dims of O^T by alpha once the previous chunk's products are
          // done. A wait that gives up here shows in the next vote.
          ok = wait_warp(chunk_done(it - 1), ((it - 1) / kBuf) & 1);
          tc_fence_after();
#pragma unroll 1
          for (int cg = 0; cg < 16; ++cg) {  // 4 slices x 4 groups of 16 heads
            uint32_t o[16];
            const uint32_t ta = lane_base + kColO + 16 * cg;
            tmem_ld_x16(ta, o);
            tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < 16; ++h)
              o[h] = __float_as_uint(__uint_as_float(o[h]) * S.alpha[16 * (cg & 3) + h]);
            tmem_st_x16(ta, o);
          }
          tmem_st_wait();
          count_softmax(false);  // alpha has been read
        }
        // (the P buffer was read by the products of chunk it - 2: see S above)
        // K-major tile [head][64 rows]: 8 x 8 pieces of 16-bit values, four a store: column groups
        // 2 c and 2 c + 1 of heads 16w .. 16w + 7 and 16w + 8 .. 16w + 15. Lane l gives the
        // address of row l % 8 of piece l / 8 (heads + 8 in odd pieces).
        {
          const uint32_t pt = smem_u32(base + kOffP + slot * kSlotP);
          const int head = 16 * warp + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            stmatrix_x4(pt + sw128(head, 2 * c + (lane >> 4)), sv[4 * c], sv[4 * c + 1],
                        sv[4 * c + 2], sv[4 * c + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[slot]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], 1);
        lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], 2);
      }
      // ---- epilogue ----
      pdl_wait();  // the rotation, written beside the tiles
      // rotation of dim 32 (warp - 2) + lane of the last half slice
      const float2 rot = warp >= 2 ? P.rope[(size_t)x.bt * 32 + 16 * (warp - 2) + (lane >> 1)]
                                   : make_float2(1.f, 0.f);
      const int h0 = (x.stream - x.bt * P.G) * kHg;
      const bool single = P.nsplit == 1;
      float* pp = P.part + (size_t)x.w * kPartFloats;
      if (quad == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int head = hq + 8 * h;
          if (single) {
            const float zs = a.sink ? a.sink[h0 + head] * 1.44269504088896341f : -INFINITY;
            float f = 0.f;
            if (lsum[h] != 0.f) {  // a NaN stays one
              const float M = fmaxf(mu[h], zs);
              const float e = exp2f(mu[h] - M);
              f = e / (lsum[h] * e + (zs == -INFINITY ? 0.f : exp2f(zs - M)));
            }
            S.fin[head] = f;
          } else {
            pp[head] = mu[h];
            pp[kHg + head] = lsum[h];
          }
        }
      }
      const bool have = ok && wait_warp(chunk_done(it - 1), ((it - 1) / kBuf) & 1);
      ok = have;
      bar_softmax();  // S.fin
      tc_fence_after();
      if (single) {
        // A lane has a dim of every slice, for all heads. Neighbouring lanes trade values, so that
        // the even one has dims d, d + 1 of head h and the odd one those of head h + 1: 64 bytes of
        // a head's row per half warp, straight from registers (through shared memory, in 16-byte
        // pieces, 5071 queries with lists of 3 took 472 instead of 456 us).
        const bool odd = lane & 1;
        uint8_t* out = reinterpret_cast<uint8_t*>(static_cast<__nv_bfloat16*>(a.out) +
                                                  ((size_t)x.bt * a.H + h0 + odd) * kC + 32 * warp +
                                                  (lane & ~1));
#pragma unroll 1
        for (int sl = 0; sl < 4; ++sl, out += 256) {
          uint32_t o[64];
          if (have) {
            tmem_ld_32x32b_x64(lane_base + kColO + 64 * sl, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int h = 0; h < kHg; ++h) o[h] = 0u;
          }
          float* y = reinterpret_cast<float*>(o);
#pragma unroll
          for (int h = 0; h < kHg; h += 4) {
            const float4 f = *reinterpret_cast<const float4*>(S.fin + h);
            y[h] *= f.x;
            y[h + 1] *= f.y;
            y[h + 2] *= f.z;
            y[h + 3] *= f.w;
          }
          if (sl == 3 && warp >= 2) {  // by -t: (u, v) turns to (u c + v s, v c - u s)
            const float sn = odd ? -rot.y : rot.y;
#pragma unroll
            for (int h = 0; h < kHg; ++h)
              y[h] = y[h] * rot.x + __shfl_xor_sync(0xffffffffu, y[h], 1) * sn;
          }
#pragma unroll
          for (int h = 0; h < kHg; h += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? y[h] : y[h + 1], 1);
            *reinterpret_cast<uint32_t*>(out + h * (kC * 2)) =
                odd ? pack2<kBf16>(got, y[h + 1]) : pack2<kBf16>(y[h], got);
          }
        }
        tc_fence_before();
      } else {
        // fp32 O^T [slice][head][128 dims] through the KV buffers, which nothing uses any more,
        // and from there in bulk: 128 KB in 4-byte stores took 2.8 us
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
          float* st = reinterpret_cast<float*>(base + kOffKV) + sl * (kHg * 128) + tid;
#pragma unroll
          for (int h = 0; h < 64; ++h) st[h * 128] = __uint_as_float(o[h]);
          fence_proxy_async_smem();
          bar_softmax();
          if (tid == 32 * sl)
            bulk_store(pp + 2 * kHg + (size_t)sl * (kHg * 128),
                       base + kOffKV + (size_t)sl * (kHg * 128 * 4), kHg * 128 * 4);
        }
        if (lane == 0) bulk_store_wait();
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

// Merge the partials, add the sink, rotate by -t. A warp per (head, 128 dims), four dims a lane:
// lane s has split s's maximum and sum, the loads of sixteen splits go out before anything is
// computed, and no barrier is needed. Every merged value is a sum over the splits in order.
__global__ void __launch_bounds__(256) k_attn_fp4_combine(const __grid_constant__ Params P) {
  const MqaArgs& a = P.a;
  const int lane = threadIdx.x & 31, ns = P.nsplit;
  const uint32_t w = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int stream = (int)(w / (4 * kHg)), h = (int)(w / 4) % kHg, quarter = (int)(w & 3);
  const int bt = stream / P.G, g = stream % P.G;
  const float* base = P.part + (size_t)stream * ns * kPartFloats;
  const float* ob = base + 2 * kHg + quarter * (kHg * 128) + h * 128 + 4 * lane;
  const float zs = a.sink ? a.sink[g * kHg + h] * 1.44269504088896341f : -INFINITY;
  pdl_wait();
  pdl_trigger();
  const float m = lane < ns ? base[(size_t)lane * kPartFloats + h] : -INFINITY;
  const float l = lane < ns ? base[(size_t)lane * kPartFloats + kHg + h] : 0.f;
  constexpr int kBatch = 16;
  float4 v[kBatch];
#pragma unroll
  for (int s = 0; s < kBatch; ++s)
    if (s < ns) v[s] = *reinterpret_cast<const float4*>(ob + (size_t)s * kPartFloats);
  const int d = 128 * quarter + 4 * lane;
  float2 c0 = make_float2(1.f, 0.f), c1 = c0;  // of +t
  if (d >= kNope) {
    c0 = P.rope[(size_t)bt * 32 + ((d - kNope) >> 1)];
    c1 = P.rope[(size_t)bt * 32 + ((d - kNope) >> 1) + 1];
  }
  const float M = fmaxf(warp_max(m), zs);
  const float f = m == -INFINITY ? 0.f : exp2f(m - M);
  float den = warp_sum(f * l);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& x, float fs) {
    o.x = fmaf(x.x, fs, o.x);
    o.y = fmaf(x.y, fs, o.y);
    o.z = fmaf(x.z, fs, o.z);
    o.w = fmaf(x.w, fs, o.w);
  };
#pragma unroll
  for (int s = 0; s < kBatch; ++s)
    if (s < ns) add(v[s], __shfl_sync(0xffffffffu, f, s));
#pragma unroll 4
  for (int s = kBatch; s < ns; ++s)
    add(*reinterpret_cast<const float4*>(ob + (size_t)s * kPartFloats), __shfl_sync(0xffffffffu, f, s));
  float r = 0.f;
  if (den != 0.f) {  // a NaN stays one
    den += zs == -INFINITY ? 0.f : exp2f(zs - M);
    r = 1.f / den;
  }
  o.x *= r, o.y *= r, o.z *= r, o.w *= r;
  __nv_bfloat162 out[2] = {
      __floats2bfloat162_rn(o.x * c0.x + o.y * c0.y, o.y * c0.x - o.x * c0.y),
      __floats2bfloat162_rn(o.z * c1.x + o.w * c1.y, o.w * c1.x - o.z * c1.y)};
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) +
                            ((size_t)bt * a.H + g * kHg + h) * kC + d) = *reinterpret_cast<uint2*>(out);
}

// CTAs per stream: as many as fill the SMs, at most one per chunk of the longest list, at most
// kMaxSplit, and no more than the largest share needs. With one chunk a CTA the partials (128 KB
// each, written and read again, the merge in batches of 16 to a stream) can cost more than a second
// chunk does. One against two chunks a CTA over lists, in us (graph replay, 64 heads):
//   streams x chunks   3 x 26 14.9 / 14.7   3 x 28 14.6 / 14.9   3 x 32 15.2 / 14.9
//                      4 x 18 14.0 / 14.8   4 x 20 13.9 / 14.9   4 x 22 15.4 / 15.0   4 x 32 17.5 / 15.4
//                      5 x 14 13.9 / 14.8   5 x 17 15.5 / 14.7   5 x 24 16.8 / 15.2
//                      6 x 14 14.4 / 15.0   6 x 17 15.7 / 15.3   6 x 24 17.3 / 16.3
//                      8 x 14 15.1 / 15.4   8 x 16 16.1 / 15.6   8 x 18 17.6 / 15.7
//                      1 or 2 x 17 to 32: one is faster by 1 to 0 (60 CTAs and fewer)
// (2 x and 4 x 64 of 128 heads: the same to 0.3.) So two chunks where there are more than 16 one-chunk
// partials to a stream, and CTAs for more than 4/7 of the SMs (84 of 148). With 16 and fewer the two
// lie within 0.5 us of each other up to 120 CTAs.
int choose_split(const MqaArgs& a) {
  const int64_t streams = (int64_t)a.B * a.T * (a.H / kHg);
  const int64_t rows = a.k > 0 ? a.k : a.n_cap;
  const int64_t chunks = (rows + kRows - 1) / kRows + ((int64_t)a.n_win + kRows - 1) / kRows;
  int64_t ns = device_sm_count() / (streams > 0 ? streams : 1);
  ns = ns < chunks ? ns : chunks;
  ns = ns < 1 ? 1 : (ns > kMaxSplit ? kMaxSplit : ns);
  int64_t share = (chunks + ns - 1) / ns;
  if (share == 1 && ns > 16 && 7 * streams * ns > 4 * device_sm_count()) share = 2;
  return share > 0 ? (int)((chunks + share - 1) / share) : 1;
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
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(k_attn_fp4, (int)smem, allowed);
  if (e != cudaSuccess) return e;
  e = launch_q_tiles(a, false, w, w + q_tiles_bytes(a, false), st);
  if (e != cudaSuccess) return e;
  P.items = (int)(streams * P.nsplit);
  const int grid = P.items < device_sm_count() ? P.items : device_sm_count();
  e = launch(true, k_attn_fp4, dim3((unsigned)grid), dim3(kThreads), smem, st, P);
  if (e != cudaSuccess || P.nsplit == 1) return e;
  return launch(true, k_attn_fp4_combine, dim3((unsigned)(streams * kHg / 2)), dim3(256), 0, st, P);
}

cudaError_t attn_fp4_device_error(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, tc::g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(tc::g_device_error, &zero, sizeof(int));
}

}  // namespace csa
