// Building blocks of the kernels that stream a query's KV rows through the tensor cores in
// chunks of 64 rows (attn_fp4.cu, attn_mass.cu): the row list of a query, the warp that
// resolves a chunk's rows to addresses, the nine warps that bring one 64-value atom of every
// row each into 128B-swizzled shared memory (widening 4-bit rows on the way). The query
// operand comes as a tile that q_tiles.cu prepared.
//
// A 4-bit cache row (CSA_MIXED_MXFP4_BF16, c = 512, r = 64) is 368 bytes:
//   bytes   0-223  448 e2m1 codes, element 2j in the low nibble of byte j
//   bytes 224-239  14 e8m0 exponents (one per 32 values), then 2 zero bytes
//   bytes 240-367  the 64 RoPE values, bf16
// Its operands are f16. An e2m1 value times 2^E with E in [-14, 13] (the writers clamp E to
// that range) is an f16 number, and so is every bf16 value of magnitude 2^-14 .. 65504, so
// widening a row rounds nothing (smaller RoPE or window values keep an absolute step of
// 2^-24); q_hat and P carry 11 bits where bf16 operands would carry 8.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace csa {
namespace rows {

using namespace tc;

constexpr int kC = 512, kR = 64, kNope = kC - kR;
constexpr int kHg = 64;            // heads of a CTA
constexpr int kRows = 64;          // rows of a chunk
constexpr int kAtoms = kC / 64;    // 64-value (128 B) atoms of a row
constexpr int kAtomBytes = kRows * 128;
constexpr int kFp4RowBytes = 368, kFp4Exps = 224, kFp4Rope = 240;
constexpr int kRing = 4;           // chunks of resolved addresses

enum Fmt { kFp4 = 0, kBf16 = 1 };

// One lane of a converged warp. Unlike a test of the lane number it leaves the operands of the
// MMAs behind it warp-uniform: an MMA of 64 x 64 x 16 then issues in its 32 cycles, not in 46
// (measured).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t chunk) {
  return row * 128u + ((chunk ^ (row & 7u)) << 4);
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The rows of a query: cache chunks (selected or visible entries), then window chunks. Each
// kind starts a chunk of its own, so every row of a chunk has one storage format.
struct List {
  int64_t t, lo;
  uint32_t n_vis, n_sel, n_w;
  int nc, n_chunks;
};

__device__ __forceinline__ List make_list(const MqaArgs& a, int64_t t) {
  List l;
  l.t = t;
  l.n_vis = 0;
  if (t >= 0) {
    const int64_t e = t <= 0x7fffffff ? (int64_t)((uint32_t)t / (uint32_t)a.m) : t / a.m;
    l.n_vis = (uint32_t)(e < a.n_cap ? e : a.n_cap);
  }
  l.n_sel = a.k > 0 ? (uint32_t)a.k : l.n_vis;
  l.lo = (t - a.n_win + 1) > 0 ? (t - a.n_win + 1) : 0;
  l.n_w = (a.n_win > 0 && t >= 0) ? (uint32_t)(t - l.lo + 1) : 0u;
  l.nc = (int)((l.n_sel + (kRows - 1)) / kRows);
  l.n_chunks = l.nc + (int)((l.n_w + (kRows - 1)) / kRows);
  return l;
}

// A work item: the chunks [c0, c1) of split `split` of stream (query, 64 heads) `stream`.
struct Item {
  int stream, split, bt, b, c0, c1;
  List l;
  __device__ __forceinline__ void set(const MqaArgs& a, int w, int G, int nsplit, int64_t t) {
    stream = (int)((uint32_t)w / (uint32_t)nsplit);
    split = w - stream * nsplit;
    bt = (int)((uint32_t)stream / (uint32_t)G);
    b = (int)((uint32_t)bt / (uint32_t)a.T);
    l = make_list(a, t);
    const int each = (int)((uint32_t)l.n_chunks / (uint32_t)nsplit), more = l.n_chunks - each * nsplit;
    c0 = each * split + min(split, more);
    c1 = c0 + each + (split < more ? 1 : 0);
  }
};
__device__ __forceinline__ int64_t item_pos(const MqaArgs& a, int w, int G, int nsplit) {
  return a.q_pos[(uint32_t)w / ((uint32_t)nsplit * (uint32_t)G)];
}

// What a masked row is read from: zero codes and zero bf16 values, so that the gather's loads
// need no predicate.
static __device__ __align__(16) uint8_t g_zero_row[kC * 2];

// Resolved addresses of kRing chunks (masked rows: g_zero_row), their masks of valid rows and
// what they hold.
enum Kind : uint32_t { kWindow = 0, kCache = 1, kEnd = 2 };  // kEnd: no further chunk
struct AddrRing {
  uint64_t src[kRing][kRows];
  uint32_t mask[kRing][2], kind[kRing];
  uint64_t full[kRing], free[kRing];
};

// The entries of kRing chunks and their pages, one row of each half chunk per lane: the two
// dependent round trips (index list, page table) are shared by four chunks.
struct RowBatch {
  uint32_t r[kRing][2];  // row within its page
  int32_t pg[kRing][2];  // page; kEvicted: no row
  __device__ __forceinline__ void lookup(const MqaArgs& a, const Item& x, int j0) {
    const int lane = threadIdx.x & 31;
    int e[kRing][2];
#pragma unroll
    for (int i = 0; i < kRing; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t s = (uint32_t)(j0 + i) * kRows + 32 * h + lane;
        e[i][h] = -1;
        if (j0 + i < x.c1 && s < x.l.n_sel) e[i][h] = a.k > 0 ? a.idx[(size_t)x.bt * a.k + s] : (int)s;
      }
#pragma unroll
    for (int i = 0; i < kRing; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        pg[i][h] = kEvicted;
        if (e[i][h] >= 0 && e[i][h] < a.n_cap) {
          const uint32_t lp = (uint32_t)e[i][h] / (uint32_t)a.page_rows;
          r[i][h] = (uint32_t)e[i][h] - lp * (uint32_t)a.page_rows;
          pg[i][h] = a.page_table[(size_t)x.b * a.max_pages + lp];
        }
      }
  }
};

// The address warp: the chunks of item x, the first batch already looked up; `it` counts the
// CTA's chunks. `code`: error code of a wait that gave up; code + 5: a page id outside the pool
// (an evicted page is masked quietly). begin() is called where the item's first chunk has its
// place in the ring.
template <int kFmt, class Begin>
__device__ __forceinline__ bool resolve_rows(RowBatch& rb, const MqaArgs& a, const Item& x,
                                             uint32_t& it, AddrRing& ring, int code, Begin begin) {
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kRowBytes = kFmt == kFp4 ? kFp4RowBytes : kC * 2;
  const uint64_t zero_row = reinterpret_cast<uint64_t>(g_zero_row);
  for (int j0 = x.c0; j0 < x.c1; j0 += kRing) {
    if (j0 > x.c0) rb.lookup(a, x, j0);
    const int n = min(kRing, x.c1 - j0);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int j = j0 + i;
      uint64_t src[2] = {0, 0};
      if (j < x.l.nc) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int32_t p = rb.pg[0][h];
          if (p >= 0 && p < a.n_pages)
            src[h] = reinterpret_cast<uint64_t>(a.kv) +
                     ((uint64_t)(uint32_t)p * (uint32_t)a.page_rows + rb.r[0][h]) * kRowBytes;
          else if (p != kEvicted)
            set_error(code + 5);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t s = (uint32_t)(j - x.l.nc) * kRows + 32 * h + lane;
          if (s < x.l.n_w) {
            const int64_t pos = x.l.lo + s;
            // win_pos0 == nullptr: the state cache's ring (position p in row p mod l_raw)
            const int64_t rr = a.win_pos0 != nullptr ? pos - a.win_pos0[x.b]
                               : pos <= 0x7fffffff   ? (int64_t)((uint32_t)pos % (uint32_t)a.l_raw)
                                                     : pos % a.l_raw;
            if (rr >= 0 && rr < a.l_raw)
              src[h] = reinterpret_cast<uint64_t>(a.win) + ((uint64_t)x.b * a.l_raw + rr) * (kC * 2);
          }
        }
      }
#pragma unroll
      for (int k = 0; k + 1 < kRing; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          rb.pg[k][h] = rb.pg[k + 1][h];
          rb.r[k][h] = rb.r[k + 1][h];
        }
      const uint32_t rs = it % kRing;
      if (!__all_sync(0xffffffffu, mbar_wait(&ring.free[rs], ((it / kRing) & 1) ^ 1, code)))
        return false;
      if (j == x.c0) begin();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ring.src[rs][32 * h + lane] = src[h] != 0 ? src[h] : zero_row;
        const uint32_t m = __ballot_sync(0xffffffffu, src[h] != 0);
        if (lane == 0) ring.mask[rs][h] = m;
      }
      if (lane == 0) ring.kind[rs] = j < x.l.nc ? kCache : kWindow;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.full[rs]);
      // towards L2 while the gather warps are still chunks behind; one instruction serves 32
      // rows (the bulk form, one row each, took 80 cycles a row). A line per 128 bytes from the row's
      // start: a 368-byte row that reaches into a fourth line fetches that one with the gather.
      if (j > x.c0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (src[h] != 0) {
            const uint32_t bytes = j < x.l.nc ? kRowBytes : kC * 2;
            for (uint32_t o = 0; o < bytes; o += 128)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(src[h] + o));
          }
      }
      ++it;
    }
  }
  return true;
}

// After the last item: tells the gather warps to stop.
template <class Begin>
__device__ __forceinline__ void resolve_end(uint32_t it, AddrRing& ring, int code, Begin begin) {
  const uint32_t rs = it % kRing;
  if (!__all_sync(0xffffffffu, mbar_wait(&ring.free[rs], ((it / kRing) & 1) ^ 1, code))) return;
  begin();
  if ((threadIdx.x & 31) == 0) {
    ring.kind[rs] = kEnd;
    mbar_arrive(&ring.full[rs]);
  }
}

// Eight e2m1 codes (a 32-bit word, element 0 in the low nibble) times the f16x2 scale.
__device__ __forceinline__ uint4 widen8(uint32_t w, __half2 scale) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), scale);
    h[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// 2^E of an exponent byte as f16x2. The format holds E to [-14, 13]; the five bits of E + 15 are
// all that is used of any other byte.
__device__ __forceinline__ __half2 scale_h2(uint32_t ex) {
  const uint32_t u = ((ex - 112u) & 31u) * 0x04000400u;
  return *reinterpret_cast<const __half2*>(&u);
}

// Two bf16 values to f16 (exact for magnitudes 2^-14 .. 65504; larger ones become infinite).
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  const __half2 h = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The gather warps: nine, warps 0-6 one atom (64 values) of all 64 rows each, warps 7 and 8 the
// last atom of 32 rows each (bf16 in either format, twice the bytes of a 4-bit atom). A warp's
// share is held in registers between the loads and the stores.
// Codes: lane -> 16-byte unit lane % 2 (one exponent block) of rows lane / 2 + 16 i, four units
// a lane; the four 16-byte stores of eight neighbouring lanes fall into distinct banks. bf16
// values: unit lane % 8 of rows first + lane / 8 + 4 i, eight a lane per 32 rows.
// The loops over a lane's units are rolled, the held values moving down through the registers:
// sixteen warps of six kinds share the instruction caches, and with everything unrolled a
// quarter more time went into waiting for instructions.
constexpr int kGatherWarps = 9;

__device__ __forceinline__ void st_shared(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

struct Codes {
  uint4 raw[4];
  uint32_t ex[4];
  // off: the lane's byte offset in a row's codes; exo: its exponent's
  __device__ __forceinline__ void load(const uint64_t* src, int off, int exo) {
    const uint64_t* p = src + ((threadIdx.x & 31) >> 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* row = reinterpret_cast<const uint8_t*>(p[16 * i]);
      raw[i] = __ldg(reinterpret_cast<const uint4*>(row + off));
      ex[i] = __ldg(row + exo);
    }
  }
  // at: the lane's first row in the atom; sw: its swizzled 16-byte pieces
  __device__ __forceinline__ void store(uint32_t at, const uint32_t (&sw)[4]) {
#pragma unroll 2
    for (int i = 0; i < 4; ++i, at += 16 * 128) {
      const __half2 s = scale_h2(ex[0]);
      const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) st_shared(at + sw[k], widen8(w[k], s));
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        raw[k] = raw[k + 1];
        ex[k] = ex[k + 1];
      }
    }
  }
};

template <int kFmt>
struct Halves {  // bf16 values of rows first .. first + 31
  uint4 raw[8];
  __device__ __forceinline__ void load(const uint64_t* src, int offset, int first) {
    const int lane = threadIdx.x & 31;
    const uint64_t* p = src + first + (lane >> 3);
    const uint32_t off = offset + 16 * (lane & 7);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      raw[i] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p[4 * i]) + off));
  }
  __device__ __forceinline__ void store(uint32_t atom, int first) {
    const int lane = threadIdx.x & 31;
    const uint32_t r0 = first + (lane >> 3), c = lane & 7;
    // rows r0 + 4 i: even i share a swizzle, and so do odd ones
    uint32_t at = atom + r0 * 128;
    const uint32_t sw0 = (c ^ (r0 & 7)) << 4, sw1 = 512 + ((c ^ ((r0 + 4) & 7)) << 4);
#pragma unroll 1
    for (int i = 0; i < 8; i += 2, at += 1024) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint4 o = raw[k];
        if constexpr (kFmt == kFp4)
          o = make_uint4(bf16x2_to_f16x2(o.x), bf16x2_to_f16x2(o.y), bf16x2_to_f16x2(o.z),
                         bf16x2_to_f16x2(o.w));
        st_shared(at + (k ? sw1 : sw0), o);
      }
#pragma unroll
      for (int k = 0; k < 6; ++k) raw[k] = raw[k + 2];
    }
  }
};

// Two fp32 values to 16-bit operands (f16 for 4-bit caches, else bf16).
template <int kFmt>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kFmt == kFp4) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <int kFmt>
__device__ __forceinline__ float unpack_lo(uint32_t w) {
  if constexpr (kFmt == kFp4) return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
  else return __uint_as_float(w << 16);
}
template <int kFmt>
__device__ __forceinline__ float unpack_hi(uint32_t w) {
  if constexpr (kFmt == kFp4) return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  else return __uint_as_float(w & 0xffff0000u);
}

// `bytes` bytes (a multiple of 16) of device memory into shared memory, both 16-byte aligned;
// and back, in this thread's bulk group.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void bulk_prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(src)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_store_wait_read() {  // the shared memory may be rewritten
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// One gather warp's loop over the CTA's chunks: kBufs KV buffers of kAtoms atoms at `kv`, kFull
// full barriers per buffer (1: an arrival per gather warp; kAtoms: one per atom, two for the
// last) and kFree free barriers, each for kAtoms / kFree atoms. The next chunk's loads are issued
// once this one is stored, and are in flight until its buffer is given back.
template <int kFmt, int kBufs, int kFull, int kFree>
__device__ __forceinline__ void gather_loop(uint8_t* kv, int gw, AddrRing& ring, uint64_t* full,
                                            uint64_t* free, int code) {
  const int lane = threadIdx.x & 31;
  const int atom = gw < kAtoms - 1 ? gw : kAtoms - 1;
  const bool last = atom == kAtoms - 1;
  const int first = gw == kGatherWarps - 1 ? 32 : 0;  // of a warp of the last atom
  auto wait = [&](uint64_t* bar, uint32_t parity, int c) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, c));
  };
  auto address = [&](uint32_t it) {  // the chunk's kind, or kEnd
    return wait(&ring.full[it % kRing], (it / kRing) & 1, code) ? ring.kind[it % kRing]
                                                                : (uint32_t)kEnd;
  };
  auto read = [&](uint32_t it) {  // this warp has read the chunk's addresses
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.free[it % kRing]);
  };
  const uint32_t kv0 = smem_u32(kv) + atom * kAtomBytes;
  auto dst_of = [&](uint32_t it) { return kv0 + (it % kBufs) * (kAtoms * kAtomBytes); };
  auto buffer = [&](uint32_t it) {
    return wait(&free[(it % kBufs) * kFree + atom / (kAtoms / kFree)], ((it / kBufs) & 1) ^ 1,
                code + 1);
  };
  auto publish = [&](uint32_t it) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[(it % kBufs) * kFull + atom / (kAtoms / kFull)]);
  };
  uint32_t it = 0, kind = address(0);
  if (kFmt == kFp4 && !last) {
    Codes v;
    const int u = lane & 1, r = lane >> 1, off = 32 * atom + 16 * u, exo = kFp4Exps + 2 * atom + u;
    uint32_t sw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sw[k] = r * 128 + (((4 * u + k) ^ (r & 7)) << 4);
    if (kind == kCache) {
      v.load(ring.src[0], off, exo);
      read(0);
    }
    while (kind != kEnd) {
      if (kind == kCache) {
        if (!buffer(it)) return;
        v.store(dst_of(it), sw);
        publish(it);
      } else {  // window rows, in two halves
        Halves<kFmt> h0, h1;
        h0.load(ring.src[it % kRing], 128 * atom, 0);
        h1.load(ring.src[it % kRing], 128 * atom, 32);
        read(it);
        if (!buffer(it)) return;
        h0.store(dst_of(it), 0);
        h1.store(dst_of(it), 32);
        publish(it);
      }
      kind = address(++it);
      if (kind == kCache) {
        v.load(ring.src[it % kRing], off, exo);
        read(it);
      }
    }
  } else if (last) {
    Halves<kFmt> v;
    auto offset = [&](uint32_t k) { return kFmt == kFp4 && k == kCache ? kFp4Rope : 128 * atom; };
    if (kind != kEnd) {
      v.load(ring.src[0], offset(kind), first);
      read(0);
    }
    while (kind != kEnd) {
      if (!buffer(it)) return;
      v.store(dst_of(it), first);
      publish(it);
      kind = address(++it);
      if (kind != kEnd) {
        v.load(ring.src[it % kRing], offset(kind), first);
        read(it);
      }
    }
  } else {  // bf16 rows: both halves, one chunk at a time
    for (; kind != kEnd; kind = address(++it)) {
      Halves<kFmt> h0, h1;
      h0.load(ring.src[it % kRing], 128 * atom, 0);
      h1.load(ring.src[it % kRing], 128 * atom, 32);
      read(it);
      if (!buffer(it)) return;
      h0.store(dst_of(it), 0);
      h1.store(dst_of(it), 32);
      publish(it);
    }
  }
}

}  // namespace rows
}  // namespace csa
