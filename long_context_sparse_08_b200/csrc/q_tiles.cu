// q_hat = RoPE_t(RMSNorm(q) * w) (【论文解读】DeepSeek-V4 一(三)3(1), 3(2)) as operand tiles of the
// kernels that read rows through kv_rows.cuh: per (query, 64 heads) the 128B-swizzled image of
// the A operand in shared memory, [atom of 64 values][row][128 bytes], so that one bulk copy
// brings it there. Forms: 64 f16 rows (attention), or 128 rows with two 16-bit parts hi + lo of
// each head, head 16 w + i in rows 32 w + i and 32 w + 16 + i (attention weight; f16 or bf16).
// Also the cos / sin of the query positions, for the rotation by -t of the output.
//
// A kernel of its own: a stream's splits (up to 32 CTAs) would each repeat this work, and its
// code (a double-precision angle, 130 instructions a head) took 5 us at the start of every
// attention CTA, more than this launch, which overlaps the look-up and the gather of the
// first rows (programmatic launch). A warp per head; bound by latency for a decode batch and
// by HBM (1 KB in, 1 or 2 KB out per head) for a prefill chunk: 2048 queries x 64 heads take 47 us
// (268 MB, 5.7 TB/s), a decode batch 2.6 us of which 1.5 overlap the attention's start.
#include "common.cuh"
#include "internal.h"
#include "kv_rows.cuh"

namespace csa {

namespace {

using namespace rows;

struct QParams {
  MqaArgs a;
  uint8_t* tiles;
  float2* rope;  // [B * T][32]
  double inv_freq[kR / 2];
};

// kSplit: hi + lo parts. kPer: heads per warp (one after another).
template <int kFmt, bool kSplit, int kPer>
__global__ void __launch_bounds__(256) k_q_tiles(const __grid_constant__ QParams P) {
  const MqaArgs& a = P.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t gh0 = ((int64_t)blockIdx.x * 8 + warp) * kPer;  // head of all B * T * H
  const int64_t bt = gh0 / a.H;
  pdl_wait();
  pdl_trigger();
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + gh0 * kC);
  // (plain loads: q may be the work of the launch before, beside whose end this kernel starts, and
  // the read-only path is for data that no one writes while the kernel runs)
  uint4 raw[2] = {src[lane], src[lane + 32]};
  float w[16];
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w[8 * half + k] = a.q_rms_w ? __bfloat162float(static_cast<const __nv_bfloat16*>(
                                        a.q_rms_w)[256 * half + 8 * lane + k])
                                  : 1.f;
  // pair `lane`'s angle; lanes 24-31 turn pairs 4 (lane - 24) ..
  float cs1, sn1, cs[4], sn[4];
  rope_angle_cs((double)a.q_pos[bt], P.inv_freq[lane], &cs1, &sn1);
  if (gh0 % a.H == 0) P.rope[bt * 32 + lane] = make_float2(cs1, sn1);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int from = (4 * (lane - 24) + k) & 31;
    cs[k] = __shfl_sync(0xffffffffu, cs1, from);
    sn[k] = __shfl_sync(0xffffffffu, sn1, from);
  }
#pragma unroll 1
  for (int i = 0; i < kPer; ++i) {
    const uint4 cur[2] = {raw[0], raw[1]};
    if (i + 1 < kPer) {
      raw[0] = src[(i + 1) * (kC / 8) + lane];
      raw[1] = src[(i + 1) * (kC / 8) + lane + 32];
    }
    float y[16], ss = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t w4[4] = {cur[half].x, cur[half].y, cur[half].z, cur[half].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float lo = __uint_as_float(w4[k] << 16), hi = __uint_as_float(w4[k] & 0xffff0000u);
        y[8 * half + 2 * k] = lo;
        y[8 * half + 2 * k + 1] = hi;
        ss = fmaf(lo, lo, ss);
        ss = fmaf(hi, hi, ss);
      }
    }
    const float rstd = 1.f / sqrtf(warp_sum(ss) * (1.f / (float)kC) + a.eps);
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] = y[k] * rstd * w[k];
    if (lane >= 24) {  // dims 256 + 8 lane >= 448
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float u = y[8 + 2 * k], v = y[9 + 2 * k];
        y[8 + 2 * k] = u * cs[k] - v * sn[k];
        y[9 + 2 * k] = u * sn[k] + v * cs[k];
      }
    }
    const int64_t gh = gh0 + i;
    const int head = (int)(gh % kHg);
    constexpr int kTileRows = kSplit ? 2 * kHg : kHg, kAtom = kTileRows * 128;
    uint8_t* tile = P.tiles + (gh / kHg) * (int64_t)(kAtoms * kAtom);
    const int row = kSplit ? 32 * (head / 16) + head % 16 : head;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float u = y[8 * half + 2 * k], v = y[8 * half + 2 * k + 1];
        hi[k] = pack2<kFmt>(u, v);
        if (kSplit) lo[k] = pack2<kFmt>(u - unpack_lo<kFmt>(hi[k]), v - unpack_hi<kFmt>(hi[k]));
      }
      const int c = lane + 32 * half;  // 16-byte piece of the row
      uint8_t* at = tile + (c >> 3) * kAtom;
      *reinterpret_cast<uint4*>(at + sw128(row, c & 7)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (kSplit)
        *reinterpret_cast<uint4*>(at + sw128(row + 16, c & 7)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
}

}  // namespace

size_t q_tiles_bytes(const MqaArgs& a, bool split) {
  return (size_t)a.B * a.T * a.H * (split ? 2048 : 1024);
}
size_t q_rope_bytes(const MqaArgs& a) { return ((size_t)a.B * a.T * 256 + 255) / 256 * 256; }

cudaError_t launch_q_tiles(const MqaArgs& a, bool split, void* tiles, void* rope, cudaStream_t st) {
  QParams P;
  P.a = a;
  P.tiles = static_cast<uint8_t*>(tiles);
  P.rope = static_cast<float2*>(rope);
  for (int p = 0; p < kR / 2; ++p) P.inv_freq[p] = rope_inv_freq(p, kR, (double)a.rope_base);
  const int64_t heads = (int64_t)a.B * a.T * a.H;
  // eight heads a warp once that still gives every SM several blocks (the angle is then worked
  // out once for eight heads), one head a warp for a decode batch
  const int per = heads >= 8 * 8 * 1024 ? 8 : 1;
  auto kern = !split ? (per == 8 ? k_q_tiles<kFp4, false, 8> : k_q_tiles<kFp4, false, 1>)
              : a.fp4 ? (per == 8 ? k_q_tiles<kFp4, true, 8> : k_q_tiles<kFp4, true, 1>)
                      : (per == 8 ? k_q_tiles<kBf16, true, 8> : k_q_tiles<kBf16, true, 1>);
  // It touches nothing before its own wait, so it may start behind any unfinished kernel, and a
  // decode call after another then takes 1.5 to 2.5 us less (14.4 -> 12.7 us, 30.0 -> 27.1 us); a
  // long one, whose early blocks take the places that its own attention waits for, takes more
  // (2048 queries 338 -> 352 us).
  return launch(a.chained || per == 1, kern, dim3((unsigned)(heads / (8 * per))), dim3(256), 0, st, P);
}

}  // namespace csa
