// 8-bit activation checkpoints: bf16 X [m x k] kept for the backward pass as
// int8 codes and one bf16 scale per block of 64 consecutive elements of a row.
//
//   c  = max |x| over the block
//   sc = bf16_rne(c / 127)
//   q  = clamp(rint_even(x / sc), -127, 127)     (sc == 0: q = 0)
//   X^ = bf16_rne(q . sc)
//
// "QLoRA and Quantized Training", The idea: only the adapters hold gradients,
// so the only use a QLoRA layer has for its saved input is dA = U^T X.  The
// rounding |X^ - X| <= sc / 2 (+ bf16 rounding) is at most c / 253 of the
// block's largest element.  An int8 grid keeps an activation block's error
// about four times smaller than E4M3 would (half a step of c/127 everywhere
// against 2^-4 of each element), and a bf16 scale makes X^ one exact product
// and one rounding.
//
// Exactness without a division per element: x and sc are 8-bit significands,
// so x / sc either is a multiple of 1/2 or differs from one by more than
// 2^-17 relative; Markstein's quotient (y = RN(1/sc), q0 = RN(x y),
// rho = fma(-q0, sc, x), q = fma(rho, y, q0)) is the correctly rounded
// one, so rint gives the definition's code, ties included.
//
// Both kernels are bound by HBM: 2 B read and 1.03 B written per element
// (save), the reverse for the restore.  X [8192 x 11008], a second of them on
// end: 49 and 43 us, 5.6 and 6.3 TB/s (0.85 and 0.97 of a copy); the first ones
// take 44 and 43.  Wider pieces in the save (16 elements a thread, so that
// codes leave in 16-byte stores: 45 us against 52 with 8) and narrower ones in
// the restore (one 16-byte store a piece: 43 us against 49 .. 58 with two)
// keep every warp's stores in whole consecutive lines.
#include "act8.cuh"
#include "common.cuh"
#include "internal.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kSaveUnroll = 4;     // pieces in flight per thread (16 elements, 8 elements)
constexpr int kRestoreUnroll = 2;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// The codes of 8 elements from their quotients by the block's scale: rint to
// even by the 1.5 * 2^23 constant, the code is the low byte.
__device__ __forceinline__ uint2 pack_codes(const float (&q)[8]) {
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(__fadd_rn(fminf(fmaxf(q[e], -127.f), 127.f), 12582912.0f));
  return make_uint2(prmt(prmt(b[0], b[1], 0x0040), prmt(b[2], b[3], 0x0040), 0x5410),
                    prmt(prmt(b[4], b[5], 0x0040), prmt(b[6], b[7], 0x0040), 0x5410));
}
__device__ __forceinline__ float element(const uint4 &x, int e) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  return e & 1 ? bf16hi_to_f32(w[e >> 1]) : bf16lo_to_f32(w[e >> 1]);
}
__device__ __forceinline__ uint2 encode8(const uint4 &x, float sc, float y) {
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v = element(x, e), q0 = __fmul_rn(v, y);
    q[e] = __fmaf_rn(__fmaf_rn(-q0, sc, v), y, q0);
  }
  return pack_codes(q);
}
// Blocks so small that the remainder could lose bits below the normal range.
__device__ __noinline__ uint2 encode8_tiny(uint4 x, float sc) {
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = sc > 0.f ? __fdiv_rn(element(x, e), sc) : 0.f;
  return pack_codes(q);
}

// One piece is 16 elements (32 bytes of X, 16 of codes); 4 consecutive lanes
// hold a block.
__global__ void __launch_bounds__(kThreads) act_quantize_kernel(const uint4 *__restrict__ X, int64_t pieces,
                                                                uint4 *__restrict__ codes,
                                                                uint16_t *__restrict__ scale) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kSaveUnroll) + threadIdx.x;
  uint4 v[kSaveUnroll][2];
#pragma unroll
  for (int u = 0; u < kSaveUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    v[u][0] = i < pieces ? __ldg(X + 2 * i) : make_uint4(0u, 0u, 0u, 0u);
    v[u][1] = i < pieces ? __ldg(X + 2 * i + 1) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < kSaveUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    // Magnitudes of bf16 order like their bit patterns.
    uint32_t mx = 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {v[u][h].x, v[u][h].y, v[u][h].z, v[u][h].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = max_u16x2(mx, w[e] & 0x7FFF7FFFu);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) mx = max_u16x2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const uint32_t top = (mx & 0xFFFFu) > (mx >> 16) ? (mx & 0xFFFFu) : (mx >> 16);
    const uint32_t sbits = pack_bf16x2(__fdiv_rn(__uint_as_float(top << 16), 127.0f), 0.f) & 0xFFFFu;
    const float sc = __uint_as_float(sbits << 16);
    const float y = __frcp_rn(sc);
    if (i < pieces) {
      uint2 a = encode8(v[u][0], sc, y), b = encode8(v[u][1], sc, y);
      if (sc < 0x1p-90f) {
        a = encode8_tiny(v[u][0], sc);
        b = encode8_tiny(v[u][1], sc);
      }
      codes[i] = make_uint4(a.x, a.y, b.x, b.y);
      if ((threadIdx.x & 3) == 0) scale[i >> 2] = static_cast<uint16_t>(sbits);
    }
  }
}

// One piece is 8 codes (8 bytes in, 16 bytes of X out); 8 consecutive pieces
// share a block's scale.
__global__ void __launch_bounds__(kThreads) act_dequant_kernel(const uint2 *__restrict__ codes, int64_t pieces,
                                                               const uint16_t *__restrict__ scale,
                                                               uint4 *__restrict__ X) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kRestoreUnroll) + threadIdx.x;
  uint2 v[kRestoreUnroll];
  uint32_t s[kRestoreUnroll];
#pragma unroll
  for (int u = 0; u < kRestoreUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    v[u] = i < pieces ? __ldg(codes + i) : make_uint2(0u, 0u);
    s[u] = i < pieces ? __ldg(scale + (i >> 3)) : 0u;
  }
#pragma unroll
  for (int u = 0; u < kRestoreUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    if (i >= pieces) continue;
    const uint32_t s2 = s[u] * 0x10001u;
    uint4 o;
    act8_decode4(v[u].x, s2, o.x, o.y);
    act8_decode4(v[u].y, s2, o.z, o.w);
    X[i] = o;
  }
}

unsigned blocks_for(int64_t pieces, int unroll) {
  return static_cast<unsigned>((pieces + kThreads * unroll - 1) / (kThreads * unroll));
}

}  // namespace

cudaError_t launch_act_quantize(const uint16_t *X, int64_t numel, int8_t *codes, uint16_t *scale,
                                cudaStream_t stream) {
  const int64_t pieces = numel / 16;
  if (pieces <= 0) return cudaSuccess;
  act_quantize_kernel<<<blocks_for(pieces, kSaveUnroll), kThreads, 0, stream>>>(
      reinterpret_cast<const uint4 *>(X), pieces, reinterpret_cast<uint4 *>(codes), scale);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_act_dequant(const int8_t *codes, const uint16_t *scale, int64_t numel, uint16_t *X,
                               cudaStream_t stream) {
  const int64_t pieces = numel / 8;
  if (pieces <= 0) return cudaSuccess;
  act_dequant_kernel<<<blocks_for(pieces, kRestoreUnroll), kThreads, 0, stream>>>(
      reinterpret_cast<const uint2 *>(codes), pieces, scale, reinterpret_cast<uint4 *>(X));
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace qlora
