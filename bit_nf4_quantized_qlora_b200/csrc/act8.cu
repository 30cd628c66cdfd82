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
// (save), the reverse for the restore.
#include "act8.cuh"
#include "common.cuh"
#include "internal.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;        // 16-byte pieces in flight per thread

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// One piece is 8 elements (16 bytes of X); 8 consecutive lanes hold a block.
__global__ void __launch_bounds__(kThreads) act_quantize_kernel(const uint4 *__restrict__ X, int64_t pieces,
                                                                uint2 *__restrict__ codes,
                                                                uint16_t *__restrict__ scale) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint4 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    v[u] = i < pieces ? __ldg(X + i) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    // Magnitudes of bf16 order like their bit patterns.
    uint32_t mx = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = max_u16x2(mx, w[e] & 0x7FFF7FFFu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) mx = max_u16x2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const uint32_t top = (mx & 0xFFFFu) > (mx >> 16) ? (mx & 0xFFFFu) : (mx >> 16);
    const uint32_t sbits = pack_bf16x2(__fdiv_rn(__uint_as_float(top << 16), 127.0f), 0.f) & 0xFFFFu;
    const float sc = __uint_as_float(sbits << 16);
    float q[8];
    if (sc >= 0x1p-90f) {
      const float y = __frcp_rn(sc);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = e & 1 ? bf16hi_to_f32(w[e >> 1]) : bf16lo_to_f32(w[e >> 1]);
        const float q0 = __fmul_rn(x, y);
        q[e] = __fmaf_rn(__fmaf_rn(-q0, sc, x), y, q0);
      }
    } else {
      // Tiny blocks: the remainder could lose bits below the normal range.
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = e & 1 ? bf16hi_to_f32(w[e >> 1]) : bf16lo_to_f32(w[e >> 1]);
        q[e] = sc > 0.f ? __fdiv_rn(x, sc) : 0.f;
      }
    }
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // rint to even by the 1.5 * 2^23 constant: the code is the low byte.
      const float c = fminf(fmaxf(q[e], -127.f), 127.f);
      b[e] = __float_as_uint(__fadd_rn(c, 12582912.0f));
    }
    if (i < pieces) {
      uint2 o;
      o.x = prmt(prmt(b[0], b[1], 0x0040), prmt(b[2], b[3], 0x0040), 0x5410);
      o.y = prmt(prmt(b[4], b[5], 0x0040), prmt(b[6], b[7], 0x0040), 0x5410);
      codes[i] = o;
      if ((threadIdx.x & 7) == 0) scale[i >> 3] = static_cast<uint16_t>(sbits);
    }
  }
}

// One piece is 16 codes; four consecutive pieces share a block's scale.
__global__ void __launch_bounds__(kThreads) act_dequant_kernel(const uint4 *__restrict__ codes, int64_t pieces,
                                                               const uint16_t *__restrict__ scale,
                                                               uint4 *__restrict__ X) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint4 v[kUnroll];
  uint32_t s[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    v[u] = i < pieces ? __ldg(codes + i) : make_uint4(0u, 0u, 0u, 0u);
    s[u] = i < pieces ? __ldg(scale + (i >> 2)) : 0u;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    if (i >= pieces) continue;
    const uint32_t s2 = s[u] * 0x10001u;
    uint4 o[2];
    act8_decode4(v[u].x, s2, o[0].x, o[0].y);
    act8_decode4(v[u].y, s2, o[0].z, o[0].w);
    act8_decode4(v[u].z, s2, o[1].x, o[1].y);
    act8_decode4(v[u].w, s2, o[1].z, o[1].w);
    X[2 * i] = o[0];
    X[2 * i + 1] = o[1];
  }
}

unsigned blocks_for(int64_t pieces) {
  return static_cast<unsigned>((pieces + kThreads * kUnroll - 1) / (kThreads * kUnroll));
}

}  // namespace

cudaError_t launch_act_quantize(const uint16_t *X, int64_t numel, int8_t *codes, uint16_t *scale,
                                cudaStream_t stream) {
  const int64_t pieces = numel / 8;
  if (pieces <= 0) return cudaSuccess;
  act_quantize_kernel<<<blocks_for(pieces), kThreads, 0, stream>>>(
      reinterpret_cast<const uint4 *>(X), pieces, reinterpret_cast<uint2 *>(codes), scale);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_act_dequant(const int8_t *codes, const uint16_t *scale, int64_t numel, uint16_t *X,
                               cudaStream_t stream) {
  const int64_t pieces = numel / 16;
  if (pieces <= 0) return cudaSuccess;
  act_dequant_kernel<<<blocks_for(pieces), kThreads, 0, stream>>>(reinterpret_cast<const uint4 *>(codes), pieces,
                                                                  scale, reinterpret_cast<uint4 *>(X));
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace qlora
