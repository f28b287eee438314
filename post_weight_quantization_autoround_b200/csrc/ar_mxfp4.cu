// MXFP4 fake quantization (QDQ) of a bf16 matrix, its straight-through backward
// (alone, or with the SignSGD update of a tuning step), and the expansion of
// packed weights to bf16.
//
// A further data type enters the tuning through its tensor-level QDQ function
// ([AR] §4 "Why the Tuning Stage Must Take the QDQ Path", point 3; [AR] =
// "Low-Bit Quantization in Practice with vLLM: Core Mechanisms and Architectural
// Optimizations of AutoRound").  The format is the OCP microscaling one: E2M1
// values (1 sign, 2 exponent, 1 mantissa bits; largest 6) with one power-of-two
// scale (E8M0: the code is the exponent + 127) per block of 32 values.  Per block
// b along K, with amax_b = max |W|:
//   X_b = 2^(floor(log2(alpha_b amax_b)) - 2), at least 2^-127
//   q = E2M1(W / X_b + V),  W_hat = q X_b      (0 for a block of zeros)
// Everything is decided on exact values although the arithmetic is fp32:
//  * W / X_b is a bf16 times a power of two, exact;
//  * floor(log2(alpha amax)) is the exponent of the product truncated toward
//    zero, which no rounding can carry past a power of two;
//  * W / X_b + V is rounded to odd: of the sums rounded down and up, the one
//    whose last bit is set (the same number when the sum is exact).  A number
//    rounded to odd at 24 bits rounds on to the two significant bits of E2M1,
//    ties to even, as the exact sum does, and lies above 6 exactly when it does.
//
// All kernels stream at memory speed: a lane holds 8 consecutive values (16 bytes
// of bf16), the 4 lanes of a block combine maxima and sums with two shuffles, and
// every load of a thread's two chunks is issued before the first is used.
// Measured: 8192 x 28672 with V and alpha given, W_hat, codes and scales written (8.66
// bytes a weight): 321 us, 6.3 TB/s; the gradient of 4096 x 4096 (14.25 bytes): 39 us,
// 6.1 TB/s.  A copy of a large tensor runs at 6.4 TB/s on the same GPU.
#include "ar_internal.h"

namespace ar {
namespace {

constexpr int kMxBlock = 32;
constexpr int kMxThreads = 256;
constexpr int kMxChunks = 2;  // chunks of 8 values per thread, one block of threads apart
constexpr float kE2M1Max = 6.0f;

__device__ __forceinline__ uint32_t mx_max_mag8(const uint4& v) {
  uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

// E8M0 code of a block's scale from the bf16 bits of its largest magnitude; 255
// (NaN) when that or alpha is not finite.
__device__ __forceinline__ int mx_scale_code(uint32_t max_bits, float alpha) {
  const float top = __fmul_rz(alpha, __uint_as_float(max_bits << 16));
  const int biased = static_cast<int>((__float_as_uint(top) >> 23) & 0xFFu);
  // truncation cannot make an infinity, so the product alone does not show one
  if (max_bits >= 0x7F80u || !(fabsf(alpha) <= 3.4028235e38f)) return 255;
  return top > 0.0f ? max(biased - 2, 0) : 0;
}

__device__ __forceinline__ float mx_pow2(int code) {  // 2^(code - 127), code 0..254
  return __uint_as_float(code > 0 ? static_cast<uint32_t>(code) << 23 : 0x00400000u);
}

// a + b rounded to odd
__device__ __forceinline__ float add_odd(float a, float b) {
  const float lo = __fadd_rd(a, b), hi = __fadd_ru(a, b);
  return (__float_as_uint(lo) & 1u) ? lo : hi;
}

// what one lane knows of its 8 values
struct MxLane {
  int code;        // E8M0 code of the block
  bool zero, bad;  // block of zeros; not finite
  float X, inv;    // scale and its reciprocal
};

__device__ __forceinline__ MxLane mx_lane(const uint4& w, float alpha) {
  uint32_t m = mx_max_mag8(w);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  MxLane l;
  l.code = mx_scale_code(m, alpha);
  l.zero = m == 0;
  l.bad = l.code == 255;
  const int c = l.bad ? 127 : l.code;
  l.X = mx_pow2(c);
  l.inv = __uint_as_float(static_cast<uint32_t>(254 - c) << 23);  // 2^(127 - c): c <= 252 here, so never zero
  return l;
}

__device__ __forceinline__ void mx_unpack(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}

// two values -> E2M1 pair (low nibble a) and back to floats
__device__ __forceinline__ uint32_t e2m1_pair(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %2, %1;\n\tcvt.u32.u8 %0, q;\n\t}" : "=r"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 e2m1_values(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 q;\n\tcvt.u8.u32 q, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, q;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__global__ void __launch_bounds__(kMxThreads) qdq_mxfp4_kernel(const uint16_t* __restrict__ W,
                                                               const float* __restrict__ V,
                                                               const float* __restrict__ alpha, int64_t n,
                                                               uint16_t* __restrict__ W_hat,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  const int64_t base = (blockIdx.x * static_cast<int64_t>(kMxThreads * kMxChunks) + threadIdx.x) * 8;
  uint4 w[kMxChunks];
  float4 v[kMxChunks][2];
  float a[kMxChunks];
#pragma unroll
  for (int c = 0; c < kMxChunks; ++c) {
    const int64_t e0 = base + c * kMxThreads * 8;
    const bool live = e0 < n;  // n is a multiple of 32: a block is all in or all out
    w[c] = make_uint4(0u, 0u, 0u, 0u);
    v[c][0] = v[c][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    a[c] = 1.0f;
    if (live) {
      w[c] = __ldcs(reinterpret_cast<const uint4*>(W + e0));
      if (V) {
        v[c][0] = __ldcs(reinterpret_cast<const float4*>(V + e0));
        v[c][1] = __ldcs(reinterpret_cast<const float4*>(V + e0 + 4));
      }
      if (alpha) a[c] = __ldg(alpha + e0 / kMxBlock);
    }
  }
#pragma unroll
  for (int c = 0; c < kMxChunks; ++c) {
    const int64_t e0 = base + c * kMxThreads * 8;
    const MxLane l = mx_lane(w[c], a[c]);
    if (e0 >= n) continue;
    float x[8];
    mx_unpack(w[c], x);
    const float vv[8] = {v[c][0].x, v[c][0].y, v[c][0].z, v[c][0].w, v[c][1].x, v[c][1].y, v[c][1].z, v[c][1].w};
    uint32_t word = 0;
    uint32_t out[4];
    bool bad = l.bad;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float t0 = add_odd(__fmul_rn(x[2 * i], l.inv), vv[2 * i]);
      const float t1 = add_odd(__fmul_rn(x[2 * i + 1], l.inv), vv[2 * i + 1]);
      bad |= !(fabsf(t0) <= 3.4028235e38f) || !(fabsf(t1) <= 3.4028235e38f);
      const uint32_t q = (l.zero || l.bad) ? 0u : e2m1_pair(t0, t1);
      word |= q << (8 * i);
      const float2 f = e2m1_values(q);
      out[i] = l.bad ? 0x7FC07FC0u : pack_bf16x2(__fmul_rn(f.x, l.X), __fmul_rn(f.y, l.X));
    }
    if (bad) raise_status(kStatusNonFinite);
    if (W_hat) __stcs(reinterpret_cast<uint4*>(W_hat + e0), make_uint4(out[0], out[1], out[2], out[3]));
    if (codes) __stcs(reinterpret_cast<unsigned int*>(codes + e0 / 2), word);
    if (scales && (threadIdx.x & 3) == 0) scales[e0 / kMxBlock] = static_cast<uint8_t>(l.code);
  }
}

// Straight-through backward from g = dL/dW_hat (fp32): both roundings (of the
// scale's exponent and of the codes) count as the identity, the gradient passes
// where |W/X + V| <= 6 (m = 1), products use the forward's values:
//   dV = g X m,   dalpha_b = (X / alpha_b) sum_block g (q - m W / X)
// (d X / d alpha = X / alpha when the exponent's rounding is the identity).  A
// block of zeros has no gradient, nor has alpha where X is held at 2^-127.
// UPDATE: V <- clamp(V - lr sign(dV)), alpha <- clamp(alpha - lr sign(dalpha))
// in place ([AR] §3 "SignSGD"; sign(0) = 0, a NaN gradient counts as 0 and raises
// the non-finite status).  The four lanes of a block add their parts in a fixed
// tree, so results do not depend on timing.
struct MxStep {
  float lr, v_min, v_max, c_min, c_max;
};

__device__ __forceinline__ float mx_sign(float d) { return d > 0.f ? 1.f : (d < 0.f ? -1.f : 0.f); }

template <bool UPDATE>
__global__ void __launch_bounds__(kMxThreads) bwd_mxfp4_kernel(const float* __restrict__ dW,
                                                               const uint16_t* __restrict__ W, const float* V,
                                                               const float* alpha, int64_t n, float* V_out,
                                                               float* alpha_out, MxStep step, float* dV_out,
                                                               float* da_out) {
  const int64_t base = (blockIdx.x * static_cast<int64_t>(kMxThreads * kMxChunks) + threadIdx.x) * 8;
  uint4 w[kMxChunks];
  float4 v[kMxChunks][2], g[kMxChunks][2];
  float a[kMxChunks];
#pragma unroll
  for (int c = 0; c < kMxChunks; ++c) {
    const int64_t e0 = base + c * kMxThreads * 8;
    w[c] = make_uint4(0u, 0u, 0u, 0u);
    v[c][0] = v[c][1] = g[c][0] = g[c][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    a[c] = 1.0f;
    if (e0 < n) {
      w[c] = __ldcs(reinterpret_cast<const uint4*>(W + e0));
      g[c][0] = __ldcs(reinterpret_cast<const float4*>(dW + e0));
      g[c][1] = __ldcs(reinterpret_cast<const float4*>(dW + e0 + 4));
      if (V) {
        v[c][0] = __ldcs(reinterpret_cast<const float4*>(V + e0));
        v[c][1] = __ldcs(reinterpret_cast<const float4*>(V + e0 + 4));
      }
      if (alpha) a[c] = alpha[e0 / kMxBlock];
    }
  }
#pragma unroll
  for (int c = 0; c < kMxChunks; ++c) {
    const int64_t e0 = base + c * kMxThreads * 8;
    const MxLane l = mx_lane(w[c], a[c]);
    float x[8];
    mx_unpack(w[c], x);
    const float vv[8] = {v[c][0].x, v[c][0].y, v[c][0].z, v[c][0].w, v[c][1].x, v[c][1].y, v[c][1].z, v[c][1].w};
    const float gg[8] = {g[c][0].x, g[c][0].y, g[c][0].z, g[c][0].w, g[c][1].x, g[c][1].y, g[c][1].z, g[c][1].w};
    const bool dead = l.zero || l.bad || !(a[c] > 0.0f);
    float dv[8], sum = 0.0f;
    bool bad = l.bad;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s0 = __fmul_rn(x[2 * i], l.inv), s1 = __fmul_rn(x[2 * i + 1], l.inv);
      const float t0 = add_odd(s0, vv[2 * i]), t1 = add_odd(s1, vv[2 * i + 1]);
      const float2 q = e2m1_values(e2m1_pair(t0, t1));
      const bool m0 = fabsf(t0) <= kE2M1Max, m1 = fabsf(t1) <= kE2M1Max;
      dv[2 * i] = m0 && !dead ? __fmul_rn(gg[2 * i], l.X) : 0.0f;
      dv[2 * i + 1] = m1 && !dead ? __fmul_rn(gg[2 * i + 1], l.X) : 0.0f;
      sum = __fmaf_rn(gg[2 * i], m0 ? q.x - s0 : q.x, sum);
      sum = __fmaf_rn(gg[2 * i + 1], m1 ? q.y - s1 : q.y, sum);
      bad |= !(fabsf(gg[2 * i]) <= 3.4028235e38f) || !(fabsf(gg[2 * i + 1]) <= 3.4028235e38f);
    }
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
    if (e0 >= n) continue;
    if (bad) raise_status(kStatusNonFinite);
    const float da = dead || l.code == 0 ? 0.0f : __fmul_rn(__fdiv_rn(l.X, a[c]), sum);
    if (dV_out) {
      __stcs(reinterpret_cast<float4*>(dV_out + e0), make_float4(dv[0], dv[1], dv[2], dv[3]));
      __stcs(reinterpret_cast<float4*>(dV_out + e0 + 4), make_float4(dv[4], dv[5], dv[6], dv[7]));
    }
    if (da_out && (threadIdx.x & 3) == 0) da_out[e0 / kMxBlock] = da;
    if (UPDATE) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] = fminf(fmaxf(__fsub_rn(vv[i], step.lr * mx_sign(dv[i])), step.v_min), step.v_max);
      __stcs(reinterpret_cast<float4*>(V_out + e0), make_float4(o[0], o[1], o[2], o[3]));
      __stcs(reinterpret_cast<float4*>(V_out + e0 + 4), make_float4(o[4], o[5], o[6], o[7]));
      if ((threadIdx.x & 3) == 0)
        alpha_out[e0 / kMxBlock] = fminf(fmaxf(__fsub_rn(a[c], step.lr * mx_sign(da)), step.c_min), step.c_max);
    }
  }
}

// Packed codes and scales -> bf16 values (exact: two significant bits times a
// power of two).  A lane takes 8 codes (one word) and writes 16 bytes.
__global__ void __launch_bounds__(kMxThreads) expand_mxfp4_kernel(const uint32_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales, int64_t n,
                                                                  uint16_t* __restrict__ out) {
  constexpr int kWords = 4;
  const int64_t base = (blockIdx.x * static_cast<int64_t>(kMxThreads * kWords) + threadIdx.x) * 8;
  uint32_t w[kWords];
  int s[kWords];
#pragma unroll
  for (int c = 0; c < kWords; ++c) {
    const int64_t e0 = base + c * kMxThreads * 8;
    w[c] = e0 < n ? __ldcs(codes + e0 / 8) : 0u;
    s[c] = e0 < n ? static_cast<int>(__ldg(scales + e0 / kMxBlock)) : 0;
  }
#pragma unroll
  for (int c = 0; c < kWords; ++c) {
    const int64_t e0 = base + c * kMxThreads * 8;
    if (e0 >= n) continue;
    const float X = s[c] == 255 ? __uint_as_float(0x7FC00000u) : mx_pow2(s[c]);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e2m1_values((w[c] >> (8 * i)) & 0xFFu);
      o[i] = pack_bf16x2(__fmul_rn(f.x, X), __fmul_rn(f.y, X));
    }
    *reinterpret_cast<uint4*>(out + e0) = make_uint4(o[0], o[1], o[2], o[3]);  // read by the next kernel: kept in L2
  }
}

int64_t blocks_for(int64_t n, int chunks) {
  const int64_t per = static_cast<int64_t>(kMxThreads) * chunks * 8;
  return (n + per - 1) / per;
}

}  // namespace

cudaError_t launch_qdq_mxfp4(const uint16_t* W, const float* V, const float* alpha, int64_t n, uint16_t* W_hat,
                             uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
  const int64_t blocks = blocks_for(n, kMxChunks);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  {
    LaunchScope scope(stream, "qdq_mxfp4_kernel");
    qdq_mxfp4_kernel<<<static_cast<unsigned>(blocks), kMxThreads, 0, stream>>>(W, V, alpha, n, W_hat, codes, scales);
  }
  return cudaGetLastError();
}

cudaError_t launch_bwd_mxfp4(const float* dW, const uint16_t* W, const float* V, const float* alpha, int64_t n,
                             float* dV_out, float* da_out, cudaStream_t stream) {
  const int64_t blocks = blocks_for(n, kMxChunks);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  {
    LaunchScope scope(stream, "bwd_mxfp4_kernel");
    bwd_mxfp4_kernel<false><<<static_cast<unsigned>(blocks), kMxThreads, 0, stream>>>(
        dW, W, V, alpha, n, nullptr, nullptr, MxStep{}, dV_out, da_out);
  }
  return cudaGetLastError();
}

cudaError_t launch_fold_mxfp4(const float* dW, const uint16_t* W, float* V, float* alpha, int64_t n, float lr,
                              float v_min, float v_max, float c_min, float c_max, float* dV_out, float* da_out,
                              cudaStream_t stream) {
  const int64_t blocks = blocks_for(n, kMxChunks);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  {
    LaunchScope scope(stream, "fold_mxfp4_kernel");
    bwd_mxfp4_kernel<true><<<static_cast<unsigned>(blocks), kMxThreads, 0, stream>>>(
        dW, W, V, alpha, n, V, alpha, MxStep{lr, v_min, v_max, c_min, c_max}, dV_out, da_out);
  }
  return cudaGetLastError();
}

cudaError_t launch_expand_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t n, uint16_t* out,
                                cudaStream_t stream) {
  const int64_t blocks = blocks_for(n, 4);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  {
    LaunchScope scope(stream, "expand_mxfp4_kernel");
    expand_mxfp4_kernel<<<static_cast<unsigned>(blocks), kMxThreads, 0, stream>>>(
        reinterpret_cast<const uint32_t*>(codes), scales, n, out);
  }
  return cudaGetLastError();
}

}  // namespace ar
