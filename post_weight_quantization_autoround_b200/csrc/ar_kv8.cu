// Appending to a paged 8-bit cache: the new tokens' queries and keys are rotated by
// their positions, keys and values are quantized and written into their sequences'
// pages, all in one pass over the stacked projection's output.
//
// A page holds `page` tokens of one sequence, per key/value head a [page][d] array of
// E4M3 codes and one power-of-two scale (E8M0) for keys and one for values.  E4M3 is
// itself a floating-point type, so a finer scale would buy range, not precision; a
// power of two makes the reader's scale an exponent and lets a page whose scale grows
// be re-coded exactly (but for subnormal codes, which round once more):
//   e = the smallest exponent with max |x| <= 448 2^e over the page's new tokens of the
//       head, within [-100, 120]; at least the page's present e when the page holds
//       older tokens, whose codes then become E4M3(code 2^(e_old - e))
//   code = E4M3(x 2^-e), nearest even
//   rotation: (x_i, x_{i+d/2}) -> (x_i c - x_{i+d/2} s, x_{i+d/2} c + x_i s), c, s =
//       cos, sin of position base^(-2i/d); fp32, quantized without another rounding
// The angle is taken in turns, position * base^(-2i/d) / 2 pi in fp64, and only what is
// left of whole turns goes to fp32: at position 10^6 an fp32 angle is off by 0.03.
//
// One block owns (sequence, page, a range of key/value heads): it alone writes the
// page's codes and scale of those heads, so there are no atomics and the result does
// not depend on timing.  The kernel is bound by memory (read 2 B, write 2 B a query
// element, read 2 B, write 1 B a key or value element); the block's cosines and sines
// are computed once in shared memory and serve all its heads, and a token's keys stay
// in registers, as loaded, between the maximum and the codes.
#include <cuda_fp8.h>

#include "ar_internal.h"

namespace ar {
namespace {

constexpr int kExpMin = -100;
constexpr int kExpMax = 120;

struct RopeTurns {
  double f[64];  // base^(-2i/d) / (2 pi)
};

// the smallest e with top <= 448 * 2^e = 1.75 * 2^(e + 8), within the scale's range
__device__ __forceinline__ int exponent_for(float top) {
  const uint32_t b = __float_as_uint(top);
  int e = static_cast<int>(b >> 23) - 127 - 8;
  if ((b & 0x7FFFFFu) > 0x600000u) ++e;
  return min(max(e, kExpMin), kExpMax);
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_values(uint32_t two) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3)));
}

// a lane's 16 elements of a head as loaded: 8 of the first half and the 8 they rotate with
struct Raw {
  uint4 lo, hi;
};

struct Sixteen {
  float lo[8], hi[8];
};

__device__ __forceinline__ Raw load_raw(const uint16_t* p, int half) {
  return {__ldg(reinterpret_cast<const uint4*>(p)), __ldg(reinterpret_cast<const uint4*>(p + half))};
}

__device__ __forceinline__ Sixteen values_of(const Raw& r) {
  const uint32_t a[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w}, b[4] = {r.hi.x, r.hi.y, r.hi.z, r.hi.w};
  Sixteen x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.lo[2 * i] = bf16_lo(a[i]);
    x.lo[2 * i + 1] = bf16_hi(a[i]);
    x.hi[2 * i] = bf16_lo(b[i]);
    x.hi[2 * i + 1] = bf16_hi(b[i]);
  }
  return x;
}

__device__ __forceinline__ Sixteen rotated(const Raw& r, const float2* cs) {
  Sixteen x = values_of(r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = *reinterpret_cast<const float4*>(cs + 2 * i);  // two pairs (cos, sin)
    const float a0 = x.lo[2 * i], b0 = x.hi[2 * i], a1 = x.lo[2 * i + 1], b1 = x.hi[2 * i + 1];
    x.lo[2 * i] = a0 * t.x - b0 * t.y;
    x.hi[2 * i] = b0 * t.x + a0 * t.y;
    x.lo[2 * i + 1] = a1 * t.z - b1 * t.w;
    x.hi[2 * i + 1] = b1 * t.z + a1 * t.w;
  }
  return x;
}

// max(m, |x|), a NaN wins
__device__ __forceinline__ float max_mag(float m, float x) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(m), "f"(x));
  return r;
}

// D: head dimension; PASSES * (threads / (D / 16)) covers the new tokens that a page can take
template <int D, int PASSES, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS)
    kv8_append_kernel(const Kv8Args a, const uint16_t* __restrict__ qkv, const __grid_constant__ RopeTurns turns,
                      uint8_t* __restrict__ k_pages, uint8_t* __restrict__ v_pages, uint8_t* __restrict__ k_scales,
                      uint8_t* __restrict__ v_scales, uint16_t* __restrict__ q_out, int heads_per_block) {
  constexpr int kHalf = D / 2;
  constexpr int kLanes = D / 16;             // lanes that share a token's head
  constexpr int kTokens = THREADS / kLanes;  // tokens per pass
  constexpr int kWarps = THREADS / 32;
  extern __shared__ __align__(16) float2 cs[];  // [tokens][D / 2]
  __shared__ float warp_max[2][kWarps];

  const int s = blockIdx.y;
  const int tid = threadIdx.x;
  const int64_t first_row = a.cu[s], rows = a.cu[s + 1] - first_row;
  const int len = a.lens[s];
  // bounds that do not fit the arrays: nothing of the sequence is touched
  if (rows < 0 || rows > a.max_new || first_row < 0 || first_row + rows > a.T || len < rows ||
      len > static_cast<int64_t>(a.max_pages) * a.page) {
    if (tid == 0) raise_status(kStatusBadIndex);
    return;
  }
  const int n_new = static_cast<int>(rows);
  const int start = len - n_new;
  const int pi = start / a.page + static_cast<int>(blockIdx.x);
  const int page0 = pi * a.page;
  if (n_new == 0 || page0 >= len) return;
  const int lo = max(start, page0), hi = min(len, page0 + a.page);
  const int n = hi - lo;  // new tokens in this page
  const int physical = a.table[static_cast<int64_t>(s) * a.max_pages + pi];
  const bool page_ok = physical >= 0 && physical < a.n_pages;
  if (!page_ok && tid == 0) raise_status(kStatusBadIndex);  // the queries are still written

  for (int i = tid; i < n * kHalf; i += THREADS) {
    const int t = i / kHalf, f = i - t * kHalf;
    const double turn = static_cast<double>(lo + t) * turns.f[f];
    const float rest = static_cast<float>(turn - rint(turn));
    float sn, c;
    sincospif(2.0f * rest, &sn, &c);
    cs[i] = make_float2(c, sn);
  }
  __syncthreads();

  const int el = 8 * (tid % kLanes);  // this lane's elements: el .. el + 7 and D / 2 further
  const int tok0 = tid / kLanes;
  const int64_t row0 = first_row + (lo - start);
  const int64_t ld = static_cast<int64_t>(a.n_heads + 2 * a.n_kv) * D;
  const int group = a.n_heads / a.n_kv;
  const int h0 = blockIdx.z * heads_per_block;
  const int h1 = min(a.n_kv, h0 + heads_per_block);
  int buf = 0;

  // the largest magnitude over the block (a NaN wins); every thread gets it
  auto block_max = [&](float top) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_mag(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if ((tid & 31) == 0) warp_max[buf][tid >> 5] = top;
    __syncthreads();
    top = warp_max[buf][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = max_mag(top, warp_max[buf][w]);
    buf ^= 1;  // the next maximum is written while this one may still be read
    return top;
  };

  for (int h = h0; h < h1; ++h) {
    Raw kv[2][PASSES];  // keys and values: loaded before the queries are worked on
    if (page_ok) {
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          const int t = tok0 + p * kTokens;
          kv[part][p] = t < n ? load_raw(qkv + (row0 + t) * ld + (a.n_heads + part * a.n_kv + h) * D + el, kHalf)
                              : Raw{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        }
    }
    // queries of the heads that read this one, two loads in flight beside the keys' and values'
    constexpr int kQ = PASSES < 2 ? PASSES : 2;
    for (int j0 = tok0; j0 < n * group; j0 += kQ * kTokens) {
      Raw q[kQ];
#pragma unroll
      for (int p = 0; p < kQ; ++p) {
        const int j = j0 + p * kTokens, t = j / group;
        if (j < n * group) q[p] = load_raw(qkv + (row0 + t) * ld + (h * group + (j - t * group)) * D + el, kHalf);
      }
#pragma unroll
      for (int p = 0; p < kQ; ++p) {
        const int j = j0 + p * kTokens, t = j / group;
        if (j >= n * group) continue;
        const Sixteen x = rotated(q[p], cs + t * kHalf + el);
        uint16_t* o = q_out + ((row0 + t) * a.n_heads + h * group + (j - t * group)) * D + el;
        __stcs(reinterpret_cast<uint4*>(o), make_uint4(pack_bf16x2(x.lo[0], x.lo[1]), pack_bf16x2(x.lo[2], x.lo[3]),
                                                       pack_bf16x2(x.lo[4], x.lo[5]), pack_bf16x2(x.lo[6], x.lo[7])));
        __stcs(reinterpret_cast<uint4*>(o + kHalf), make_uint4(pack_bf16x2(x.hi[0], x.hi[1]), pack_bf16x2(x.hi[2], x.hi[3]),
                                                               pack_bf16x2(x.hi[4], x.hi[5]), pack_bf16x2(x.hi[6], x.hi[7])));
      }
    }
    if (!page_ok) continue;  // uniform over the block
#pragma unroll
    for (int part = 0; part < 2; ++part) {  // keys, then values
      uint8_t* pages = part == 0 ? k_pages : v_pages;
      uint8_t* scale = (part == 0 ? k_scales : v_scales) + static_cast<int64_t>(physical) * a.n_kv + h;
      // the values are formed twice, for the maximum and for the codes: holding them would cost a block of occupancy
      auto value = [&](int p) {
        const int t = min(tok0 + p * kTokens, n - 1);
        return part == 0 ? rotated(kv[0][p], cs + t * kHalf + el) : values_of(kv[1][p]);
      };
      float top = 0.0f;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const Sixteen x = value(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max_mag(max_mag(top, x.lo[i]), x.hi[i]);
      }
      // older tokens keep at least their exponent
      const int before = lo > page0 ? min(max(static_cast<int>(*scale) - 127, kExpMin), kExpMax) : kExpMin;
      top = block_max(top);
      const bool bad = !(top <= 3.4028235e38f);
      if (bad) {  // the largest finite magnitude decides; a NaN is stored as 0, an infinity as the largest code
        if (tid == 0) raise_status(kStatusNonFinite);
        top = 0.0f;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          const Sixteen x = value(p);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (fabsf(x.lo[i]) <= 3.4028235e38f) top = fmaxf(top, fabsf(x.lo[i]));
            if (fabsf(x.hi[i]) <= 3.4028235e38f) top = fmaxf(top, fabsf(x.hi[i]));
          }
        }
        top = block_max(top);
      }
      const int e = max(exponent_for(top), before);
      uint8_t* dst = pages + (static_cast<int64_t>(physical) * a.n_kv + h) * a.page * D;
      const float inv = pow2f(-e);
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int t = tok0 + p * kTokens;
        if (t >= n) continue;
        Sixteen x = value(p);
        if (bad) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (x.lo[i] != x.lo[i]) x.lo[i] = 0.0f;
            if (x.hi[i] != x.hi[i]) x.hi[i] = 0.0f;
          }
        }
        uint8_t* o = dst + static_cast<int64_t>(lo - page0 + t) * D + el;
        *reinterpret_cast<uint2*>(o) = make_uint2(e4m3x4(x.lo[0] * inv, x.lo[1] * inv, x.lo[2] * inv, x.lo[3] * inv),
                                                  e4m3x4(x.lo[4] * inv, x.lo[5] * inv, x.lo[6] * inv, x.lo[7] * inv));
        *reinterpret_cast<uint2*>(o + kHalf) = make_uint2(e4m3x4(x.hi[0] * inv, x.hi[1] * inv, x.hi[2] * inv, x.hi[3] * inv),
                                                          e4m3x4(x.hi[4] * inv, x.hi[5] * inv, x.hi[6] * inv, x.hi[7] * inv));
      }
      if (lo > page0 && e > before) {
        const float f = before - e < -126 ? 0.0f : pow2f(before - e);
        uint32_t* w = reinterpret_cast<uint32_t*>(dst);
        for (int i = tid; i < (lo - page0) * (D / 4); i += THREADS) {
          const float2 p0 = e4m3x2_values(w[i] & 0xFFFFu), p1 = e4m3x2_values(w[i] >> 16);
          w[i] = e4m3x4(p0.x * f, p0.y * f, p1.x * f, p1.y * f);
        }
      }
      // every thread has read the old scale: the maximum's barrier lies between
      if (tid == 0) *scale = static_cast<uint8_t>(e + 127);
    }
  }
}

template <int D, int PASSES, int THREADS>
cudaError_t append(const Kv8Args& a, const uint16_t* qkv, const RopeTurns& turns, uint8_t* k_pages, uint8_t* v_pages,
                   uint8_t* k_scales, uint8_t* v_scales, uint16_t* q_out, cudaStream_t stream) {
  // pages that max_new tokens can touch, whatever their place in the first
  const int per_seq = (a.max_new + a.page - 2) / a.page + 1;
  const int tokens = a.max_new < a.page ? a.max_new : a.page;
  const int smem = tokens * (D / 2) * 8;
  auto kern = kv8_append_kernel<D, PASSES, THREADS>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), 128 * (D / 2) * 8, allowed);
  if (e != cudaSuccess) return e;
  // as many heads to a block as leave four blocks to an SM: they share its cosines and sines
  const int64_t blocks = static_cast<int64_t>(per_seq) * a.S;
  int heads = 1;
  while (heads < a.n_kv && blocks * ((a.n_kv + 2 * heads - 1) / (2 * heads)) >= 4 * num_sms()) heads *= 2;
  {
    LaunchScope scope(stream, "kv8_append_kernel");
    kern<<<dim3(per_seq, a.S, (a.n_kv + heads - 1) / heads), THREADS, smem, stream>>>(a, qkv, turns, k_pages, v_pages,
                                                                                       k_scales, v_scales, q_out, heads);
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t append_d(const Kv8Args& a, const uint16_t* qkv, const RopeTurns& t, uint8_t* kp, uint8_t* vp, uint8_t* ks,
                     uint8_t* vs, uint16_t* q, cudaStream_t st) {
  // passes x tokens per pass >= the new tokens that a page can take
  constexpr int kPer128 = 128 / (D / 16), kPer256 = 256 / (D / 16);
  const int most = a.max_new < a.page ? a.max_new : a.page;
  if (most <= kPer128) return append<D, 1, 128>(a, qkv, t, kp, vp, ks, vs, q, st);
  if (most <= kPer256) return append<D, 1, 256>(a, qkv, t, kp, vp, ks, vs, q, st);
  if (most <= 2 * kPer256) return append<D, 2, 256>(a, qkv, t, kp, vp, ks, vs, q, st);
  if constexpr (D == 128) return append<D, 4, 256>(a, qkv, t, kp, vp, ks, vs, q, st);
  return cudaErrorInvalidValue;  // not reached: a page has at most 128 tokens
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Args& a, const uint16_t* qkv, double rope_base, uint8_t* k_pages,
                              uint8_t* v_pages, uint8_t* k_scales, uint8_t* v_scales, uint16_t* q_out,
                              cudaStream_t stream) {
  RopeTurns t{};
  for (int i = 0; i < a.head_dim / 2; ++i)
    t.f[i] = pow(rope_base, -2.0 * i / a.head_dim) * 0.15915494309189533577;  // 1 / (2 pi)
  if (a.head_dim == 128) return append_d<128>(a, qkv, t, k_pages, v_pages, k_scales, v_scales, q_out, stream);
  return append_d<64>(a, qkv, t, k_pages, v_pages, k_scales, v_scales, q_out, stream);
}

}  // namespace ar
