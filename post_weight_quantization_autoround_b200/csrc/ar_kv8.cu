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
// not depend on timing.  The bytes are the floor (read 2 B, write 2 B a query
// element, read 2 B, write 1 B a key or value element).  A thread owns 16 elements of one
// token for all the block's heads, so its 8 cosines and sines are computed once (in shared memory,
// at an address of its own: 16 registers more would spill), a page's tokens are all there at once, and keys and values share one barrier a head.
//  * Up to 128 threads' worth of new tokens in a page (a decode step): loads straight to
//    registers, idle threads take query heads.
//  * More: a head's tokens come as TMA boxes through a ring in shared memory, so
//    that loads stay in flight across the barrier: 8 prompts of 2048 tokens, 32 + 32 heads of 128, 162 us
//    (671 MB, 4.1 TB/s, 63 % of a copy's rate); in registers 210 us.  Latency bounds it: 1.7 instructions a cycle
//    of 4, a quarter of the SM's warps (one block of 512 threads), which wait for loads first; a block's angles
//    and first boxes overlap with nothing.
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
  return {__ldcs(reinterpret_cast<const uint4*>(p)), __ldcs(reinterpret_cast<const uint4*>(p + half))};
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

// cs: this thread's (cos, sin) pairs, two to a 16-byte word, THREADS words apart: a
// thread reads its own, so the words of a warp lie side by side
template <int THREADS>
__device__ __forceinline__ Sixteen rotated(const Raw& r, const float4* cs) {
  Sixteen x = values_of(r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = cs[i * THREADS];
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

__device__ __forceinline__ uint32_t max_mag(const Sixteen& x) {  // bits: a NaN lies above infinity
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_mag(max_mag(m, x.lo[i]), x.hi[i]);
  return __float_as_uint(m);
}

__device__ __forceinline__ uint32_t max_mag(const Raw& r) {  // of unrotated values: bf16 magnitudes order like integers
  const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16) << 16;
}

__device__ __forceinline__ uint32_t max_finite(const Sixteen& x) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (fabsf(x.lo[i]) <= 3.4028235e38f) m = fmaxf(m, fabsf(x.lo[i]));
    if (fabsf(x.hi[i]) <= 3.4028235e38f) m = fmaxf(m, fabsf(x.hi[i]));
  }
  return __float_as_uint(m);
}

constexpr int kRing = 4;  // units (a head's new tokens of the page) in shared memory

struct RingCtl {
  uint64_t full[kRing], empty[kRing];
  int abort_flag;
};

// D: head dimension; PASSES THREADS / (D / 16) tokens at most are new in a page; RING: through shared memory
// (else PASSES = 1)
template <int D, int THREADS, int PASSES, bool RING>
__global__ void __launch_bounds__(THREADS, RING ? 512 / THREADS : 4)
    kv8_append_kernel(const __grid_constant__ CUtensorMap tm, const Kv8Args a, const uint16_t* __restrict__ qkv,
                      const __grid_constant__ RopeTurns turns,
                      uint8_t* __restrict__ k_pages, uint8_t* __restrict__ v_pages, uint8_t* __restrict__ k_scales,
                      uint8_t* __restrict__ v_scales, uint16_t* __restrict__ q_out, int heads_per_block) {
  constexpr int kHalf = D / 2;
  constexpr int kLanes = D / 16;             // threads that share a token's head
  constexpr int kPass = THREADS / kLanes;    // tokens at once
  constexpr int kSlots = PASSES * kPass;     // tokens
  constexpr int kWarps = THREADS / 32;
  constexpr int kUnitBytes = kSlots * D * 2;  // a box: a head of the page's tokens
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));  // TMA boxes
  __shared__ uint2 warp_max[2][kWarps];
  __shared__ RingCtl ctl;

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
  const int n = hi - lo;  // new tokens in this page, at most kSlots
  const int physical = a.table[static_cast<int64_t>(s) * a.max_pages + pi];
  const bool page_ok = physical >= 0 && physical < a.n_pages;
  if (!page_ok && tid == 0) raise_status(kStatusBadIndex);  // the queries are still written

  // thread -> elements el .. el + 7 and D / 2 further of token t (in the ring: and t + kPass, ...); without the
  // ring copy `rep` of the tokens takes every `reps`-th query head
  const int el = 8 * (tid % kLanes);
  const int slot = tid / kLanes;
  const int reps = RING ? 1 : kSlots / n, rep = RING ? 0 : slot / n, t = slot - rep * n;
  const bool live = rep < reps, holds = live && rep == 0;
  float4* cs = reinterpret_cast<float4*>(ring + (RING ? kRing * kUnitBytes : 0)) + tid;
#pragma unroll
  for (int p = 0; p < PASSES; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float c[2], sn[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const double turn = static_cast<double>(lo + t + p * kPass) * turns.f[el + 2 * i + j];
        sincospif(2.0f * static_cast<float>(turn - rint(turn)), &sn[j], &c[j]);
      }
      cs[(4 * p + i) * THREADS] = make_float4(c[0], sn[0], c[1], sn[1]);
    }
  const int64_t row = first_row + (lo - start) + t;
  const int64_t ld = static_cast<int64_t>(a.n_heads + 2 * a.n_kv) * D;
  const int group = a.n_heads / a.n_kv;
  const int h0 = blockIdx.z * heads_per_block;
  const int h1 = min(a.n_kv, h0 + heads_per_block);
  const uint16_t* src = qkv + row * ld + el;
  const Raw none{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};

  // the ring's units in order: for every head its keys, its values, the queries that read them
  const int per_head = 2 + group, units = (h1 - h0) * per_head;
  int issued = 0;
  bool alive = true;
  auto issue = [&]() {  // thread 0
    const int u = issued, slot_u = u % kRing;
    if (u >= kRing && !mbar_wait(&ctl.empty[slot_u], ((u / kRing) - 1) & 1, &ctl.abort_flag)) return;
    const int h = h0 + u / per_head, j = u % per_head;
    const int col = (j == 0 ? a.n_heads + h : j == 1 ? a.n_heads + a.n_kv + h : h * group + j - 2) * D;
    mbar_arrive_expect_tx(&ctl.full[slot_u], kUnitBytes);
    tma_load_2d(ring + slot_u * kUnitBytes, &tm, &ctl.full[slot_u], col, static_cast<int>(first_row) + (lo - start));
    ++issued;
  };
  if (RING) {
    if (tid == 0) {
      for (int i = 0; i < kRing; ++i) {
        mbar_init(&ctl.full[i], 1);
        mbar_init(&ctl.empty[i], kWarps);
      }
      ctl.abort_flag = 0;
      fence_barrier_init();
      for (int i = 0; i < kRing && i < units; ++i) issue();
    }
    __syncthreads();
  }
  auto wait_unit = [&](int u) {
    if (alive) alive = mbar_wait(&ctl.full[u % kRing], (u / kRing) & 1, &ctl.abort_flag);
  };
  auto release_unit = [&](int u) {
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(&ctl.empty[u % kRing]);
    // refill the slot before this one: its last warp is likely done, this one's is not
    if (tid == 0 && alive && issued < units && issued - kRing < u) issue();
  };
  auto unit = [&](int u, int p) {
    const uint4* at = reinterpret_cast<const uint4*>(ring + (u % kRing) * kUnitBytes + (slot + p * kPass) * (D * 2) + el * 2);
    return Raw{at[0], at[kHalf / 8]};
  };
  const bool older = lo > page0;
  int buf = 0;

  // the largest of both over the block; every thread gets them
  auto block_max = [&](uint32_t k, uint32_t v) {
    k = __reduce_max_sync(0xFFFFFFFFu, k);
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if ((tid & 31) == 0) warp_max[buf][tid >> 5] = make_uint2(k, v);
    __syncthreads();
    const uint2 m = warp_max[buf][(tid & 31) < kWarps ? (tid & 31) : 0];
    buf ^= 1;  // the next maximum is written while this one may still be read
    return make_uint2(__reduce_max_sync(0xFFFFFFFFu, m.x), __reduce_max_sync(0xFFFFFFFFu, m.y));
  };
  auto store_codes = [&](uint8_t* pages, const Sixteen& x, int64_t head, float inv, int p) {
    uint8_t* o = pages + (head * a.page + (lo - page0 + t + p * kPass)) * D + el;
    *reinterpret_cast<uint2*>(o) = make_uint2(e4m3x4(x.lo[0] * inv, x.lo[1] * inv, x.lo[2] * inv, x.lo[3] * inv),
                                              e4m3x4(x.lo[4] * inv, x.lo[5] * inv, x.lo[6] * inv, x.lo[7] * inv));
    *reinterpret_cast<uint2*>(o + kHalf) = make_uint2(e4m3x4(x.hi[0] * inv, x.hi[1] * inv, x.hi[2] * inv, x.hi[3] * inv),
                                                      e4m3x4(x.hi[4] * inv, x.hi[5] * inv, x.hi[6] * inv, x.hi[7] * inv));
  };
  auto recode = [&](uint8_t* pages, int64_t head, int before, int e) {  // the page's older tokens, to a larger scale
    const float f = before - e < -126 ? 0.0f : pow2f(before - e);
    uint32_t* w = reinterpret_cast<uint32_t*>(pages + head * a.page * D);
    for (int i = tid; i < (lo - page0) * (D / 4); i += THREADS) {
      const float2 p0 = e4m3x2_values(w[i] & 0xFFFFu), p1 = e4m3x2_values(w[i] >> 16);
      w[i] = e4m3x4(p0.x * f, p0.y * f, p1.x * f, p1.y * f);
    }
  };
  auto no_nan = [](Sixteen& x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (x.lo[i] != x.lo[i]) x.lo[i] = 0.0f;
      if (x.hi[i] != x.hi[i]) x.hi[i] = 0.0f;
    }
  };

  Raw k = none, v = none;  // without the ring: this head's, and loads of the next in flight
  auto queries = [&](const Raw& q, int qh, int p) {
    const Sixteen x = rotated<THREADS>(q, cs + 4 * p * THREADS);
    uint16_t* o = q_out + ((row + p * kPass) * a.n_heads + qh) * D + el;
    __stcs(reinterpret_cast<uint4*>(o), make_uint4(pack_bf16x2(x.lo[0], x.lo[1]), pack_bf16x2(x.lo[2], x.lo[3]),
                                                   pack_bf16x2(x.lo[4], x.lo[5]), pack_bf16x2(x.lo[6], x.lo[7])));
    __stcs(reinterpret_cast<uint4*>(o + kHalf), make_uint4(pack_bf16x2(x.hi[0], x.hi[1]), pack_bf16x2(x.hi[2], x.hi[3]),
                                                           pack_bf16x2(x.hi[4], x.hi[5]), pack_bf16x2(x.hi[6], x.hi[7])));
  };
  if (!RING && holds && page_ok) {
    k = load_raw(src + (a.n_heads + h0) * D, kHalf);
    v = load_raw(src + (a.n_heads + a.n_kv + h0) * D, kHalf);
  }
  for (int h = h0; h < h1; ++h) {
    const int u = (h - h0) * per_head;
    if (RING) {
      wait_unit(u);
      wait_unit(u + 1);
    }
    if (page_ok) {  // uniform over the block
      const int64_t head = static_cast<int64_t>(physical) * a.n_kv + h;
      Raw k_next = none, v_next = none;
      if (!RING && holds && h + 1 < h1) {  // in flight while this head's maximum is found
        k_next = load_raw(src + (a.n_heads + h + 1) * D, kHalf);
        v_next = load_raw(src + (a.n_heads + a.n_kv + h + 1) * D, kHalf);
      }
      // a token's keys and values; formed once for the maximum and again for the codes, which costs less than
      // holding them across the barrier
      auto key_raw = [&](int p) { return RING ? unit(u, p) : k; };
      auto value_raw = [&](int p) { return RING ? unit(u + 1, p) : v; };
      auto has = [&](int p) { return RING ? slot + p * kPass < n : holds; };
      // older tokens keep at least their exponent
      const int bk = older ? min(max(static_cast<int>(k_scales[head]) - 127, kExpMin), kExpMax) : kExpMin;
      const int bv = older ? min(max(static_cast<int>(v_scales[head]) - 127, kExpMin), kExpMax) : kExpMin;
      uint32_t mk = 0u, mv = 0u;
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (has(p)) {
          mk = max(mk, max_mag(rotated<THREADS>(key_raw(p), cs + 4 * p * THREADS)));
          mv = max(mv, max_mag(value_raw(p)));
        }
      uint2 top = block_max(mk, mv);
      const bool bad = max(top.x, top.y) >= 0x7F800000u;
      if (bad) {
        // the largest finite magnitude decides; a NaN is stored as 0, an infinity as the largest code
        if (tid == 0) raise_status(kStatusNonFinite);
        mk = mv = 0u;
        for (int p = 0; p < PASSES; ++p)
          if (has(p)) {
            mk = max(mk, max_finite(rotated<THREADS>(key_raw(p), cs + 4 * p * THREADS)));
            mv = max(mv, max_finite(values_of(value_raw(p))));
          }
        top = block_max(mk, mv);
      }
      const int ek = max(exponent_for(__uint_as_float(top.x)), bk), ev = max(exponent_for(__uint_as_float(top.y)), bv);
      const float ik = pow2f(-ek), iv = pow2f(-ev);
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (has(p)) {
          Sixteen x = rotated<THREADS>(key_raw(p), cs + 4 * p * THREADS);
          if (bad) no_nan(x);
          store_codes(k_pages, x, head, ik, p);
          x = values_of(value_raw(p));
          if (bad) no_nan(x);
          store_codes(v_pages, x, head, iv, p);
        }
      if (older && ek > bk) recode(k_pages, head, bk, ek);
      if (older && ev > bv) recode(v_pages, head, bv, ev);
      if (tid == 0) {  // every thread has read the old scales: the maximum's barrier lies between
        k_scales[head] = static_cast<uint8_t>(ek + 127);
        v_scales[head] = static_cast<uint8_t>(ev + 127);
      }
      k = k_next;
      v = v_next;
    }
    if (RING) {
      release_unit(u);
      release_unit(u + 1);
      for (int j = 0; j < group; ++j) {
        wait_unit(u + 2 + j);
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
          if (slot + p * kPass < n) queries(unit(u + 2 + j, p), h * group + j, p);
        release_unit(u + 2 + j);
      }
    } else if (live) {
      for (int j = rep; j < group; j += reps) queries(load_raw(src + (h * group + j) * D, kHalf), h * group + j, 0);
    }
  }
  if (RING && tid == 0) {
    // a wait that gave up leaves copies in flight: they land before the block may end
    for (int u = issued > kRing ? issued - kRing : 0; u < issued; ++u) mbar_wait_drain(&ctl.full[u % kRing], (u / kRing) & 1);
  }
}

template <int D, int THREADS, int PASSES, bool RING>
cudaError_t append(const Kv8Args& a, const uint16_t* qkv, const RopeTurns& turns, uint8_t* k_pages, uint8_t* v_pages,
                   uint8_t* k_scales, uint8_t* v_scales, uint16_t* q_out, cudaStream_t stream) {
  // pages that max_new tokens can touch, whatever their place in the first
  const int per_seq = (a.max_new + a.page - 2) / a.page + 1;
  // as many heads to a block as leave six rounds of blocks: they share its angles
  const int64_t blocks = static_cast<int64_t>(per_seq) * a.S, want = 6ll * num_sms() * (RING ? 512 / THREADS : 4);
  int heads = 1;
  while (heads < a.n_kv && blocks * ((a.n_kv + 2 * heads - 1) / (2 * heads)) >= want) heads *= 2;
  auto kern = kv8_append_kernel<D, THREADS, PASSES, RING>;
  CUtensorMap tm{};
  constexpr int kSlots = PASSES * THREADS / (D / 16);
  constexpr int smem = (RING ? kRing * kSlots * D * 2 : 0) + PASSES * THREADS * 64 + 128;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed);
  if (e != cudaSuccess) return e;
  if (RING) {
    // a box: one head's columns of the page's tokens
    e = make_tmap_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, qkv, static_cast<uint64_t>(a.T),
                     static_cast<uint64_t>(a.n_heads + 2 * a.n_kv) * D, D, kSlots, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
  }
  {
    LaunchScope scope(stream, RING ? "kv8_append_kernel<ring>" : "kv8_append_kernel");
    kern<<<dim3(per_seq, a.S, (a.n_kv + heads - 1) / heads), THREADS, smem, stream>>>(tm, a, qkv, turns, k_pages, v_pages,
                                                                                       k_scales, v_scales, q_out, heads);
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t append_d(const Kv8Args& a, const uint16_t* qkv, const RopeTurns& t, uint8_t* kp, uint8_t* vp, uint8_t* ks,
                     uint8_t* vs, uint16_t* q, cudaStream_t st) {
  // threads for the most new tokens that a page can take
  constexpr int kLanes = D / 16;
  const int most = (a.max_new < a.page ? a.max_new : a.page) * kLanes;
  if (most <= 128) return append<D, 128, 1, false>(a, qkv, t, kp, vp, ks, vs, q, st);
  if (most <= 256) return append<D, 256, 1, true>(a, qkv, t, kp, vp, ks, vs, q, st);
  if (most <= 512) return append<D, 512, 1, true>(a, qkv, t, kp, vp, ks, vs, q, st);
  if constexpr (D == 128) return append<D, 512, 2, true>(a, qkv, t, kp, vp, ks, vs, q, st);
  return cudaErrorInvalidValue;  // not reached: a page has at most 128 tokens
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Args& a, const uint16_t* qkv, double rope_base, uint8_t* k_pages,
                              uint8_t* v_pages, uint8_t* k_scales, uint8_t* v_scales, uint16_t* q_out,
                              cudaStream_t stream) {
  RopeTurns t{};
  // one power, then products: 64 roundings of 2^-53 turn position 10^9 by 10^-5 rad at most, and 64 powers would be a
  // fifth of a small call's time on the host
  const double step = pow(rope_base, -2.0 / a.head_dim);
  t.f[0] = 0.15915494309189533577;  // 1 / (2 pi)
  for (int i = 1; i < a.head_dim / 2; ++i) t.f[i] = t.f[i - 1] * step;
  if (a.head_dim == 128) return append_d<128>(a, qkv, t, k_pages, v_pages, k_scales, v_scales, q_out, stream);
  return append_d<64>(a, qkv, t, k_pages, v_pages, k_scales, v_scales, q_out, stream);
}

}  // namespace ar
