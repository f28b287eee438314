// Product of a few tokens (T <= 8) with MXFP4 weights: out[t][n] = sum_k A[t][k] 2^(s - 127) E2M1.
//
// Every weight is read once for at most 8 products, so the packed bytes (0.53 a weight)
// set the floor and the instructions a word of 8 codes costs decide how near the kernel
// comes: 7 for the codes, 1 product, 2.5 for scales and sums, 2 loads.
//
//  * The weights are the left operand of mma.sync m16n8k16 (16 rows, 8 tokens as columns),
//    f16 in and fp32 out.  E2M1 is a subset of f16 and the hardware converts two codes to
//    an operand register in one instruction; bf16 operands would take three and a multiply.
//  * Activations become f16 by a power of two per token and 256 k (largest value in
//    [2^13, 2^14)): what f16 loses lies 2^-38 below that span's largest value.  The factor goes
//    back on when the span's sum is added.  Two kinds of span are summed again with a power of two per
//    token and block of 32, joined with the block's scale (careful_span): where a sum is not finite before
//    the factor (scale codes from about 232 on), so that the result overflows only where the product does; and
//    where a block's largest activation lies more than 2^16 below the span's, since the block's scale may
//    make up for it.  A block so loses 2^-22 of its largest activation at most, as much as the fp32 sum rounds.
//  * A 32-code block of a row is 16 bytes: lane c of a row's four takes word c, so the two
//    instructions of a block use 8 consecutive k a lane, activations are one 16-byte load,
//    and the block's scale multiplies the fp32 sums of exactly that block.
//  * Warps stream 16 rows x 256 k (2 KB boxes, 128-byte swizzle) through private rings; each takes an equal run of its block's (row tile, span) units and leaves a tile's
//    part in a slot of its own.  The CTAs of a cluster split k, so that a block's share of
//    the activations stays in shared memory; their sums meet through distributed shared
//    memory.  Parts are added in a fixed order.
//
// 5 tokens through 8192 x 28672 (125 MB of codes and scales): 46 us, 2.7 TB/s, 42 % of a copy's
// rate; 58 % of the issue slots and 55 % of the integer pipe are busy, about 58 instructions a
// block and tile, half of them the box's control; 1 us of it looks for sums that are not finite.  One token 41 us.
// Spans summed again take about four times as long: one in 112 2 us more, all of them 160 us.
// Four CTAs to a cluster instead of two 48 us (132 of 148 SMs hold clusters of four), 8 warps 66 us.
#include "ar_internal.h"

namespace ar {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;        // rows of a tile
constexpr int kSpan = 256;       // k of a unit: 128 bytes of codes a row
constexpr int kBoxBytes = kRows * 128;
constexpr int kStagesMax = 4;    // boxes of a warp's ring, as many as the activations leave room for, at least 2
constexpr int kPassTiles = 8;    // row tiles between two reductions
constexpr int kSlots = kPassTiles + kWarps;  // (tile, warp) pairs along the warps' runs: tile + warp is unique
constexpr int kRingBytes = kWarps * kBoxBytes;  // per stage
constexpr int kFixedBytes = (kSlots + kPassTiles) * 128 * 4 + 1024 + 1024;  // slots, sums, barriers, alignment
constexpr int kSmemMax = 226 * 1024;
constexpr uint32_t kFarBlock = 16;  // binary places that a block's activations may lie below the span's
constexpr int kActBytesMax = kSmemMax - kFixedBytes - 2 * kRingBytes;

struct DecCtl {
  uint64_t full[kWarps][kStagesMax];
  int abort_flag;
};

struct DecParams {
  const uint16_t* A;
  const uint8_t* scales;
  uint16_t* out;
  int T, N, K;
  int spans;       // of 256 k, in all
  int spans_cta;   // of a CTA (the last may have fewer)
  int tiles;       // row tiles
  int stages;
  int wide;        // a row's scale bytes of a span are one aligned 8-byte word
};

// the 8 codes of a word, two to a register, in order
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t e8m0x2_bf16(uint32_t two) {
  uint32_t d;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\t}" : "=r"(d) : "r"(two));
  return d;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, const float (&c)[4]) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// the largest magnitude, NaN if one is
__device__ __forceinline__ float max_mag4(const float (&x)[4]) {
  float m;
  asm("{\n\t.reg .f32 a, b, c, d;\n\tabs.f32 a, %1;\n\tabs.f32 b, %2;\n\tabs.f32 c, %3;\n\tabs.f32 d, %4;\n\t"
      "max.NaN.f32 a, a, b;\n\tmax.NaN.f32 c, c, d;\n\tmax.NaN.f32 %0, a, c;\n\t}"
      : "=f"(m)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
  return m;
}

// x 2^e for |e| <= 254 in two exact steps: an infinity or a lost bit is the product's own
__device__ __forceinline__ float times_pow2(float x, int e) {
  const int half = e / 2, rest = e - half;  // -127 .. 127
  auto pow2 = [](int n) { return __uint_as_float(n > -127 ? static_cast<uint32_t>(n + 127) << 23 : 0x00400000u); };
  return x * pow2(half) * pow2(rest);
}

// A warp's unit (16 rows x 256 k) with a power of two per token and block of 32 for the activations, which come from
// `A` again; a block's scale and its token's factor are one power of two.  Adds to the sums.
__device__ __noinline__ float4 careful_span(uint32_t w, uint32_t flip, uint2 s0, uint2 s1, const uint16_t* A, int T, int K, int k0,
                                            float4 tot) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint16_t* row = A + static_cast<int64_t>(min(g, T - 1)) * K;
  const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int b = 0; b < 8; ++b) {
    const int k = k0 + 32 * b + 8 * c;
    const uint4 raw = k < K ? __ldg(reinterpret_cast<const uint4*>(row + k)) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t m = __vmaxu2(__vmaxu2(raw.x & 0x7FFF7FFFu, raw.y & 0x7FFF7FFFu), __vmaxu2(raw.z & 0x7FFF7FFFu, raw.w & 0x7FFF7FFFu));
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const int e = min(126, max(-120, 13 + 127 - static_cast<int>(m >> 7)));
    const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t a[4], h0[4], h1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = pack_f16x2(bf16_lo(r[j]) * up, bf16_hi(r[j]) * up);
    const uint32_t off = static_cast<uint32_t>(b << 4) ^ flip;
    e2m1x8_f16(lds32(w + off), h0);
    e2m1x8_f16(lds32(w + off + 1024), h1);
    float d[4];
    mma_f16(d, h0[0], h1[0], h0[1], h1[1], a[0], a[1], zero);
    mma_f16(d, h0[2], h1[2], h0[3], h1[3], a[2], a[3], d);
    const int shift = 8 * (b & 3);
    const int x0 = static_cast<int>(((b < 4 ? s0.x : s0.y) >> shift) & 0xFFu), x1 = static_cast<int>(((b < 4 ? s1.x : s1.y) >> shift) & 0xFFu);
    const int ea = __shfl_sync(0xFFFFFFFFu, e, 8 * c) + 127, eb = __shfl_sync(0xFFFFFFFFu, e, 8 * c + 4) + 127;
    const float nan = __uint_as_float(0x7FC00000u);
    tot.x += x0 == 255 ? nan : times_pow2(d[0], x0 - ea);
    tot.y += x0 == 255 ? nan : times_pow2(d[1], x0 - eb);
    tot.z += x1 == 255 ? nan : times_pow2(d[2], x1 - ea);
    tot.w += x1 == 255 ? nan : times_pow2(d[3], x1 - eb);
  }
  return tot;
}

template <int CL>
__global__ void __launch_bounds__(kThreads, 1) mxfp4_dec_kernel(const __grid_constant__ CUtensorMap tmW, const DecParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* slots = reinterpret_cast<float*>(smem + p.stages * kRingBytes);  // [kSlots][16 rows][8 tokens]
  float* sums = slots + kSlots * 128;                               // [kPassTiles][16][8]
  DecCtl* ctl = reinterpret_cast<DecCtl*>(sums + kPassTiles * 128);
  float* factor = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ctl) + 1024);  // [spans_cta][8 tokens]
  uint8_t* act = reinterpret_cast<uint8_t*>(factor + p.spans_cta * 8);              // [span][block][T][64 bytes]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster = static_cast<int>(blockIdx.x) / CL, clusters = static_cast<int>(gridDim.x) / CL;
  const int s0 = min(p.spans, rank * p.spans_cta), s1 = min(p.spans, s0 + p.spans_cta);
  const int C = s1 - s0;
  const int tile0 = static_cast<int>(static_cast<int64_t>(p.tiles) * cluster / clusters);
  const int tile1 = static_cast<int>(static_cast<int64_t>(p.tiles) * (cluster + 1) / clusters);
  const int stages = p.stages;
  uint8_t* ring = smem + warp * stages * kBoxBytes;
  const int blocks_row = p.K / 32;

  if (threadIdx.x == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < kStagesMax; ++s) mbar_init(&ctl->full[w][s], 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
  }
  __syncthreads();

  uint32_t stage = 0, phase = 0;
  bool alive = true;
  for (int pass = tile0; pass < tile1; pass += kPassTiles) {
    const int nt = min(kPassTiles, tile1 - pass);
    const int U = nt * C;
    const int u0 = U * warp / kWarps, u1 = U * (warp + 1) / kWarps;
    // unit u: tile pass + u / C, span s0 + u % C; the copies' own place runs ahead of the sums'
    int next = u0, i_tile = C > 0 ? u0 / C : 0, i_span = C > 0 ? u0 % C : 0;
    auto issue = [&](uint32_t st) {
      const int row = (pass + i_tile) * kRows, sp = s0 + i_span;
      if (lane == 0) {
        mbar_arrive_expect_tx(&ctl->full[warp][st], kBoxBytes);
        tma_load_2d(ring + st * kBoxBytes, &tmW, &ctl->full[warp][st], sp * 32, row);
      }
      // the scales are read later: bring them into L2 with the codes (32 bytes are four spans)
      if ((next == u0 || (sp & 3) == 0) && lane < kRows && row + lane < p.N)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.scales + static_cast<int64_t>(row + lane) * blocks_row + sp * 8));
      ++next;
      if (++i_span == C) {
        i_span = 0;
        ++i_tile;
      }
    };
    uint32_t ahead = stage;
    if (alive) {
      for (int i = 0; i < stages && next < u1; ++i) {
        issue(ahead);
        ahead = ahead + 1 == stages ? 0 : ahead + 1;
      }
    }
    if (pass == tile0) {
      // this CTA's activations to f16, a warp per (span, token): 8 values a lane
      const int items = C * p.T;
      constexpr int kBatch = 8;
      for (int i0 = warp; i0 < items; i0 += kWarps * kBatch) {
        uint4 raw[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int i = i0 + b * kWarps, sp = i / p.T, t = i - sp * p.T;
          const int k = (s0 + sp) * kSpan + 8 * lane;
          raw[b] = i < items && k < p.K ? __ldg(reinterpret_cast<const uint4*>(p.A + static_cast<int64_t>(t) * p.K + k))
                                        : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int i = i0 + b * kWarps, sp = i / p.T, t = i - sp * p.T;
          uint32_t m = __vmaxu2(__vmaxu2(raw[b].x & 0x7FFF7FFFu, raw[b].y & 0x7FFF7FFFu),
                                __vmaxu2(raw[b].z & 0x7FFF7FFFu, raw[b].w & 0x7FFF7FFFu));
          m = max(m & 0xFFFFu, m >> 16);
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          const uint32_t block = m;  // four lanes hold a block of 32
          m = __reduce_max_sync(0xFFFFFFFFu, m);
          const bool far = __any_sync(0xFFFFFFFFu, block != 0u && (m >> 7) - (block >> 7) > kFarBlock);
          if (i >= items) continue;
          const int e = min(126, max(-120, 13 + 127 - static_cast<int>(m >> 7)));
          const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
          const uint32_t r[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = pack_f16x2(bf16_lo(r[j]) * up, bf16_hi(r[j]) * up);
          *reinterpret_cast<uint4*>(act + ((sp * 8 + (lane >> 2)) * p.T + t) * 64 + (lane & 3) * 16) =
              make_uint4(h[0], h[1], h[2], h[3]);
          if (lane == 0) factor[sp * 8 + t] = (far ? -1.0f : 1.0f) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // negative: careful_span
        }
      }
      // columns past the last token: a factor that keeps their sums finite
      for (int i = threadIdx.x; i < C * 8; i += kThreads)
        if (i % 8 >= p.T) factor[i] = 0.0f;
      __syncthreads();
    }

    float tot[4] = {0.f, 0.f, 0.f, 0.f};
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t act_lane = smem_u32(act) + min(g, p.T - 1) * 64 + c * 16;
    const uint32_t act_block = p.T * 64;
    const uint32_t lane_off = g * 128 + c * 4, flip = g << 4;
    int tl = C > 0 ? u0 / C : 0, sp = C > 0 ? u0 % C : 0;
    const uint8_t* rows[2];  // this lane's two rows of scales, at the CTA's first span
    auto set_rows = [&](int tile) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        rows[h] = p.scales + static_cast<int64_t>(min((pass + tile) * kRows + g + 8 * h, p.N - 1)) * blocks_row + s0 * 8;
    };
    auto load_scales = [&](int span, uint2 (&sc)[2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* src = rows[h] + span * 8;
        if (p.wide) {
          sc[h] = __ldg(reinterpret_cast<const uint2*>(src));
        } else {
          uint32_t v[2] = {0u, 0u};
#pragma unroll
          for (int b = 0; b < 8; ++b)
            if ((s0 + span) * 8 + b < blocks_row) v[b >> 2] |= static_cast<uint32_t>(__ldg(src + b)) << (8 * (b & 3));
          sc[h] = make_uint2(v[0], v[1]);
        }
      }
    };
    uint2 sc[2], sn[2];
    if (u0 < u1) {
      set_rows(tl);
      load_scales(sp, sc);
    }
    for (int u = u0; alive && u < u1; ++u) {
      const bool last = sp == C - 1;
      sn[0] = sc[0];
      sn[1] = sc[1];
      if (u + 1 < u1) {  // the next unit's scales, while this one is summed
        if (last) set_rows(tl + 1);
        load_scales(last ? 0 : sp + 1, sn);
      }
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->full[warp][stage], phase, &ctl->abort_flag))) {
        alive = false;
        // copies in flight land before the block may end
        uint32_t st = stage, ph = phase;
        for (int i = u; i < next; ++i) {
          mbar_wait_drain(&ctl->full[warp][st], ph);
          if (++st == stages) {
            st = 0;
            ph ^= 1u;
          }
        }
        break;
      }
      const uint32_t w = smem_u32(ring + stage * kBoxBytes) + lane_off;
      uint32_t ab = act_lane + sp * 8 * act_block;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t bf[2] = {0u, 0u};
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const uint32_t off = static_cast<uint32_t>(b << 4) ^ flip;
        const uint32_t x0 = lds32(w + off), x1 = lds32(w + off + 1024);
        const uint4 a = lds128(ab);
        ab += act_block;
        float d[4];
        uint32_t h0[4], h1[4];
        e2m1x8_f16(x0, h0);
        e2m1x8_f16(x1, h1);
        mma_f16(d, h0[0], h1[0], h0[1], h1[1], a.x, a.y, zero);
        mma_f16(d, h0[2], h1[2], h0[3], h1[3], a.z, a.w, d);
        if ((b & 1) == 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) bf[h] = e8m0x2_bf16((b < 4 ? sc[h].x : sc[h].y) >> (8 * (b & 2)));
        }
        const float f0 = (b & 1) ? bf16_hi(bf[0]) : bf16_lo(bf[0]), f1 = (b & 1) ? bf16_hi(bf[1]) : bf16_lo(bf[1]);
        acc[0] = fmaf(d[0], f0, acc[0]);
        acc[1] = fmaf(d[1], f0, acc[1]);
        acc[2] = fmaf(d[2], f1, acc[2]);
        acc[3] = fmaf(d[3], f1, acc[3]);
      }
      const float2 fa = *reinterpret_cast<const float2*>(factor + sp * 8 + 2 * c);
      if (__any_sync(0xFFFFFFFFu, !(max_mag4(acc) <= 3.4028235e38f) || fminf(fa.x, fa.y) < 0.0f)) {
        const float4 t = careful_span(w, flip, sc[0], sc[1], p.A, p.T, p.K, (s0 + sp) * kSpan, make_float4(tot[0], tot[1], tot[2], tot[3]));
        tot[0] = t.x;
        tot[1] = t.y;
        tot[2] = t.z;
        tot[3] = t.w;
      } else {
        tot[0] = fmaf(acc[0], fa.x, tot[0]);
        tot[1] = fmaf(acc[1], fa.y, tot[1]);
        tot[2] = fmaf(acc[2], fa.x, tot[2]);
        tot[3] = fmaf(acc[3], fa.y, tot[3]);
      }
      __syncwarp();  // the slot has been read
      if (next < u1) issue(stage);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
      sc[0] = sn[0];
      sc[1] = sn[1];
      if (last || u + 1 == u1) {  // this warp's part of the tile ends
        float* slot = slots + (tl + warp) * 128;
        *reinterpret_cast<float2*>(slot + g * 8 + 2 * c) = make_float2(tot[0], tot[1]);
        *reinterpret_cast<float2*>(slot + (g + 8) * 8 + 2 * c) = make_float2(tot[2], tot[3]);
        tot[0] = tot[1] = tot[2] = tot[3] = 0.f;
      }
      if (++sp == C) {
        sp = 0;
        ++tl;
      }
    }
    __syncthreads();
    auto emit = [&](int i, float v) {  // i: tile of the pass, token, row
      const int row = (pass + i / 128) * kRows + i % 16, t = (i / 16) % 8;
      if (t < p.T && row < p.N) p.out[static_cast<int64_t>(t) * p.N + row] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    };
    for (int i = threadIdx.x; i < nt * 128; i += kThreads) {
      const int tl = i / 128, e = (i % 16) * 8 + (i / 16) % 8;  // row, token
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int a = max(U * w / kWarps, tl * C), b = min(U * (w + 1) / kWarps, tl * C + C);
        if (a < b) v += slots[(tl + w) * 128 + e];
      }
      if (CL == 1) emit(i, v);
      else sums[i] = v;
    }
    if (CL > 1) {
      cluster_sync_all();
      for (int i = threadIdx.x + rank * kThreads; i < nt * 128; i += kThreads * CL) {
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < CL; ++r) {
          float x;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(mapa_shared(smem_u32(sums + i), r)) : "memory");
          v += x;
        }
        emit(i, v);
      }
      cluster_sync_all();  // the sums stay until every CTA has read them
    } else {
      __syncthreads();  // the slots are free again
    }
  }
}

template <int CL>
cudaError_t launch(const CUtensorMap& tmW, const DecParams& p, int smem, cudaStream_t stream) {
  auto kern = mxfp4_dec_kernel<CL>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), 227 * 1024, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // clusters that are resident at once (by the GPCs' sizes; the same for every call of a device)
  static std::atomic<int> resident[64];
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int clusters = dev < 64 ? resident[dev].load(std::memory_order_relaxed) : 0;
  if (clusters == 0) {
    cfg.gridDim = dim3(num_sms() / CL * CL);
    cfg.dynamicSmemBytes = kSmemMax;
    e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) resident[dev].store(clusters, std::memory_order_relaxed);
  }
  if (clusters > p.tiles) clusters = p.tiles;
  cfg.gridDim = dim3(clusters * CL);
  cfg.dynamicSmemBytes = smem;
  LaunchScope scope(stream, CL == 1 ? "mxfp4_dec_kernel" : CL == 2 ? "mxfp4_dec_kernel<split2>" : "mxfp4_dec_kernel<split4>");
  e = cudaLaunchKernelEx(&cfg, kern, tmW, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_mxfp4_dec(const uint16_t* A, int T, const uint8_t* codes, const uint8_t* scales, int N, int K,
                             uint16_t* out, cudaStream_t stream) {
  if (T < 1 || T > 8) return cudaErrorNotSupported;
  DecParams p{};
  p.A = A;
  p.scales = scales;
  p.out = out;
  p.T = T;
  p.N = N;
  p.K = K;
  p.spans = static_cast<int>((static_cast<int64_t>(K) + kSpan - 1) / kSpan);
  p.tiles = static_cast<int>((static_cast<int64_t>(N) + kRows - 1) / kRows);
  p.wide = K % kSpan == 0;
  // CTAs that share k.  A cluster's row tiles come in whole numbers, so more CTAs to a cluster balance better and
  // each holds fewer of the activations; meeting in distributed shared memory costs about what 22 units do (2 of
  // 45 us at 392 units).  8 tokens through 4096 x 4096: 12.0 us with two, 10.6 alone; one token is 10.5 either
  // way, the host's time for a call.
  auto act = [&](int n) { return static_cast<int64_t>((p.spans + n - 1) / n) * (T * 512 + 32); };
  int cl = 0;
  int64_t best = INT64_MAX;
  for (int n = 1; n <= 4 && n <= p.spans; n *= 2) {
    if (act(n) > kActBytesMax) continue;
    const int clusters = num_sms() / n;
    const int64_t cost = static_cast<int64_t>((p.tiles + clusters - 1) / clusters) * ((p.spans + n - 1) / n) + (n > 1 ? 22 : 0);
    if (cost < best) {
      best = cost;
      cl = n;
    }
  }
  if (cl == 0) return cudaErrorNotSupported;
  p.spans_cta = (p.spans + cl - 1) / cl;
  const int act_bytes = static_cast<int>(act(cl));
  p.stages = (kSmemMax - kFixedBytes - act_bytes) / kRingBytes;
  if (p.stages > kStagesMax) p.stages = kStagesMax;
  const int smem = kFixedBytes + p.stages * kRingBytes + act_bytes;
  CUtensorMap tmW;
  cudaError_t e = make_tmap_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, codes, static_cast<uint64_t>(N),
                               static_cast<uint64_t>(K) / 8, 32, kRows, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  return cl == 1 ? launch<1>(tmW, p, smem, stream) : cl == 2 ? launch<2>(tmW, p, smem, stream) : launch<4>(tmW, p, smem, stream);
}

}  // namespace ar
