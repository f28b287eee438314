// Attention over the paged 8-bit cache on the fifth-generation tensor cores (tcgen05), head
// dimension 128, for calls with enough rows to fill the GPU with tiles of 128 (prompts and pieces
// of prompts).  The method is attn_kv8_kernel's (ar_attn_kv8.cu): f16 operands, queries normalised
// by a power of two per row, the caches' scales taken into the softmax's exponent,
//   u = z log2(e) + e_v,  P' = 2^(u - m),  O = sum P' v',  l = sum P' 2^-e_v.
//
// One CTA per 128 rows (new token, head of the group) of one sequence and key/value head, over
// blocks of 128 keys.  Warp roles:
//  * 0: tensor memory; one lane issues S = Q K^T (M = 128 rows, N = 128 keys, K = 128).
//  * 1: one lane issues O += P V (A = P as f16 pairs in tensor memory, B = V MN-major).
//  * 2-17: softmax.  Warp w reads TMEM lanes 32 (w % 4) .. (a row a thread) and a quarter of the block's
//    keys; the four warps of a row exchange their maxima through shared memory (a bounded barrier).
//    The reference m only moves when a block's maximum passes it by 2^8, which f16 holds with room:
//    O is then rescaled in tensor memory, which almost no block needs after the first.
//  * 18-25: expansion.  Codes come straight from the pages to registers a block ahead, each
//    conversion instruction makes two f16, and the tile is written as the MMAs read it (128-byte
//    swizzle; the same layout serves K as the K-major and V as the MN-major operand).
//
// A block of 128 x 128 costs 1024 cycles of MMAs and the same of exponentials (16 a cycle and SM):
// the two overlap, so half the tensor rate is what exponentials leave.  2 x 512 new tokens of 4000, 64 heads
// over 8: 199 us, 412 TFLOP/s, tensor pipe 20 %; a block takes 3900 cycles, because the softmax warps of a block
// wait for one another's maxima and so reach their exponentials together.  Eight softmax warps 258 us; the
// mma.sync kernel 587 us.
// TMEM columns: S buffers [0, 256), P buffers [256, 384), O [384, 512).
#include "ar_attn_tc.cuh"

namespace ar {
namespace {

constexpr int kD = 128;
constexpr int kBlk = 128;                 // rows of a tile, keys of a block
constexpr int kBox = kBlk * 128;          // 128 rows x 64 f16
constexpr int kTile = 2 * kBox;
constexpr int kSmWarps = 16;
constexpr int kPerQ = kSmWarps / 4;       // softmax warps of a row
constexpr int kSmWarp0 = 2;
constexpr int kExWarps = 8;
constexpr int kExWarp0 = kSmWarp0 + kSmWarps;
constexpr int kExThreads = kExWarps * 32;
constexpr int kThreads = (kExWarp0 + kExWarps) * 32;
constexpr int kCols = kBlk / kPerQ;       // keys of a block, and columns of O, of a softmax warp
static_assert(kCols == 32, "a softmax warp loads and stores 32-column slices");
constexpr int kGroups = kCols / 16;       // of 16 tokens: one scale each
constexpr uint32_t kColS = 0, kColP = 256, kColO = 384;
constexpr float kSlack = 8.0f;            // a block's maximum may pass the reference by 2^8
constexpr int kRowsPerThread = kBlk * 8 / kExThreads;  // 16-byte pieces of a tile a thread expands

struct Ctl {
  uint64_t q_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2];
  uint64_t ex_full[4][2];                 // maxima of a lane quarter's warps
  uint64_t o_full, done_s, done_pv;
  uint32_t tmem_base;
  int abort_flag;
  float ex[2][4][kPerQ][32];              // [block parity][quarter][part][row]
  float fac[kBlk];                        // a row's factor to log2 units
};

constexpr int kSmem = 5 * kTile + static_cast<int>(sizeof(Ctl)) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");

struct Params {
  Kv8Args a;
  const uint16_t* q;
  const uint8_t *k, *v, *ks, *vs;
  uint16_t* out;
  float* lse;
  float scale_log2;
  int page_shift;
};

// f16 operands, fp32 sums
__host__ __device__ constexpr uint32_t idesc_f16(bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(kBlk >> 3) << 17) | (static_cast<uint32_t>(kBlk >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  uint32_t r[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[16 * h + i]);
    at_tmem_st16(taddr + 16 * h, r);
  }
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// place of 16-byte chunk c (of 16: 8 dimensions each) of row r in a swizzled tile of two boxes
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return static_cast<uint32_t>((c >> 3) * kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__global__ void __launch_bounds__(kThreads, 1) attn_kv8_tc_kernel(const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sK = sQ + kTile;
  uint8_t* sV = sK + 2 * kTile;
  Ctl* ctl = reinterpret_cast<Ctl*>(sV + 2 * kTile);
  volatile int* abort_flag = &ctl->abort_flag;
  const Kv8Args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.y, s = blockIdx.z;
  const int group = a.n_heads / a.n_kv;

  // the sequence's bounds, checked against the arrays (a sequence that does not fit is not touched)
  const int64_t c0 = a.cu[s], new64 = a.cu[s + 1] - c0, len64 = a.lens[s];
  const bool fits = new64 >= 0 && new64 <= a.max_new && c0 >= 0 && c0 + new64 <= a.T && len64 >= 0 &&
                    len64 <= static_cast<int64_t>(a.max_pages) * a.page;
  if (!fits) {
    if (threadIdx.x == 0) raise_status(kStatusBadIndex);
    return;
  }
  const int n_new = static_cast<int>(new64), len = static_cast<int>(len64), first = static_cast<int>(c0);
  const int n_rows = n_new * group;
  const int tiles = (n_rows + kBlk - 1) / kBlk;
  if (static_cast<int>(blockIdx.x) >= tiles) return;
  const int row0 = (tiles - 1 - static_cast<int>(blockIdx.x)) * kBlk;  // the longest rows first
  const int start = len - n_new;
  const int keys = max(0, start + min(n_rows - 1, row0 + kBlk - 1) / group + 1);  // that the tile's last row sees
  const int n_kb = (keys + kBlk - 1) / kBlk;
  const int full_below = start + row0 / group + 1;                                // tokens that every row sees
  const int32_t* table = a.table + static_cast<int64_t>(s) * a.max_pages;

  if (threadIdx.x == 0) {
    mbar_init(&ctl->q_full, kExWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->k_full[i], kExWarps);
      mbar_init(&ctl->k_empty[i], 1);
      mbar_init(&ctl->v_full[i], kExWarps);
      mbar_init(&ctl->v_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->s_empty[i], kSmWarps);
      mbar_init(&ctl->p_full[i], kSmWarps);
      mbar_init(&ctl->p_empty[i], 1);
      for (int q = 0; q < 4; ++q) mbar_init(&ctl->ex_full[q][i], kPerQ);
    }
    mbar_init(&ctl->o_full, 1);
    mbar_init(&ctl->done_s, 1);
    mbar_init(&ctl->done_pv, 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16(false);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
      bool ok = mbar_wait(&ctl->q_full, 0, abort_flag);
      tc_fence_after();
      for (int j = 0; ok && j < n_kb; ++j) {
        const int b = j & 1;
        if (!mbar_wait(&ctl->k_full[b], (j >> 1) & 1, abort_flag) || !mbar_wait(&ctl->s_empty[b], ((j >> 1) & 1) ^ 1, abort_flag)) break;
        tc_fence_after();
        const uint64_t k_desc = sdesc_sw128(smem_u32(sK + b * kTile), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kBox + (kk & 3) * 32;
          umma_bf16(tmem + kColS + b * kBlk, at_desc_add(q_desc, off), at_desc_add(k_desc, off), idesc, kk > 0 ? 1u : 0u);
        }
        umma_commit(&ctl->s_full[b]);
        umma_commit(&ctl->k_empty[b]);
      }
      umma_commit(&ctl->done_s);  // every MMA issued completes before tensor memory is released
      mbar_wait_drain(&ctl->done_s, 0);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ P V issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16(true);
      bool ok = true;
      for (int j = 0; ok && j < n_kb; ++j) {
        const int b = j & 1;
        ok = mbar_wait(&ctl->p_full[b], (j >> 1) & 1, abort_flag) && mbar_wait(&ctl->v_full[b], (j >> 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint64_t v_desc = sdesc_sw128(smem_u32(sV + b * kTile), kBox, 1024);
#pragma unroll
        for (int kk = 0; kk < kBlk / 16; ++kk)
          at_mma_ta(tmem + kColO, tmem + kColP + b * 64 + 8 * kk, at_desc_add(v_desc, kk * 2048), idesc, (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&ctl->p_empty[b]);
        umma_commit(&ctl->v_empty[b]);
      }
      if (ok) umma_commit(&ctl->o_full);
      umma_commit(&ctl->done_pv);
      mbar_wait_drain(&ctl->done_pv, 0);
    }
  } else if (warp < kExWarp0) {
    // ------------------------------------------------------------ softmax and output
    const int quarter = warp & 3, sub = (warp - kSmWarp0) >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int k0 = sub * kCols;
    const int rr = row0 + r;
    const int lim = rr < n_rows ? start + rr / group + 1 : 0;  // keys the row sees
    // lane i < kGroups looks up group i of a block: page two blocks ahead, scale codes one block ahead
    auto page_of = [&](int j) {
      const int t = j * kBlk + k0 + 16 * lane;
      return lane < kGroups && t < keys ? __ldg(table + (t >> p.page_shift)) : -1;
    };
    auto exps_of = [&](int pg) {
      if (pg < 0 || pg >= a.n_pages) return -1;
      const int64_t ph = static_cast<int64_t>(pg) * a.n_kv + head;
      return static_cast<int>(__ldg(p.ks + ph)) | (static_cast<int>(__ldg(p.vs + ph)) << 8);
    };
    int pg_next = page_of(1);
    int exps = exps_of(page_of(0)), exps_next = -1;
    bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->q_full, 0, abort_flag));
    const float fac = ctl->fac[r];
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; ok && j < n_kb; ++j) {
      const int b = j & 1;
      const uint32_t par = static_cast<uint32_t>(j >> 1) & 1u;
      exps_next = exps_of(pg_next);
      pg_next = page_of(j + 2);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->s_full[b], par, abort_flag));
      if (!ok) break;
      tc_fence_after();
      float x[kCols];
      tmem_ld32(tmem + lane_off + kColS + b * kBlk + k0, x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->s_empty[b]);
      float back[kGroups];
      float top = -INFINITY;
      const int tb = j * kBlk + k0;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int e = __shfl_sync(0xFFFFFFFFu, exps, g);
        const uint32_t ek = static_cast<uint32_t>(e) & 0xFFu, ev = (static_cast<uint32_t>(e) >> 8) & 0xFFu;
        const float f = fac * __uint_as_float(max(min(ek, 254u), 1u) << 23);
        const float fe = static_cast<float>(static_cast<int>(ev) - 127);
        back[g] = __uint_as_float(max(254u - min(ev, 253u), 1u) << 23);  // 2^-ev
        const int o = 16 * g;
        const int end = e < 0 ? 0 : lim;  // a group whose page is not in the pool, or past the keys: nothing
        if (tb + 16 * g + 16 > full_below || e < 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[o + i] = tb + 16 * g + i < end ? fmaf(x[o + i], f, fe) : -INFINITY;
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 v = fma2(make_float2(x[o + i], x[o + i + 1]), make_float2(f, f), make_float2(fe, fe));
            x[o + i] = v.x;
            x[o + i + 1] = v.y;
          }
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) top = max3(top, x[o + i], x[o + i + 1]);
      }
      exps = exps_next;
      // the row's maximum over all parts
      ctl->ex[b][quarter][sub][lane] = top;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->ex_full[quarter][b]);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->ex_full[quarter][b], par, abort_flag));
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kPerQ; ++i) top = fmaxf(top, ctl->ex[b][quarter][i][lane]);
      // all warps of a row come to the same decision
      const bool move = top > m + kSlack || (m == -INFINITY && top > -INFINITY);
      if (__any_sync(0xFFFFFFFFu, move)) {
        const float to = move ? top : m;
        const float f = m == -INFINITY ? 1.0f : at_ex2(m - to);  // nothing summed yet where m is -inf
        l *= f;
        m = to;
        if (j > 0) {
          // O holds the blocks before: wait for the last of their products, rescale this warp's 32 columns
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->p_empty[b ^ 1], static_cast<uint32_t>((j - 1) >> 1) & 1u, abort_flag));
          if (!ok) break;
          tc_fence_after();
          float o[kCols];
          tmem_ld32(tmem + lane_off + kColO + k0, o);
#pragma unroll
          for (int i = 0; i < kCols; ++i) o[i] *= f;
          tmem_st32(tmem + lane_off + kColO + k0, o);
          at_tmem_st_wait();
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      uint32_t pk[kCols / 2];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 d = add2(make_float2(x[16 * g + 2 * i], x[16 * g + 2 * i + 1]), make_float2(-ref, -ref));
          const float2 e = make_float2(at_ex2(d.x), at_ex2(d.y));
          sum = add2(sum, e);
          pk[8 * g + i] = pack_f16x2(e.x, e.y);
        }
        l = fmaf(sum.x + sum.y, back[g], l);
      }
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->p_empty[b], par ^ 1u, abort_flag));
      if (!ok) break;
      tc_fence_after();
      at_tmem_st16(tmem + lane_off + kColP + b * 64 + k0 / 2, pk);
      at_tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[b]);
    }
    // the row sum over all parts, through the same exchange (one phase further), added in their order
    const int b = n_kb & 1;
    ctl->ex[b][quarter][sub][lane] = l;
    __syncwarp();
    if (ok) {
      if (lane == 0) mbar_arrive(&ctl->ex_full[quarter][b]);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->ex_full[quarter][b], static_cast<uint32_t>(n_kb >> 1) & 1u, abort_flag));
    }
    if (ok && n_kb > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->o_full, 0, abort_flag));
    if (ok) {
      tc_fence_after();
      l = 0.0f;
#pragma unroll
      for (int i = 0; i < kPerQ; ++i) l += ctl->ex[b][quarter][i][lane];
      const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
      const int tok = rr / group;
      const int64_t row = static_cast<int64_t>(first + tok) * a.n_heads + head * group + (rr - tok * group);
      float o[kCols];
      if (n_kb > 0) {
        tmem_ld32(tmem + lane_off + kColO + k0, o);
      } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) o[i] = 0.0f;
      }
      if (rr < n_rows) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + row * kD + k0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[i] = make_uint4(pack_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv), pack_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                              pack_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
        if (sub == 0 && p.lse) p.lse[row] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
      }
      tc_fence_before();
    }
  } else {
    // ------------------------------------------------------------ expansion
    const int tid = threadIdx.x - kExWarp0 * 32;
    // queries: two threads a row, 64 dimensions each
    {
      const int r = tid >> 1, part = tid & 1, rr = row0 + r;
      uint4 w[8];
      uint32_t mag = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (rr < n_rows) {
        const int tok = rr / group;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (static_cast<int64_t>(first + tok) * a.n_heads + head * group + (rr - tok * group)) * kD + part * 64);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __ldg(src + i);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu), __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu)));
      mag = max(mag & 0xFFFFu, mag >> 16);
      mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
      const int qe = min(126, max(-120, 13 + 127 - static_cast<int>(mag >> 7)));  // 2^qe q lies below 2^14
      const float up = __uint_as_float(static_cast<uint32_t>(qe + 127) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(sQ + chunk_at(r, part * 8 + i)) =
            make_uint4(pack_f16x2(bf16_lo(w[i].x) * up, bf16_hi(w[i].x) * up), pack_f16x2(bf16_lo(w[i].y) * up, bf16_hi(w[i].y) * up),
                       pack_f16x2(bf16_lo(w[i].z) * up, bf16_hi(w[i].z) * up), pack_f16x2(bf16_lo(w[i].w) * up, bf16_hi(w[i].w) * up));
      if (part == 0) ctl->fac[r] = __uint_as_float(static_cast<uint32_t>(127 - qe) << 23) * p.scale_log2;
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full);
    }
    // tiles: 16-byte piece tid % 8 of tokens tid / 8 + 32 i
    const int c16 = tid & 7, t0 = tid >> 3;
    int pg[kRowsPerThread];
    auto pages = [&](int j) {  // of block j, -1 past the keys
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        const int t = j * kBlk + t0 + 32 * i;
        pg[i] = t < keys ? __ldg(table + (t >> p.page_shift)) : -1;
      }
    };
    bool bad = false;
    int at[kRowsPerThread];  // row of the cache, of the block being loaded; -1: nothing
    const uint32_t to_lo = chunk_at(t0, 2 * c16), to_hi = chunk_at(t0, 2 * c16 + 1);  // 32 rows further: 4096 bytes further
    auto places = [&](int j) {
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        const int t = j * kBlk + t0 + 32 * i;
        const bool in = pg[i] >= 0 && pg[i] < a.n_pages;
        bad |= t < keys && !in;
        at[i] = in ? (((pg[i] * a.n_kv + head) << p.page_shift) + (t & (a.page - 1))) : -1;
      }
    };
    auto load = [&](const uint8_t* src, uint4 (&w)[kRowsPerThread]) {
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i)
        w[i] = at[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + c16 * 16 + static_cast<int64_t>(at[i]) * kD)) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto expand = [&](uint8_t* tile, const uint4 (&w)[kRowsPerThread]) {
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        uint4 lo, hi;
        e4m3x4_f16(w[i].x, lo.x, lo.y);
        e4m3x4_f16(w[i].y, lo.z, lo.w);
        e4m3x4_f16(w[i].z, hi.x, hi.y);
        e4m3x4_f16(w[i].w, hi.z, hi.w);
        *reinterpret_cast<uint4*>(tile + to_lo + 4096 * i) = lo;
        *reinterpret_cast<uint4*>(tile + to_hi + 4096 * i) = hi;
      }
      fence_async();
      __syncwarp();
    };
    uint4 wk[kRowsPerThread], wv[kRowsPerThread];
    if (n_kb > 0) {
      pages(0);
      places(0);
      load(p.k, wk);
      load(p.v, wv);
      pages(1);
    }
    for (int j = 0; j < n_kb; ++j) {
      const int b = j & 1;
      const uint32_t par = (static_cast<uint32_t>(j >> 1) & 1u) ^ 1u;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->k_empty[b], par, abort_flag))) break;
      expand(sK + b * kTile, wk);
      if (lane == 0) mbar_arrive(&ctl->k_full[b]);
      if (j + 1 < n_kb) {
        places(j + 1);
        load(p.k, wk);
      }
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->v_empty[b], par, abort_flag))) break;
      expand(sV + b * kTile, wv);
      if (lane == 0) mbar_arrive(&ctl->v_full[b]);
      if (j + 1 < n_kb) {
        load(p.v, wv);
        pages(j + 2);
      }
    }
    if (bad) raise_status(kStatusBadIndex);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

// Whether a call has row tiles of 128 enough for the kernel above.  It gives a tile to a CTA whatever its
// length, so it wants about a tile an SM; the other kernel splits few rows over their keys.
bool attn_kv8_tc_fits(const Kv8Args& a) {
  const int64_t group = a.n_heads / a.n_kv;
  if (a.head_dim != kD || a.S > 65535 || a.n_kv > 65535 || a.max_new * group < kBlk) return false;
  return (a.T * group + kBlk - 1) / kBlk * a.n_kv >= num_sms();
}

cudaError_t launch_attn_kv8_tc(const Kv8Args& a, const uint16_t* q, float sm_scale, const uint8_t* k_pages,
                               const uint8_t* v_pages, const uint8_t* k_scales, const uint8_t* v_scales, uint16_t* out,
                               float* lse, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.q = q;
  p.k = k_pages;
  p.v = v_pages;
  p.ks = k_scales;
  p.vs = v_scales;
  p.out = out;
  p.lse = lse;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  while ((1 << p.page_shift) < a.page) ++p.page_shift;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(attn_kv8_tc_kernel), kSmem, allowed);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (static_cast<int64_t>(a.max_new) * (a.n_heads / a.n_kv) + kBlk - 1) / kBlk;
  {
    LaunchScope scope(stream, "attn_kv8_tc_kernel");
    attn_kv8_tc_kernel<<<dim3(static_cast<unsigned>(tiles), a.n_kv, a.S), kThreads, kSmem, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace ar
