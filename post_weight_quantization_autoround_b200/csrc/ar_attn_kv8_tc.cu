// Attention over the paged 8-bit cache on the fifth-generation tensor cores (tcgen05), head
// dimension 128, for calls with enough rows to fill tiles of 128 (prompts and pieces of prompts).
// The method is attn_kv8_kernel's (ar_attn_kv8.cu): f16 operands, queries normalised
// by a power of two per row, the caches' scales taken into the softmax's exponent,
//   u = z log2(e) + e_v,  P' = 2^(u - m + 11),  O = sum P' v',  l = sum P' 2^(-e_v - 11).
//
// One CTA per 256 rows (new token, head of the group) of one sequence and key/value head, over blocks of
// 128 keys: two groups of warps with a tile of 128 rows each, which read the same expanded keys and values.
// A CTA with one tile only gives both groups that tile, by turns of blocks, and joins their sums at the end.
// Warp roles:
//  * 0, 1: the MMAs of a group, issued by one lane: S = Q K^T (M = 128 rows, N = 128 keys, K = 128), then
//    O += P V in two halves of the keys (A = P as f16 pairs in tensor memory, B = V MN-major).
//  * 2-9: softmax, a row a thread: warp w reads TMEM lanes 32 (w % 4) ...  S is read twice, for the row's
//    maximum and for the exponentials, which go back over S as P from the last keys down, where S has been
//    read.  The reference m only moves when a block's maximum passes it by 2^4: O is then rescaled in tensor
//    memory, which few blocks need after the first.  P' reaches 2^15 there, and 2^11 at a reference that
//    stays, so f16 is off by 2^-11 of a weight, or by 2^-36 of the row's largest where that is more (behind a
//    key that takes nearly all weight and has a small value the others count all the same).  A wider margin
//    leaves less below: 2^8 took 144 us where 2^4 takes 148 and 2^2 152 (the case below).  A block with a
//    value scale 2^80 below another's has a second look at the weights that left fp32 (kFarCodes).
//  * 10-13: expansion.  Codes come straight from the pages to registers a block ahead, each
//    conversion instruction makes two f16, and the tile is written as the MMAs read it (128-byte
//    swizzle; the same layout serves K as the K-major and V as the MN-major operand).
//
// A tile's block of 128 keys costs 1024 cycles of MMAs and the same of exponentials (16 a cycle and SM).
// The two groups take turns at the exponentials, so that one's MMAs run under the other's; left alone they
// fall into step and both wait (184 us for the case below, 168 with the turns; 149 with two loads of S in
// flight and a chunk kept for the second reading).  2 x 512 new tokens of 4000, 64 heads over 8: 149 us
// in a loop of calls, 549 TFLOP/s.  Of a group's 4800 cycles a block the scores take a quarter, the maximum an eighth,
// the exponentials two fifths: shared memory, which the MMAs read at its full rate, slows all that
// goes through it.  One tile a CTA with sixteen softmax warps took 199 us, the mma.sync kernel 587 us; the
// scores held in registers (168 a thread, MMAs issued by a softmax warp) 204 us, two threads a row 188 us.
// TMEM columns: S and P of the groups [0, 256), O [256, 512).
#include <algorithm>
#include <type_traits>

#include "ar_attn_tc.cuh"

namespace ar {
namespace {

constexpr int kD = 128;
constexpr int kBlk = 128;                 // rows of a tile, keys of a block
constexpr int kCtaRows = 2 * kBlk;
constexpr int kBox = kBlk * 128;          // 128 rows x 64 f16
constexpr int kTile = 2 * kBox;
constexpr int kSmWarps = 8;               // two groups of four: a thread has a row of its group's tile
constexpr int kSmWarp0 = 2;
constexpr int kExWarps = 4;
constexpr int kExWarp0 = kSmWarp0 + kSmWarps;
constexpr int kExThreads = kExWarps * 32;
constexpr int kThreads = (kExWarp0 + kExWarps) * 32;
constexpr int kGroups = kBlk / 16;        // of 16 tokens: one scale each
constexpr uint32_t kColS = 0, kColO = 2 * kBlk;  // of group g: + 128 g; P lies over the upper half of S
constexpr uint32_t kColP = kColS + kBlk / 2;
constexpr int kSlack = 4;                 // a block's maximum may pass the reference by 2^4
constexpr int kShift = 15 - kSlack;       // P' at the reference; the largest is 2^15
constexpr float kUnshift = 1.0f / (1 << kShift);
// Where a group's value scale lies 2^80 below another's that the row has seen, weights below 2^-126 count for the row sum:
// 2^30 of them could be more than 2^-24 of it.
constexpr uint32_t kFarCodes = 80;
constexpr int kRowStep = kExThreads / 8;
constexpr int kRowsPerThread = kBlk / kRowStep;  // 16-byte pieces of a tile a thread expands

struct Ctl {
  uint64_t q_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2][2], pv_done[2], done[2];  // of a group; P in halves
  uint64_t turn[2][4];                    // of a group's warp: its partner's exponentials are done
  uint32_t tmem_base;
  int abort_flag;
  float fac[2 * kBlk];                    // a row's factor to log2 units
  float join[2][kBlk];                    // reference and sum of the second group's rows
};

constexpr int kSmem = 6 * kTile + static_cast<int>(sizeof(Ctl)) + 1024;
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

// 32 lanes x 32 columns from tensor memory, without waiting for them
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// 16 columns, waited for
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// the wait, which the values pass through, so that no use of them moves before it
__device__ __forceinline__ void ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
        "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
        "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
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

// Powers of a block's 16-token groups, group i's in lane i: of the keys' scale, the exponent of the values', its inverse.
struct Scales {
  float f, fe, back;
};
__device__ __forceinline__ float of_group(float v, int g) { return __shfl_sync(0xFFFFFFFFu, v, g); }

// 32 of a row's products: their largest u.  kMask: of tokens t0 .. t0 + 31, only those below `lim` count, and none of a group set in `bad`.
template <bool kMask>
__device__ __forceinline__ float chunk_max(const uint32_t (&x)[32], const Scales& c, float fac, int chunk, int t0, int lim, uint32_t bad, float top) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int g = 2 * chunk + h, n = (bad >> g) & 1 ? 0 : lim - t0 - 16 * h;  // the group's tokens that count
    float z = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      float a = __uint_as_float(x[16 * h + i]), b = __uint_as_float(x[16 * h + i + 1]);
      if (kMask) {
        a = i < n ? a : -INFINITY;
        b = i + 1 < n ? b : -INFINITY;
      }
      z = max3(z, a, b);
    }
    // f >= 0: the largest product has the largest u.  Where none counts f may be anything.
    const float f = fac * of_group(c.f, g), fe = of_group(c.fe, g);
    top = fmaxf(top, kMask && z == -INFINITY ? z : fmaf(z, f, fe));
  }
  return top;
}

// 32 of a row's exponentials as f16 pairs; returns their weighted sum added to l.
template <bool kMask>
__device__ __forceinline__ float chunk_exp(const uint32_t (&x)[32], const Scales& c, float fac, float ref, int chunk, int t0, int lim,
                                           uint32_t bad, float l, uint32_t (&pk)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int g = 2 * chunk + h, n = (bad >> g) & 1 ? 0 : lim - t0 - 16 * h;  // the group's tokens that count
    const float f1 = fac * of_group(c.f, g), fe1 = of_group(c.fe, g) - ref, back = of_group(c.back, g);
    const float2 f = make_float2(f1, f1), fe = make_float2(fe1, fe1);
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      float2 d = fma2(make_float2(__uint_as_float(x[16 * h + i]), __uint_as_float(x[16 * h + i + 1])), f, fe);
      if (kMask) {
        d.x = i < n ? d.x : -INFINITY;
        d.y = i + 1 < n ? d.y : -INFINITY;
      }
      const float2 e = make_float2(at_ex2(d.x), at_ex2(d.y));
      sum = add2(sum, e);
      pk[8 * h + i / 2] = pack_f16x2(e.x, e.y);
    }
    l = fmaf(sum.x + sum.y, back, l);
  }
  return l;
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
  uint8_t* sK = sQ + 2 * kTile;
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
  if (n_rows < a.split_rows) return;
  const int tiles = (n_rows + kCtaRows - 1) / kCtaRows;
  if (static_cast<int>(blockIdx.x) >= tiles) return;
  const int row0 = (tiles - 1 - static_cast<int>(blockIdx.x)) * kCtaRows;  // the longest rows first
  const int row_end = min(n_rows, row0 + kCtaRows);
  const bool two = row_end - row0 > kBlk;  // a tile a group; else both groups share one, by turns of blocks
  const int start = len - n_new;
  const int keys = max(0, start + (row_end - 1) / group + 1);  // that the last row sees
  const int n_kb = (keys + kBlk - 1) / kBlk;
  const int32_t* table = a.table + static_cast<int64_t>(s) * a.max_pages;

  if (threadIdx.x == 0) {
    mbar_init(&ctl->q_full, kExWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->k_full[i], kExWarps);
      mbar_init(&ctl->k_empty[i], two ? 2 : 1);
      mbar_init(&ctl->v_full[i], kExWarps);
      mbar_init(&ctl->v_empty[i], two ? 2 : 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i][0], 4);
      mbar_init(&ctl->p_full[i][1], 4);
      mbar_init(&ctl->pv_done[i], 1);
      mbar_init(&ctl->done[i], 1);
      for (int q = 0; q < 4; ++q) mbar_init(&ctl->turn[i][q], 1);
    }
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

  if (warp < kSmWarp0) {
    // ------------------------------------------------------------ a group's MMAs
    if (lane == 0) {
      const int g = warp;
      constexpr uint32_t idesc_s = idesc_f16(false), idesc_o = idesc_f16(true);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ + (two ? g : 0) * kTile), 16, 1024);
      const uint32_t col_s = tmem + kColS + g * kBlk, col_p = tmem + kColP + g * kBlk, col_o = tmem + kColO + g * kBlk;
      bool ok = mbar_wait(&ctl->q_full, 0, abort_flag);
      int i = 0;
      ok = ok && ((two ? 0 : g) >= n_kb || mbar_wait(&ctl->k_full[two ? 0 : g], 0, abort_flag));
      for (int j = two ? 0 : g; ok && j < n_kb; j += two ? 1 : 2, ++i) {
        const int b = j & 1;
        const uint32_t par = static_cast<uint32_t>(j >> 1) & 1u, own = static_cast<uint32_t>(i) & 1u;
        // S lies where P was: the products that read it have to be done
        ok = i == 0 || mbar_wait(&ctl->pv_done[g], own ^ 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint64_t k_desc = sdesc_sw128(smem_u32(sK + b * kTile), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kBox + (kk & 3) * 32;
          umma_bf16(col_s, at_desc_add(q_desc, off), at_desc_add(k_desc, off), idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit(&ctl->s_full[g]);
        umma_commit(&ctl->k_empty[b]);
        const int next = j + (two ? 1 : 2);  // its keys are looked at before P is there
        ok = (next >= n_kb || mbar_wait(&ctl->k_full[next & 1], static_cast<uint32_t>(next >> 1) & 1u, abort_flag)) && mbar_wait(&ctl->v_full[b], par, abort_flag);
        const uint64_t v_desc = sdesc_sw128(smem_u32(sV + b * kTile), kBox, 1024);
#pragma unroll
        for (int h = 1; h >= 0; --h) {  // the upper keys come first
          ok = ok && mbar_wait(&ctl->p_full[g][h], own, abort_flag);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
            at_mma_ta(col_o, col_p + 8 * kk, at_desc_add(v_desc, kk * 2048), idesc_o, (i > 0 || kk != 4) ? 1u : 0u);
        }
        if (!ok) break;
        umma_commit(&ctl->v_empty[b]);
        umma_commit(&ctl->pv_done[g]);
      }
      // every MMA issued completes before tensor memory is released
      umma_commit(&ctl->done[g]);
      mbar_wait_drain(&ctl->done[g], 0);
    }
  } else if (warp < kExWarp0) {
    // ------------------------------------------------------------ softmax and output
    const int g = (warp - kSmWarp0) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t col_s = lane_off + kColS + g * kBlk, col_p = lane_off + kColP + g * kBlk, col_o = lane_off + kColO + g * kBlk;
    const int tile0 = row0 + (two ? g * kBlk : 0);
    const int rr = tile0 + r;
    const int lim = rr < row_end ? start + rr / group + 1 : 0;  // keys the row sees
    const int full_below = start + tile0 / group + 1;          // tokens that every row of the tile sees
    const int step = two ? 1 : 2;
    // lane i < kGroups looks up group i of a block: page two of the group's blocks ahead, scale codes one
    auto page_of = [&](int j) {
      const int t = j * kBlk + 16 * lane;
      return lane < kGroups && t < keys ? __ldg(table + (t >> p.page_shift)) : -1;
    };
    uint32_t ek_next = 0, ev_next = 0;  // loaded here, first used a block later: nothing waits for them
    auto scales_of = [&](int pg) {
      const uint32_t ph = pg >= 0 && pg < a.n_pages ? static_cast<uint32_t>(pg) * a.n_kv + head : 0u;
      ek_next = __ldg(p.ks + ph);
      ev_next = __ldg(p.vs + ph);
    };
    int j = two ? 0 : g;
    int pg = page_of(j), pg_next = page_of(j + step);
    scales_of(pg);
    bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->q_full, 0, abort_flag));
    const float fac = ctl->fac[(two ? g * kBlk : 0) + r];
    float m = -INFINITY, l = 0.0f;
    int i = 0;
    uint32_t ev_top = 0;  // largest value scale code so far
    auto block = [&](auto mask, uint32_t ek, uint32_t ev, uint32_t bad, uint32_t far) {
      constexpr bool kMask = decltype(mask)::value;
      const uint32_t par = static_cast<uint32_t>(i) & 1u;
      Scales c;
      c.f = __uint_as_float(max(min(ek, 254u), 1u) << 23);
      c.fe = static_cast<float>(static_cast<int>(ev) - 127);
      c.back = e8m0_inverse(ev, kShift);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->s_full[g], par, abort_flag))) return false;
      tc_fence_after();
      const int t0 = j * kBlk;
      uint32_t xa[32], xb[32];
      float top = -INFINITY;
      ld32(col_s, xa);
      ld32(col_s + 32, xb);
      ld_wait(xa);
      ld_wait(xb);
      top = chunk_max<kMask>(xa, c, fac, 0, t0, lim, bad, top);
      ld32(col_s + 64, xa);
      top = chunk_max<kMask>(xb, c, fac, 1, t0 + 32, lim, bad, top);
      ld32(col_s + 96, xb);
      ld_wait(xa);
      ld_wait(xb);
      top = chunk_max<kMask>(xa, c, fac, 2, t0 + 64, lim, bad, top);
      top = chunk_max<kMask>(xb, c, fac, 3, t0 + 96, lim, bad, top);
      // one row's need moves the warp's other rows to their maxima too: they need it less often then
      if (__any_sync(0xFFFFFFFFu, top > m + kSlack || (m == -INFINITY && top > -INFINITY))) {
        const float to = fmaxf(m, top);
        const float half = m == -INFINITY ? 1.0f : at_ex2(0.5f * (m - to)), down = half * half;  // nothing summed yet where m is -inf
        l = l * half * half;
        m = to;
        if (i > 0) {  // O holds the blocks before: S came after the last of their products
#pragma unroll 1
          for (int q = 0; q < kD; q += 32) {
            uint32_t o[32], h[16];
            ld32(col_o + q, o);
            ld_wait(o);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
              for (int n = 0; n < 16; ++n) h[n] = __float_as_uint(__uint_as_float(o[16 * k + n]) * down);
              at_tmem_st16(col_o + q + 16 * k, h);
            }
          }
          at_tmem_st_wait();
        }
      }
      // The two warps of a scheduler take turns at the exponentials, so that one group's MMAs run meanwhile.
      if ((g == 1 || i > 0) && !__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->turn[g][quarter], par ^ (g == 0 ? 1u : 0u), abort_flag))) return false;
      const float ref = m == -INFINITY ? 0.0f : m - kShift;
      if (kMask && far != 0u) {  // before P overwrites S
#pragma unroll 1
        for (int h = 0; h < kGroups; ++h) {
          if (!((far >> h) & 1)) continue;
          uint32_t x[16];
          ld16(col_s + 16 * h, x);
          const float f = fac * of_group(c.f, h), fe = of_group(c.fe, h) - ref, back = of_group(c.back, h);
          float low = 0.0f;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const float d = fmaf(__uint_as_float(x[n]), f, fe);
            if (t0 + 16 * h + n < lim && d < -126.0f) low += at_ex2(d + 126.0f);
          }
          l = fmaf(low, back * 0x1p-126f, l);
        }
      }
      // From the last 32 keys down: a chunk's P goes where S has been read already.
      uint32_t pk[16];
      auto full = [&](int h) {
        at_tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[g][h]);
      };
      l = chunk_exp<kMask>(xb, c, fac, ref, 3, t0 + 96, lim, bad, l, pk);
      at_tmem_st16(col_p + 48, pk);
      ld32(col_s + 32, xb);
      l = chunk_exp<kMask>(xa, c, fac, ref, 2, t0 + 64, lim, bad, l, pk);
      at_tmem_st16(col_p + 32, pk);
      full(1);
      ld_wait(xb);
      ld32(col_s, xa);
      l = chunk_exp<kMask>(xb, c, fac, ref, 1, t0 + 32, lim, bad, l, pk);
      at_tmem_st16(col_p + 16, pk);
      ld_wait(xa);
      l = chunk_exp<kMask>(xa, c, fac, ref, 0, t0, lim, bad, l, pk);
      at_tmem_st16(col_p, pk);
      full(0);
      if (lane == 0) mbar_arrive(&ctl->turn[g ^ 1][quarter]);
      return true;
    };
    for (; ok && j < n_kb; j += step, ++i) {
      const uint32_t ek = ek_next, ev = ev_next;
      const uint32_t bad = __ballot_sync(0xFFFFFFFFu, lane < kGroups && (pg < 0 || pg >= a.n_pages));  // nothing of these
      // lanes without a group, and groups past the keys or of a page that is not in the pool, have no scale
      const uint32_t code = lane < kGroups && !((bad >> lane) & 1) ? ev : 0u;
      ev_top = max(ev_top, __reduce_max_sync(0xFFFFFFFFu, code));
      const uint32_t far = __ballot_sync(0xFFFFFFFFu, code != 0u && code + kFarCodes < ev_top);
      pg = pg_next;
      scales_of(pg);
      pg_next = page_of(j + 2 * step);
      if ((j + 1) * kBlk > full_below || bad != 0 || far != 0)
        ok = block(std::true_type{}, ek, ev, bad, far);
      else
        ok = block(std::false_type{}, ek, ev, 0u, 0u);
    }
    const bool any = i > 0;  // O has been written
    ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->done[g], 0, abort_flag));
    float down = 1.0f, other = 0.0f;  // factors of this group's sums and of the other's
    float* osum = reinterpret_cast<float*>(sK);  // [column][row], once no product reads the tiles any more
    if (!two && n_kb > 1) {
      // the second group's sums go to the first
      if (g == 1) {
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(&ctl->done[0], 0, abort_flag));
        if (ok) {
          tc_fence_after();
          ctl->join[0][r] = m;
          ctl->join[1][r] = l;
#pragma unroll 1
          for (int q = 0; q < kD; q += 32) {
            uint32_t o[32];
            ld32(col_o + q, o);
            ld_wait(o);
#pragma unroll
            for (int n = 0; n < 32; ++n) osum[(q + n) * kBlk + r] = __uint_as_float(o[n]);
          }
        }
      }
      at_bar_sync(1, kSmWarps * 32);
      if (g == 0 && *abort_flag == 0) {
        const float m1 = ctl->join[0][r], top = fmaxf(m, m1);
        const float half0 = m == -INFINITY ? 1.0f : at_ex2(0.5f * (m - top)), half1 = m1 == -INFINITY ? 1.0f : at_ex2(0.5f * (m1 - top));
        down = half0 * half0;
        other = half1 * half1;
        l = l * half0 * half0 + ctl->join[1][r] * half1 * half1;
        m = top;
      } else {
        ok = ok && g == 0;
      }
    }
    if (!two && g == 1) ok = false;  // the first group writes
    if (ok) {
      tc_fence_after();
      const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
      const int tok = rr / group;
      const int64_t row = static_cast<int64_t>(first + tok) * a.n_heads + head * group + (rr - tok * group);
#pragma unroll 1
      for (int q = 0; q < kD; q += 32) {
        uint32_t x[32];
        if (any) {
          ld32(col_o + q, x);
          ld_wait(x);
        }
        if (rr < row_end) {
          float o[32];
#pragma unroll
          for (int n = 0; n < 32; ++n) o[n] = any ? __uint_as_float(x[n]) * down : 0.0f;  // times 2^kShift
          if (!two && n_kb > 1) {
#pragma unroll
            for (int n = 0; n < 32; ++n) o[n] = fmaf(osum[(q + n) * kBlk + r], other, o[n]);
          }
#pragma unroll
          for (int n = 0; n < 32; ++n) o[n] *= kUnshift;
          uint4* dst = reinterpret_cast<uint4*>(p.out + row * kD + q);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_uint4(pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv), pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv), pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
        }
      }
      if (rr < row_end && p.lse) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;  // a NaN stays one
      tc_fence_before();
    }
  } else {
    // ------------------------------------------------------------ expansion
    const int tid = threadIdx.x - kExWarp0 * 32;
    // queries: two threads a row, 64 dimensions each
#pragma unroll 1
    for (int u = 0; u < (two ? 4 : 2); ++u) {
      const int tile = u >> 1, r = (u & 1) * (kBlk / 2) + (tid >> 1), part = tid & 1, rr = row0 + tile * kBlk + r;
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
        *reinterpret_cast<uint4*>(sQ + tile * kTile + chunk_at(r, part * 8 + i)) =
            make_uint4(pack_f16x2(bf16_lo(w[i].x) * up, bf16_hi(w[i].x) * up), pack_f16x2(bf16_lo(w[i].y) * up, bf16_hi(w[i].y) * up),
                       pack_f16x2(bf16_lo(w[i].z) * up, bf16_hi(w[i].z) * up), pack_f16x2(bf16_lo(w[i].w) * up, bf16_hi(w[i].w) * up));
      if (part == 0) ctl->fac[tile * kBlk + r] = __uint_as_float(static_cast<uint32_t>(127 - qe) << 23) * p.scale_log2;
    }
    fence_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->q_full);
    // tiles: 16-byte piece tid % 8 of tokens tid / 8 + 16 i
    const int c16 = tid & 7, t0 = tid >> 3;
    int pg[kRowsPerThread];
    auto pages = [&](int j) {  // of block j, -1 past the keys
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        const int t = j * kBlk + t0 + kRowStep * i;
        pg[i] = t < keys ? __ldg(table + (t >> p.page_shift)) : -1;
      }
    };
    bool bad = false;
    const uint32_t to_u = chunk_at(t0, 2 * c16 + (c16 >= 4)), to_v = chunk_at(t0, 2 * c16 + (c16 < 4));  // kRowStep rows further: the same chunk
    auto load = [&](const uint8_t* src, int j, uint4 (&w)[kRowsPerThread]) {
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        const int t = j * kBlk + t0 + kRowStep * i;
        const bool in = pg[i] >= 0 && pg[i] < a.n_pages;
        bad |= t < keys && !in;
        const int64_t at = ((static_cast<int64_t>(pg[i]) * a.n_kv + head) << p.page_shift) + (t & (a.page - 1));  // row of the cache
        w[i] = in ? __ldg(reinterpret_cast<const uint4*>(src + c16 * 16 + at * kD)) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    auto expand = [&](uint8_t* tile, const uint4 (&w)[kRowsPerThread]) {
#pragma unroll
      for (int i = 0; i < kRowsPerThread; ++i) {
        // The row's upper half stores its odd chunks first: eight threads then meet all banks once.
        const uint32_t a0 = c16 < 4 ? w[i].x : w[i].z, a1 = c16 < 4 ? w[i].y : w[i].w;
        const uint32_t b0 = c16 < 4 ? w[i].z : w[i].x, b1 = c16 < 4 ? w[i].w : w[i].y;
        uint4 u, v;
        e4m3x4_f16(a0, u.x, u.y);
        e4m3x4_f16(a1, u.z, u.w);
        e4m3x4_f16(b0, v.x, v.y);
        e4m3x4_f16(b1, v.z, v.w);
        *reinterpret_cast<uint4*>(tile + to_u + kRowStep * 128 * i) = u;
        *reinterpret_cast<uint4*>(tile + to_v + kRowStep * 128 * i) = v;
      }
      fence_async();
      __syncwarp();
    };
    uint4 wk[kRowsPerThread], wv[kRowsPerThread];
    if (n_kb > 0) {
      pages(0);
      load(p.k, 0, wk);
      load(p.v, 0, wv);
      pages(1);
    }
    for (int j = 0; j < n_kb; ++j) {
      const int b = j & 1;
      const uint32_t par = (static_cast<uint32_t>(j >> 1) & 1u) ^ 1u;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->k_empty[b], par, abort_flag))) break;
      expand(sK + b * kTile, wk);
      if (lane == 0) mbar_arrive(&ctl->k_full[b]);
      if (j + 1 < n_kb) {
        load(p.k, j + 1, wk);
      }
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->v_empty[b], par, abort_flag))) break;
      expand(sV + b * kTile, wv);
      if (lane == 0) mbar_arrive(&ctl->v_full[b]);
      if (j + 1 < n_kb) {
        load(p.v, j + 1, wv);
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

// How many of a call's sequences bring more than a few rows, as far as the host can tell: by the tokens that are
// left when every sequence has one.
int64_t attn_kv8_long_seqs(const Kv8Args& a) {
  if (a.n_heads / a.n_kv > 32 || a.max_new == 1 || a.T <= a.S) return a.S;
  return std::min<int64_t>(a.S, (a.T - a.S + a.max_new - 2) / (a.max_new - 1));
}

// Whether a call runs faster on the kernel above.  It takes 104 us for a wave of CTAs (256 rows of one sequence
// and head, or what is left of them: half a CTA a sequence on average) over 4000 keys; the other kernel, which splits
// the keys over the GPU, 37 us and 1.65 us for every tile of 128 rows.  The host does not know the lengths, so the rule
// takes both to grow alike with the keys; where they do not, the choice is the one for 4000.
// Measured (here against there), 64 heads over 8, one sequence of 4000: 64 new tokens 105 against 95 us, 100: 104
// against 124, 256: 102 against 249; 16 sequences of 33 new tokens, 32 heads over 4: 114 against 271.  This kernel
// with 100 new tokens of 1000: 37 us, of 30000: 660.  The other with 64 of 1000: 37, of 30000: 486.
// Short sequences next to long ones run on the other kernel, after this one.
bool attn_kv8_tc_fits(const Kv8Args& a) {
  const int64_t group = a.n_heads / a.n_kv;
  if (a.head_dim != kD || a.S > 65535 || a.n_kv > 65535 || a.max_new * group < kBlk) return false;
  const int64_t seqs = attn_kv8_long_seqs(a);
  const int64_t rows = std::max<int64_t>(a.T - (a.S - seqs), 1) * group;
  const int64_t tiles = (rows + kBlk - 1) / kBlk * a.n_kv;
  const int64_t ctas = (rows + kCtaRows - 1 + seqs * (kCtaRows / 2)) / kCtaRows * a.n_kv;
  const int64_t waves = (ctas + num_sms() - 1) / num_sms();
  return tiles + 22 >= 64 * waves;
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
  const int64_t tiles = (static_cast<int64_t>(a.max_new) * (a.n_heads / a.n_kv) + kCtaRows - 1) / kCtaRows;
  {
    LaunchScope scope(stream, "attn_kv8_tc_kernel");
    attn_kv8_tc_kernel<<<dim3(static_cast<unsigned>(tiles), a.n_kv, a.S), kThreads, kSmem, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace ar
