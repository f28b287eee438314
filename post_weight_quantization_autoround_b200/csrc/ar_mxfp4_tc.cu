// Product with MXFP4 weights on the fifth-generation tensor cores, for more tokens than the
// decode kernel takes: out[t][n] = sum_k A[t][k] 2^(s - 127) E2M1, bf16 activations.
//
// A weight's value is exact in bf16 (two significant bits times a power of two), so a tile of
// weights is expanded once, scale included, and one fp32 accumulator runs over all of K:
// nothing is rescaled in the middle of a sum.
//
//  * One CTA owns 128 weight rows (the MMA's M) and up to 256 tokens (its N): the expansion of
//    a weight serves 256 tokens, and at N = 256 the MMAs of a 64-k stage take 512 cycles, longer
//    than its expansion (at N = 128 the two are even).
//  * Sixteen warps expand (four sets in turn, each a stage; with two the chains of one warp set the pace, a warp per 32 TMEM lanes): the codes
//    of a stage are 32 bytes a row in shared memory (TMA, 128-byte swizzle), and the bf16 tile
//    goes straight to tensor memory as the MMA's A operand.  A code's sign and its three other
//    bits, moved to the sign and to the two lowest exponent bits and highest mantissa bit of a
//    bf16, are its value times 2^-126 (0.5 as a subnormal), and one bf16x2 product by
//    2^(126 + e) gives two weights: 4 integer operations a pair.  A stage with a scale above
//    2^1 or NaN goes by tables of the values' bytes instead.
//  * One thread issues tcgen05.mma (kind::f16, M = 128, N = tokens, K = 16), activations come by
//    TMA (128-byte swizzle).  Few tiles: the CTAs of a cluster split K and add their sums
//    through distributed shared memory in rank order.
//
// 256 tokens through 8192 x 28672: 112 us in a long loop of calls, under the power cap (1.08 PFLOP/s), 98-102 for
// single launches (1.18-1.22), tensor pipe 71 % (128 of 148 SMs have a CTA); 512 tokens 176 us, 1.37 PFLOP/s; 16 tokens 86 us, where a stage's chain of expansion, hand-over and
// release sets the pace.  128-token tiles with the scales applied the same way: 187 us at 256 tokens.
#include "ar_internal.h"

namespace ar {
namespace {

constexpr int kRows = 128;
constexpr int kStageK = 64;                  // k of a stage: 4 MMAs, 32 TMEM columns of A
constexpr int kStages = 4;                   // A in tensor memory, activations in shared memory
constexpr int kSlots = 4;                    // code boxes: 128 rows x 256 k, 4 stages each
constexpr int kSlotBytes = kRows * 128;
constexpr int kStagesPerSlot = 4;
constexpr int kACols = kStageK / 2;
constexpr int kFirstWorker = 4;              // warps: activation TMA, MMA, code TMA, idle, 16 workers
constexpr int kWorkers = 16;
constexpr int kSets = kWorkers / 4;
constexpr int kThreads = (kFirstWorker + kWorkers) * 32;

template <int TN>
struct Cfg {
  static constexpr int kActBytes = TN * 128;
  static constexpr int kRingBytes = kStages * kActBytes + kSlots * kSlotBytes;
  static constexpr int kFinStride = kRows + 4;  // floats a token column
  static constexpr int kFinBytes = TN * kFinStride * 4;
  static constexpr int kBytes = kRingBytes > kFinBytes ? kRingBytes : kFinBytes;  // the sums reuse the rings
  static constexpr int kTmemCols = TN == 256 ? 512 : 256;
  static constexpr int kACol0 = kTmemCols - kStages * kACols;
  static_assert(TN <= kACol0, "accumulator and A stages share tensor memory");
};

struct Ctl {
  uint64_t full[kStages], dq_full[kStages], empty[kStages];
  uint64_t code_full[kSlots], code_empty[kSlots];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
};

struct TcParams {
  const uint8_t* scales;
  uint16_t* out;
  int N, T, blocks;   // blocks of 32 in a row
  int stages;         // of 64 k, in all
  int t_tiles;
  int wide;           // a row's 8 scales of a slot are one aligned 8-byte word
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] x B[smem]^T, bf16 inputs, fp32 accumulate
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 8 codes of a word -> 4 bf16 pairs in k order, times the factor 2^126 X (both halves)
__device__ __forceinline__ void expand8(uint32_t x, uint32_t factor, uint32_t* o) {
  const uint32_t z = x << 4;  // every byte's low nibble where its high one was
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t t = __byte_perm(z, x, ((4 + j) << 12) | (j << 4));  // codes 2j and 2j + 1 in bits 15-12 and 31-28
    o[j] = mul_bf16x2((t & 0x80008000u) | ((t >> 6) & 0x01C001C0u), factor);
  }
}

// the same for any scale, given as a bf16 pair: the values' bytes from tables (the low and the
// high bytes of bf16 0, 0.5, 1, 1.5, 2, 3, 4, 6), then the sign and the scale
__device__ __forceinline__ void expand8_any(uint32_t x, uint32_t scale, uint32_t* o) {
  const uint32_t y = x & 0x77777777u;
  const uint32_t lo[2] = {__byte_perm(0xC0800000u, 0xC0804000u, y), __byte_perm(0xC0800000u, 0xC0804000u, y >> 16)};
  const uint32_t hi[2] = {__byte_perm(0x3F3F3F00u, 0x40404040u, y), __byte_perm(0x3F3F3F00u, 0x40404040u, y >> 16)};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t m = __byte_perm(lo[j >> 1], hi[j >> 1], (j & 1) ? 0x7362 : 0x5140);
    const uint32_t s = ((x >> (8 * j)) & 8u) << 12 | ((x >> (8 * j)) & 0x80u) << 24;
    o[j] = mul_bf16x2(m | s, scale);
  }
}

template <int TN, int KS>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, const TcParams p) {
  using C = Cfg<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* codes = ring + kStages * C::kActBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(ring + C::kBytes);
  volatile int* abort_flag = &ctl->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = KS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / KS;
  const int n0 = tile / p.t_tiles * kRows, t0 = tile % p.t_tiles * TN;
  // this CTA's stages: whole slots, so that code boxes and scale words stay aligned
  const int slots = (p.stages + kStagesPerSlot - 1) / kStagesPerSlot;
  const int s_begin = slots * rank / KS * kStagesPerSlot;
  const int s_end = min(p.stages, slots * (rank + 1) / KS * kStagesPerSlot);
  const int n_stages = s_end - s_begin;  // at least 1: there are at least KS slots

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->dq_full[s], 4);  // the four warps that cover a stage's 128 rows
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&ctl->code_full[s], 1);
      mbar_init(&ctl->code_empty[s], 4 * kStagesPerSlot);
    }
    mbar_init(&ctl->mma_done, 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ activation TMA
    if (lane == 0) {
      int issued = 0;
      for (; issued < n_stages; ++issued) {
        const int st = issued % kStages;
        if (!mbar_wait_sleep(&ctl->empty[st], ((issued / kStages) & 1) ^ 1, abort_flag)) break;
        mbar_arrive_expect_tx(&ctl->full[st], C::kActBytes);
        tma_load_2d(ring + st * C::kActBytes, &tmA, &ctl->full[st], (s_begin + issued) * kStageK, t0);
      }
      for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)  // copies land before the CTA may end
        mbar_wait_drain(&ctl->full[i % kStages], (i / kStages) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kRows, TN, false, false);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(ring), 16, 1024);
      const uint32_t blo0 = static_cast<uint32_t>(bdesc0), bhi = static_cast<uint32_t>(bdesc0 >> 32);
      for (int i = 0; i < n_stages; ++i) {
        const int st = i % kStages;
        if (!mbar_wait_sleep(&ctl->dq_full[st], (i / kStages) & 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t a_col = tmem + C::kACol0 + kACols * st;
        const uint32_t blo = blo0 + st * (C::kActBytes >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_bf16_ta(tmem, a_col + 8 * k, (static_cast<uint64_t>(bhi) << 32) | (blo + 2 * k), idesc, i > 0 || k > 0);
        umma_commit(&ctl->empty[st]);
      }
      umma_commit(&ctl->mma_done);  // every MMA issued is done before tensor memory is read or freed
      mbar_wait_drain(&ctl->mma_done, 0);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ code TMA
    if (lane == 0) {
      const int n_slots = (n_stages + kStagesPerSlot - 1) / kStagesPerSlot;
      int issued = 0;
      for (; issued < n_slots; ++issued) {
        const int sl = issued % kSlots;
        if (!mbar_wait_sleep(&ctl->code_empty[sl], ((issued / kSlots) & 1) ^ 1, abort_flag)) break;
        mbar_arrive_expect_tx(&ctl->code_full[sl], kSlotBytes);
        tma_load_2d(codes + sl * kSlotBytes, &tmW, &ctl->code_full[sl], (s_begin + issued * kStagesPerSlot) * (kStageK / 8), n0);
      }
      for (int i = issued > kSlots ? issued - kSlots : 0; i < issued; ++i)
        mbar_wait_drain(&ctl->code_full[i % kSlots], (i / kSlots) & 1);
    }
  } else if (warp >= kFirstWorker) {
    // ------------------------------------------------------------ expansion
    const int set = (warp - kFirstWorker) >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane (a warp reaches lanes 32 (warp % 4) ..)
    const uint32_t sw = static_cast<uint32_t>(r & 7);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kACol0;
    const uint8_t* srow = p.scales + static_cast<int64_t>(min(n0 + r, p.N - 1)) * p.blocks;
    auto load_scales = [&](int slot) {  // the row's 8 scale codes of a slot; past the row's end 2^0 (codes there are 0)
      const int b0 = s_begin * 2 + slot * 8;
      uint2 v = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      if (p.wide) {
        if (b0 < p.blocks) v = __ldg(reinterpret_cast<const uint2*>(srow + b0));
      } else {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int b = 0; b < 8; ++b)
          w[b >> 2] |= (b0 + b < p.blocks ? static_cast<uint32_t>(__ldg(srow + b0 + b)) : 0x7Fu) << (8 * (b & 3));
        v = make_uint2(w[0], w[1]);
      }
      return v;
    };
    static_assert(kStagesPerSlot % kSets == 0 && kStages % kSets == 0, "each set waits on a ring's phases in order");
    uint2 sc = load_scales(0), sc_next = sc;
    for (int i = set; i < n_stages; i += kSets) {
      const int st = i % kStages, slot = i / kStagesPerSlot, sl = slot % kSlots, q = i % kStagesPerSlot;
      if (q == set) {  // this set's first stage of the slot
        if (slot > 0) sc = sc_next;
        if ((slot + 1) * kStagesPerSlot < n_stages) sc_next = load_scales(slot + 1);
      }
      const bool ok = mbar_wait_sleep(&ctl->code_full[sl], (slot / kSlots) & 1, abort_flag) &&
                      mbar_wait_sleep(&ctl->empty[st], ((i / kStages) & 1) ^ 1, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      tc_fence_after();
      const uint32_t at = smem_u32(codes + sl * kSlotBytes) + r * 128;
      uint4 w[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) w[v] = lds128(at + (((2 * q + v) ^ sw) << 4));
      const uint32_t two = (q & 2 ? sc.y : sc.x) >> (16 * (q & 1));  // the stage's two blocks
      const uint32_t c0 = two & 0xFFu, c1 = (two >> 8) & 0xFFu;
      uint32_t a[32];
      if (!__any_sync(0xFFFFFFFFu, max(c0, c1) > 128u)) {
        const uint32_t f[2] = {((c0 + 126u) << 7) * 0x00010001u, ((c1 + 126u) << 7) * 0x00010001u};
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          expand8(w[v].x, f[v], a + 16 * v);
          expand8(w[v].y, f[v], a + 16 * v + 4);
          expand8(w[v].z, f[v], a + 16 * v + 8);
          expand8(w[v].w, f[v], a + 16 * v + 12);
        }
      } else {
        const uint32_t c[2] = {c0, c1};
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t b = (c[v] == 0u ? 0x0040u : c[v] == 255u ? 0x7FC0u : c[v] << 7) * 0x00010001u;
          expand8_any(w[v].x, b, a + 16 * v);
          expand8_any(w[v].y, b, a + 16 * v + 4);
          expand8_any(w[v].z, b, a + 16 * v + 8);
          expand8_any(w[v].w, b, a + 16 * v + 12);
        }
      }
      tmem_st32(lane_base + kACols * st, a);
      const bool act_ok = mbar_wait_sleep(&ctl->full[st], (i / kStages) & 1, abort_flag);  // so that the MMA thread waits once
      tmem_st_wait();
      tc_fence_before();
      if (!__all_sync(0xFFFFFFFFu, act_ok)) break;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->dq_full[st]);
        mbar_arrive(&ctl->code_empty[sl]);
      }
    }
  }

  // ------------------------------------------------------------ sums: tensor memory -> shared memory -> output
  tc_fence_before();
  __syncthreads();  // MMAs done, copies landed: the rings are free
  tc_fence_after();
  float* fin = reinterpret_cast<float*>(ring);  // [token][kFinStride]
  if (warp >= kFirstWorker) {
    const int set = (warp - kFirstWorker) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    constexpr int kEpSets = TN / 16 < kSets ? TN / 16 : kSets;  // sets that read: 16 columns at a time
    constexpr int kEpCols = TN / kEpSets;
#pragma unroll 1
    for (int c = set * kEpCols; set < kEpSets && c < (set + 1) * kEpCols; c += 16) {
      uint32_t v[16];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
          "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
          "tcgen05.wait::ld.sync.aligned;"
          : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
            "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
          : "r"(addr + c)
          : "memory");
#pragma unroll
      for (int j = 0; j < 16; ++j) fin[(c + j) * C::kFinStride + r] = __uint_as_float(v[j]);
    }
  }
  tc_fence_before();
  if (KS > 1) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  // a rank sums and writes its share of the tokens, two rows a thread
  const int c_begin = TN * rank / KS, c_end = TN * (rank + 1) / KS;
  const bool pairs = (p.N & 1) == 0;
  for (int e = threadIdx.x; e < (c_end - c_begin) * (kRows / 2); e += kThreads) {
    const int c = c_begin + e / (kRows / 2), r = 2 * (e % (kRows / 2));
    const int t = t0 + c, n = n0 + r;
    if (t >= p.T || n >= p.N) continue;
    float v0 = 0.f, v1 = 0.f;
    if (KS > 1) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        float x0, x1;
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                     : "=f"(x0), "=f"(x1)
                     : "r"(mapa_shared(smem_u32(fin + c * C::kFinStride + r), k))
                     : "memory");
        v0 += x0;
        v1 += x1;
      }
    } else {
      const float2 x = *reinterpret_cast<const float2*>(fin + c * C::kFinStride + r);
      v0 = x.x;
      v1 = x.y;
    }
    uint16_t* o = p.out + static_cast<int64_t>(t) * p.N + n;
    const uint32_t both = pack_bf16x2(v0, v1);
    if (pairs) {
      *reinterpret_cast<uint32_t*>(o) = both;
    } else {
      o[0] = static_cast<uint16_t>(both & 0xFFFFu);
      if (n + 1 < p.N) o[1] = static_cast<uint16_t>(both >> 16);
    }
  }
  if (KS > 1) cluster_sync_all();  // the sums stay until every rank has read them
}

template <int TN, int KS>
cudaError_t launch(const CUtensorMap& tmA, const CUtensorMap& tmW, const TcParams& p, int tiles, cudaStream_t stream,
                   const char* name) {
  constexpr int smem = Cfg<TN>::kBytes + static_cast<int>(sizeof(Ctl)) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory per CTA");
  auto kern = mxfp4_tc_kernel<TN, KS>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = KS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * KS));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  LaunchScope scope(stream, name);
  e = cudaLaunchKernelEx(&cfg, kern, tmA, tmW, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int TN>
cudaError_t launch_tn(const uint16_t* A, const CUtensorMap& tmW, TcParams p, int K, cudaStream_t stream, const char* n1,
                      const char* n2, const char* n4) {
  CUtensorMap tmA;
  cudaError_t e = make_tmap_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, A, static_cast<uint64_t>(p.T),
                               static_cast<uint64_t>(K), kStageK, TN, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  p.t_tiles = static_cast<int>((static_cast<int64_t>(p.T) + TN - 1) / TN);
  const int64_t tiles = (static_cast<int64_t>(p.N) + kRows - 1) / kRows * p.t_tiles;
  if (tiles > INT32_MAX / 4) return cudaErrorInvalidValue;
  // CTAs that split K, while they would all be resident and each keeps two slots
  const int slots = (p.stages + kStagesPerSlot - 1) / kStagesPerSlot;
  int ks = 1;
  while (ks < 4 && tiles * ks * 2 <= num_sms() && slots >= 4 * ks) ks *= 2;
  return ks == 1   ? launch<TN, 1>(tmA, tmW, p, static_cast<int>(tiles), stream, n1)
         : ks == 2 ? launch<TN, 2>(tmA, tmW, p, static_cast<int>(tiles), stream, n2)
                   : launch<TN, 4>(tmA, tmW, p, static_cast<int>(tiles), stream, n4);
}

}  // namespace

cudaError_t launch_mxfp4_tc(const uint16_t* A, int T, const uint8_t* codes, const uint8_t* scales, int N, int K,
                            uint16_t* out, cudaStream_t stream) {
  if (T < 1 || N < 1 || K < 32 || K % 32 != 0) return cudaErrorInvalidValue;
  TcParams p{};
  p.scales = scales;
  p.out = out;
  p.N = N;
  p.T = T;
  p.blocks = K / 32;
  p.stages = static_cast<int>((static_cast<int64_t>(K) + kStageK - 1) / kStageK);
  p.wide = K % 256 == 0;
  CUtensorMap tmW;
  cudaError_t e = make_tmap_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, codes, static_cast<uint64_t>(N),
                               static_cast<uint64_t>(K) / 8, 32, kRows, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  if (T <= 32)
    return launch_tn<32>(A, tmW, p, K, stream, "mxfp4_tc_kernel<TN=32>", "mxfp4_tc_kernel<TN=32,split2>", "mxfp4_tc_kernel<TN=32,split4>");
  if (T <= 64)
    return launch_tn<64>(A, tmW, p, K, stream, "mxfp4_tc_kernel<TN=64>", "mxfp4_tc_kernel<TN=64,split2>", "mxfp4_tc_kernel<TN=64,split4>");
  if (T <= 128)
    return launch_tn<128>(A, tmW, p, K, stream, "mxfp4_tc_kernel<TN=128>", "mxfp4_tc_kernel<TN=128,split2>", "mxfp4_tc_kernel<TN=128,split4>");
  return launch_tn<256>(A, tmW, p, K, stream, "mxfp4_tc_kernel<TN=256>", "mxfp4_tc_kernel<TN=256,split2>", "mxfp4_tc_kernel<TN=256,split4>");
}

}  // namespace ar
