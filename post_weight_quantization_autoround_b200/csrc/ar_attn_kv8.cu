// Softmax attention of a batch's new tokens over a paged 8-bit cache (E4M3 codes with a
// power-of-two scale per page and head, as kv8_append_kernel writes them).
//
//   z_j = sm_scale q . k_j,  out = sum_j softmax(z)_j v_j  over the keys j <= position
//
// One token a sequence reads its whole cache for a handful of rows, so the kernel is built
// to stream: bytes of codes per second are the bound, and everything else is kept small.
//
//  * Rows are (new token, head of the group) pairs that share a key/value head: R = 8 NT of
//    them form the columns of the products, S^T = K Q^T and O^T = V^T P^T
//    (mma.sync m16n8k16, f16 in, fp32 sums): with the cache as the left operand 8 rows fill
//    an instruction, where the usual order would need 16.
//  * E4M3 is a subset of f16: one conversion instruction turns two codes into an operand
//    register, with no scale applied.  Queries become f16 after a power-of-two
//    normalisation per row (largest value in [2^13, 2^14)): what f16 loses is below 2^-38 of
//    the row's largest value.  The scales are exponents and go into the softmax: with
//    u = z log2(e) + e_v, P' = 2^(u - max u + 15) carries the value scale and lies in [0, 2^15]
//    whatever the scales, O = sum P' v', and the row sum adds P' 2^(-e_v - 15).  P' is f16 for the
//    product: off by 2^-11 of itself at most (finer than the bf16 output) down to 2^-29 of the row's
//    largest, and by 2^-40 of that below, which is why its range is used up to 2^15: behind a key
//    that takes nearly all weight and has a small value, 10^5 keys still count.  The row sum takes the
//    fp32 value; maximum, sum and O are fp32.  Where a page's value scale lies so far below the others' (a
//    page of zeros next to large values) that P' itself would leave fp32, the row sum takes those weights in a
//    second look, and sums move to a new maximum in two factors.
//  * S^T leaves the tensor core with tokens along lanes' rows; movmatrix transposes the
//    8 x 8 blocks into the B operand of O^T.  V^T comes from ldmatrix.trans on byte pairs:
//    one byte permute separates even and odd dimensions.
//  * The work is the list of (sequence, row tile, head, 32 tokens) steps.  Every warp takes an
//    equal run of it, found from the lengths on the device (the host does not know them,
//    and a captured graph keeps working as they grow), and streams it (4 KB of keys and of
//    values a step at d = 128; TMA boxes with the hardware swizzle, so neither read
//    conflicts) through a private ring: no barrier between warps.  Pages and scales are
//    looked up an item ahead and the copies run on past an item's end.
//  * An item within one warp's run goes straight to the output.  One that warps share is
//    joined from unnormalised sums in the workspace, by its block at the end of the
//    block's run, and by a second kernel where several blocks share it; always in the
//    order of the tokens: no atomics, the same result every time.
//
// 64 sequences up to 8191 keys, 64 heads over 8 of 128 (572 MB): 114 us for this kernel, 120 with the second,
// 4.8 TB/s, 74 % of a copy's rate; 2 x 131000 keys 107 us, 5.0 TB/s.  While an SM is busy it takes its share of the
// full rate, but equal runs end 134 to 170 thousand cycles in: some SMs are served faster than others.
#include <algorithm>

#include "ar_internal.h"

namespace ar {
namespace {

constexpr int kBox = 16;       // tokens of a copy: a page is a multiple of it
constexpr int kChunk = 32;     // steps whose pages and scales the lanes hold
constexpr int kMaxWarps = 8;
constexpr int kShift = 15;     // P' is at most 2^15
constexpr float kUnshift = 1.0f / (1 << kShift);
// Steps one after another that a warp may be given so that no item leaves its block (see the launch function).
constexpr int kFixedMax = 8;

template <int D, int NT>
struct AttnCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlocksPerSm = NT == 1 ? 2 : 1;
  static constexpr int kWarps = NT == 1 ? 6 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kHalves = NT == 4 ? 1 : 2;     // boxes of 16 tokens in a warp's step
  static constexpr int kTile = kBox * kHalves;        // tokens of a step
  static constexpr int kStages = D == 128 ? (NT == 4 ? 6 : NT == 2 ? 3 : 2) : 4;
  static constexpr int kBoxBytes = kBox * D;
  static constexpr int kTileBytes = kTile * D;        // of keys, and of values
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kSlotFloats = kRows * (D + 2); // a partial result: sums, then maximum and row sum per row
};

// a part of an item that one warp computed
struct Part {
  uint32_t item0;  // first step of the item
  int s, rt, head, steps;  // the item; steps = 0: no part
};

struct AttnCtl {
  uint64_t full[kMaxWarps][6];
  Part part[kMaxWarps][2];  // of an item begun before the warp's run; of one that goes on after it
  int abort_flag;
};

struct AttnParams {
  Kv8Args a;
  const uint16_t* q;
  const uint8_t* ks;
  const uint8_t* vs;
  uint16_t* out;
  float* lse;
  float* slots;       // [blocks][2][kSlotFloats], like a warp's parts
  float* warp_slots;  // [blocks][warps][2][kSlotFloats]
  int4* desc;    // [blocks]: {sequence, row tile, head, last block} of the item whose first part is the block's, or x = -1
  float scale_log2;
  int fixed;     // steps that every item counts as, a multiple of the block's warps; 0: as many as it has
};

// a sequence's bounds, checked against the arrays
struct Seq {
  int first, n_new, len;  // first new row, new tokens, tokens
};

__device__ __forceinline__ Seq load_seq(const Kv8Args& a, int s) {
  const int64_t c0 = a.cu[s], rows = a.cu[s + 1] - c0;
  const int64_t len = a.lens[s];
  Seq q;
  const bool ok = rows >= 0 && rows <= a.max_new && c0 >= 0 && c0 + rows <= a.T && len >= 0 && len <= static_cast<int64_t>(a.max_pages) * a.page;
  if (!ok) raise_status(kStatusBadIndex);
  q.first = ok ? static_cast<int>(c0) : 0;
  q.n_new = ok ? static_cast<int>(rows) : 0;
  if (a.split_rows > 0 && static_cast<int64_t>(q.n_new) * (a.n_heads / a.n_kv) >= a.split_rows) q.n_new = 0;  // the other kernel's
  q.len = ok ? static_cast<int>(len) : 0;
  return q;
}

// keys that the row tile's last row sees
__device__ __forceinline__ int tile_keys(const Seq& q, int rt, int rows, int group) {
  const int last = min(q.n_new - 1, (rt * rows + rows - 1) / group);
  return max(0, q.len - q.n_new + last + 1);
}

template <int TILE>
__device__ __forceinline__ int steps_of(int keys) {
  return keys <= TILE ? 1 : (keys + TILE - 1) / TILE;
}

__device__ __forceinline__ int row_tiles(const Seq& q, int rows, int group) {
  return (q.n_new * group + rows - 1) / rows;
}

// the 4 codes of a word, two to a register, in order
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16-byte chunk of a tile's row under the copy's swizzle (128-byte rows: chunk ^ row % 8;
// 64-byte rows: chunk ^ (row / 2) % 4)
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
  return static_cast<uint32_t>(row * D + ((D == 128 ? (chunk ^ (row & 7)) : (chunk ^ ((row >> 1) & 3))) << 4));
}

// 4 dimensions of a row, and its log-sum-exp with the first of them
template <int D>
__device__ __forceinline__ void write_row(const AttnParams& p, const Seq& seq, int head, int group, int rr, int d, float4 acc,
                                          float mx, float sum) {
  const int tok = rr / group;
  const int64_t row = static_cast<int64_t>(seq.first + tok) * p.a.n_heads + head * group + (rr - tok * group);
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  *reinterpret_cast<uint2*>(p.out + row * D + d) =
      make_uint2(pack_bf16x2(acc.x * kUnshift * inv, acc.y * kUnshift * inv), pack_bf16x2(acc.z * kUnshift * inv, acc.w * kUnshift * inv));
  if (p.lse && d == 0) p.lse[row] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;  // a NaN stays one
}

// where a warp's run of steps stands
struct Pos {
  int s, rt, head;   // sequence, row tile, key/value head
  Seq seq;
  int item_steps;    // steps of the row tile (for each head)
  uint32_t item0;    // first step of the row tile's first head
  uint32_t at;       // next step
};

// up to kChunk steps of a warp in one item, one a lane
struct Steps {
  int row[2];      // first row of the step's boxes in the cache, -1: nothing to read
  uint32_t exps;   // scale codes: key, value of the first box, key, value of the second
  uint32_t use, issue;  // steps still to be computed, still to be copied
  int n;
};

template <int D, int NT>
__global__ void __launch_bounds__(AttnCfg<D, NT>::kThreads, AttnCfg<D, NT>::kBlocksPerSm)
    attn_kv8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
  using Cfg = AttnCfg<D, NT>;
  constexpr int kRows = Cfg::kRows, kWarps = Cfg::kWarps, kThreads = Cfg::kThreads, kHalves = Cfg::kHalves;
  constexpr int kTile = Cfg::kTile;
  constexpr int kKs = D / 16;      // k-steps of S^T
  constexpr int kMt = D / 16;      // 16-dimension tiles of O^T
  constexpr int kQr = D / 64;      // 16-byte loads of a K row per lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  AttnCtl* ctl = reinterpret_cast<AttnCtl*>(smem + Cfg::kRingBytes);
  uint32_t* prefix = reinterpret_cast<uint32_t*>(ctl + 1);  // [S + 1] steps before each sequence
  const Kv8Args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int group = a.n_heads / a.n_kv;
  uint8_t* ring = smem + warp * Cfg::kStages * Cfg::kStageBytes;

  if (threadIdx.x == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < Cfg::kStages; ++s) mbar_init(&ctl->full[w][s], 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // short caches: every item counts as many steps as the longest may have, and a block's run holds whole items
  auto item_steps_of = [&](int keys) { return p.fixed > 0 ? p.fixed : steps_of<kTile>(keys); };
  // steps of every sequence: a thread each where it is one row tile, else a warp each
  if (a.max_new * group <= kRows) {
    for (int s = threadIdx.x; s < a.S; s += kThreads) {
      const Seq q = load_seq(a, s);
      uint32_t u = 0;
      for (int rt = 0; rt < row_tiles(q, kRows, group); ++rt) u += item_steps_of(tile_keys(q, rt, kRows, group));
      prefix[s + 1] = u * a.n_kv;
    }
  } else {
    for (int s = warp; s < a.S; s += kWarps) {
      const Seq q = load_seq(a, s);
      const int nrt = row_tiles(q, kRows, group);
      uint32_t u = 0;
      for (int rt = lane; rt < nrt; rt += 32) u += item_steps_of(tile_keys(q, rt, kRows, group));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
      if (lane == 0) prefix[s + 1] = u * a.n_kv;
    }
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t run = 0;
    for (int s0 = 0; s0 < a.S; s0 += 32) {
      uint32_t v = s0 + lane < a.S ? prefix[s0 + lane + 1] : 0u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += t;
      }
      if (s0 + lane < a.S) prefix[s0 + lane + 1] = run + v;
      run += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (lane == 0) prefix[0] = 0u;
  }
  __syncthreads();
  const uint32_t total = prefix[a.S];
  uint32_t quota = (total + gridDim.x * kWarps - 1) / (gridDim.x * kWarps);  // steps of a warp
  if (p.fixed > 0) quota = (total / p.fixed + gridDim.x - 1) / gridDim.x * (p.fixed / kWarps);
  const uint32_t b_begin = min(total, blockIdx.x * kWarps * quota), b_end = min(total, b_begin + kWarps * quota);
  const uint32_t u_begin = min(total, b_begin + warp * quota), u_end = min(total, u_begin + quota);
  if (threadIdx.x == 0) p.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (lane < 2) ctl->part[warp][lane].steps = 0;
  if (b_begin >= b_end) return;

  // where the run starts
  Pos cur{};
  if (u_begin < u_end) {
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (prefix[mid + 1] > u_begin) hi = mid;
      else lo = mid + 1;
    }
    cur.s = lo;
    cur.seq = load_seq(a, lo);
    cur.at = u_begin;
    cur.item0 = prefix[lo];
    for (cur.rt = 0;; ++cur.rt) {
      cur.item_steps = item_steps_of(tile_keys(cur.seq, cur.rt, kRows, group));
      const uint32_t next = cur.item0 + static_cast<uint32_t>(cur.item_steps) * a.n_kv;
      if (next > cur.at) break;
      cur.item0 = next;
    }
    cur.head = static_cast<int>((cur.at - cur.item0) / cur.item_steps);
  }
  auto first_step = [&](const Pos& q) { return q.item0 + static_cast<uint32_t>(q.head) * q.item_steps; };
  auto advance = [&](Pos& q, int n) {  // false at the end of the warp's run
    q.at += n;
    if (q.at >= u_end) return false;
    if (q.at == first_step(q) + q.item_steps) {
      if (++q.head == a.n_kv) {
        q.head = 0;
        q.item0 = q.at;
        if (++q.rt >= row_tiles(q.seq, kRows, group)) {
          q.rt = 0;
          do {
            q.seq = load_seq(a, ++q.s);
          } while (q.seq.n_new == 0 && q.s + 1 < a.S);
        }
        q.item_steps = item_steps_of(tile_keys(q.seq, q.rt, kRows, group));
      }
    }
    return true;
  };
  // the next steps at q: lane i looks up pages and scales of step i
  auto plan = [&](const Pos& q) {
    Steps f;
    const uint32_t fu = first_step(q);
    const int step0 = static_cast<int>(q.at - fu);
    f.n = static_cast<int>(min(min(u_end, fu + q.item_steps) - q.at, static_cast<uint32_t>(kChunk)));
    const int keys = tile_keys(q.seq, q.rt, kRows, group);
    f.exps = 0u;
    f.row[0] = f.row[1] = -1;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int t = (step0 + lane) * kTile + h * kBox;
      if (lane < f.n && t < keys) {
        const int pg = __ldg(a.table + static_cast<int64_t>(q.s) * a.max_pages + t / a.page);
        if (pg >= 0 && pg < a.n_pages) {
          const int64_t ph = static_cast<int64_t>(pg) * a.n_kv + q.head;
          f.row[h] = static_cast<int>(ph * a.page + t % a.page);
          f.exps |= (static_cast<uint32_t>(__ldg(p.ks + ph)) | (static_cast<uint32_t>(__ldg(p.vs + ph)) << 8)) << (16 * h);
        } else {
          raise_status(kStatusBadIndex);
        }
      }
    }
    f.use = f.issue = __ballot_sync(0xFFFFFFFFu, f.row[0] >= 0 || f.row[1] >= 0);
    return f;
  };

  uint32_t stage = 0, phase = 0, ahead = 0;  // next slot to read, its phase, next slot to fill
  int inflight = 0;
  bool alive = true;
  auto issue = [&](Steps& f) {
    const int i = __ffs(f.issue) - 1;
    f.issue &= f.issue - 1;
    int r[2] = {__shfl_sync(0xFFFFFFFFu, f.row[0], i), -1};
    if (kHalves == 2) r[1] = __shfl_sync(0xFFFFFFFFu, f.row[1], i);
    if (lane == 0) {
      uint8_t* dst = ring + ahead * Cfg::kStageBytes;
      uint64_t* bar = &ctl->full[warp][ahead];
      mbar_arrive_expect_tx(bar, (r[0] >= 0 ? 2 * Cfg::kBoxBytes : 0) + (r[1] >= 0 ? 2 * Cfg::kBoxBytes : 0));
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        if (r[h] >= 0) {
          tma_load_2d(dst + h * Cfg::kBoxBytes, &tmK, bar, 0, r[h]);
          tma_load_2d(dst + Cfg::kTileBytes + h * Cfg::kBoxBytes, &tmV, bar, 0, r[h]);
        }
    }
    ahead = ahead + 1 == Cfg::kStages ? 0 : ahead + 1;
    ++inflight;
  };

  Steps fc{}, fn{};
  Pos nxt = cur;
  bool more = false;
  if (u_begin < u_end) {
    fc = plan(cur);
    nxt = cur;
    more = advance(nxt, fc.n);
    if (more) fn = plan(nxt);
  }
  // Copies run ahead into the next steps planned, past the end of an item.  Called wherever a slot or new steps
  // come free: after a step, and after planning (a warp may have had nothing to do in two plans running).
  auto refill = [&]() {
    while (alive && inflight < Cfg::kStages && (fc.issue | fn.issue)) {
      if (fc.issue) issue(fc);
      else issue(fn);
    }
  };

  uint32_t qf[NT][kKs][2];
  float fac[NT][2];
  int lim[NT][2];
  float o[kMt][NT][4];
  float m[NT][2], l[NT][2];
  int t_first = 0, full_below = 0, keys = 0;  // of the part: its first step in the item, tokens every row sees, keys
  bool fresh = true;

  while (u_begin < u_end) {
    refill();
    const int row0 = cur.rt * kRows;
    const int n_rows = cur.seq.n_new * group;
    if (fresh) {
      // ---- a new item: queries as B operand registers, normalised; a row's factor to log2 units
      const int start = cur.seq.len - cur.seq.n_new;
      t_first = static_cast<int>(cur.at - first_step(cur));
      keys = tile_keys(cur.seq, cur.rt, kRows, group);
      full_below = start + row0 / group + 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + nt * 8 + g;
        uint32_t raw[D / 8];  // this lane's D / 4 values (dimensions D / 4 c ..), bf16 pairs
        if (r < n_rows) {
          const int tok = r / group, qh = cur.head * group + (r - tok * group);
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + (static_cast<int64_t>(cur.seq.first + tok) * a.n_heads + qh) * D + c * (D / 4));
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint4 v = __ldg(src + i);
            raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) raw[i] = 0u;
        }
        uint32_t mag = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) mag = __vmaxu2(mag, raw[i] & 0x7FFF7FFFu);
        mag = max(mag & 0xFFFFu, mag >> 16);
        mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
        mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 2));
        // 2^qe q lies below 2^14; qe is kept where both powers are normal
        const int qe = min(126, max(-120, 13 + 127 - static_cast<int>(mag >> 7)));
        const float up = __uint_as_float(static_cast<uint32_t>(qe + 127) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - qe) << 23);
#pragma unroll
        for (int i = 0; i < kKs; ++i) {
          qf[nt][i][0] = pack_f16x2(bf16_lo(raw[2 * i]) * up, bf16_hi(raw[2 * i]) * up);
          qf[nt][i][1] = pack_f16x2(bf16_lo(raw[2 * i + 1]) * up, bf16_hi(raw[2 * i + 1]) * up);
        }
        const float f = down * p.scale_log2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          fac[nt][j] = __shfl_sync(0xFFFFFFFFu, f, (2 * c + j) * 4);
          const int rr = row0 + nt * 8 + 2 * c + j;
          lim[nt][j] = rr < n_rows ? start + rr / group + 1 : 0;  // keys the row sees
          m[nt][j] = -INFINITY;
          l[nt][j] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kMt; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.f;
    }

    const int step0 = static_cast<int>(cur.at - first_step(cur));
    while (alive && fc.use) {
      const int i = __ffs(fc.use) - 1;
      fc.use &= fc.use - 1;
      const uint32_t exps = __shfl_sync(0xFFFFFFFFu, fc.exps, i);
      const int tb = (step0 + i) * kTile;  // first token of the step
      // a step whose boxes are not both there: past the keys, or a page that is not in the pool
      const uint32_t have = static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, (fc.row[0] >= 0 ? 1 : 0) | (fc.row[1] >= 0 ? 2 : 0), i));
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&ctl->full[warp][stage], phase, &ctl->abort_flag))) {
        alive = false;
        break;
      }
      uint8_t* kt = ring + stage * Cfg::kStageBytes;
      const uint32_t ka = smem_u32(kt), va = ka + Cfg::kTileBytes;
      const bool whole_boxes = have == (kHalves == 2 ? 3u : 1u);
      if (tb + kTile > keys || !whole_boxes) {
        // rows past the keys, or of a box that was not copied, hold anything, a NaN too: their values
        // become zeros (their scores are masked below)
        for (int e = lane; e < kTile * (D / 16); e += 32) {
          const int r = e / (D / 16);
          if (tb + r >= keys || !((have >> (r / kBox)) & 1u))
            *reinterpret_cast<uint4*>(kt + Cfg::kTileBytes + e * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the slot is copied into again
      }

      // ---- S^T: tokens g, g + 8 of each box; this lane's codes are dimensions D / 4 c ..
      float z[NT][kHalves][4];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) z[nt][h][j] = 0.f;
#pragma unroll
        for (int v = 0; v < kQr; ++v) {
          const uint4 x0 = lds128(ka + swz<D>(h * kBox + g, kQr * c + v));
          const uint4 x1 = lds128(ka + swz<D>(h * kBox + g + 8, kQr * c + v));
          const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_f16(w0[i4], a0, a2);
            e4m3x4_f16(w1[i4], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(z[nt][h], a0, a1, a2, a3, qf[nt][4 * v + i4][0], qf[nt][4 * v + i4][1]);
          }
        }
      }

      // ---- softmax: u = z log2(e) sm_scale 2^ek + ev
      float fk[kHalves], fe[kHalves], back[kHalves];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const uint32_t ek = (exps >> (16 * h)) & 0xFFu, ev = (exps >> (16 * h + 8)) & 0xFFu;
        fk[h] = __uint_as_float(max(min(ek, 254u), 1u) << 23);
        fe[h] = static_cast<float>(static_cast<int>(ev) - 127);
        back[h] = e8m0_inverse(ev, kShift);
      }
      const bool masked = tb + kTile > full_below || !whole_boxes;
      uint32_t pb[NT][kHalves][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float top[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[j] = -INFINITY;
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            const float f = fac[nt][j] * fk[h];
            z[nt][h][j] = fmaf(z[nt][h][j], f, fe[h]);
            z[nt][h][2 + j] = fmaf(z[nt][h][2 + j], f, fe[h]);
            if (masked) {
              const int end = ((have >> h) & 1u) ? lim[nt][j] : 0;
              if (tb + h * kBox + g >= end) z[nt][h][j] = -INFINITY;
              if (tb + h * kBox + g + 8 >= end) z[nt][h][2 + j] = -INFINITY;
            }
            top[j] = fmaxf(top[j], fmaxf(z[nt][h][j], z[nt][h][2 + j]));
          }
          top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], 4));
          top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], 8));
          top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], 16));
        }
        if (__any_sync(0xFFFFFFFFu, top[0] > m[nt][0] || top[1] > m[nt][1])) {
          float sc[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float mn = fmaxf(m[nt][j], top[j]);
            const float half = mn == -INFINITY ? 1.0f : ex2(0.5f * (m[nt][j] - mn));
            sc[j] = half * half;
            m[nt][j] = mn;
            l[nt][j] = l[nt][j] * half * half;
          }
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) {
            o[mt][nt][0] *= sc[0];
            o[mt][nt][1] *= sc[1];
            o[mt][nt][2] *= sc[0];
            o[mt][nt][3] *= sc[1];
          }
        }
        const float base[2] = {m[nt][0] == -INFINITY ? 0.0f : m[nt][0] - kShift, m[nt][1] == -INFINITY ? 0.0f : m[nt][1] - kShift};
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          float pr[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // no key yet: 2^(-inf) = 0
            pr[j] = ex2(z[nt][h][j] - base[j]);
            pr[2 + j] = ex2(z[nt][h][2 + j] - base[j]);
            l[nt][j] = fmaf(pr[j] + pr[2 + j], back[h], l[nt][j]);
          }
          pb[nt][h][0] = movmatrix(pack_f16x2(pr[0], pr[1]));
          pb[nt][h][1] = movmatrix(pack_f16x2(pr[2], pr[3]));
        }
        // Weights that went to zero (below 2^-126) count where 2^30 of them could be 2^-24 of the row's sum.
        float low = back[0];
        if (kHalves == 2) low = fmaxf(low, back[kHalves - 1]);
        low *= 0x1p-72f;
        if (__any_sync(0xFFFFFFFFu, (l[nt][0] < low && lim[nt][0] > 0) || (l[nt][1] < low && lim[nt][1] > 0))) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float x = z[nt][h][j] - base[j & 1];
              if (x < -126.0f) l[nt][j & 1] = fmaf(ex2(x + 126.0f), back[h] * 0x1p-126f, l[nt][j & 1]);
            }
        }
      }

      // ---- O^T += V^T P^T, 16 dimensions (one 16-byte chunk of the rows) at a time
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int mt = 0; mt < kMt; mt += 2) {
          uint32_t r[4];
          ldmatrix_x4_trans(r, va + swz<D>(h * kBox + 8 * ((lane >> 3) & 1) + (lane & 7), mt + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_f16(__byte_perm(r[2 * x], 0u, 0x3120), a0, a1);
            e4m3x4_f16(__byte_perm(r[2 * x + 1], 0u, 0x3120), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[mt + x][nt], a0, a1, a2, a3, pb[nt][h][0], pb[nt][h][1]);
          }
        }
      __syncwarp();  // the slot has been read
      --inflight;
      if (++stage == Cfg::kStages) {
        stage = 0;
        phase ^= 1u;
      }
      refill();
    }

    const uint32_t fu = first_step(cur);
    const int t_end = static_cast<int>(cur.at - fu) + fc.n;  // steps of the item done so far
    const bool part_ends = fu + t_end == u_end || t_end == cur.item_steps;
    if (part_ends) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[nt][j] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][j], x);
      if (t_first == 0 && t_end == cur.item_steps) {
        // the whole item: straight to the output
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int rr = row0 + nt * 8 + 2 * c + j;
            if (rr >= n_rows) continue;
            const int tok = rr / group;
            const int64_t row = static_cast<int64_t>(cur.seq.first + tok) * a.n_heads + cur.head * group + (rr - tok * group);
            const float inv = l[nt][j] > 0.0f || l[nt][j] != l[nt][j] ? 1.0f / l[nt][j] : 0.0f;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
              *reinterpret_cast<uint32_t*>(p.out + row * D + 16 * mt + 2 * g) =
                  pack_bf16x2(o[mt][nt][j] * kUnshift * inv, o[mt][nt][2 + j] * kUnshift * inv);
            if (p.lse && g == 0)
              p.lse[row] = l[nt][j] == 0.0f ? -INFINITY : (m[nt][j] + log2f(l[nt][j])) * 0.6931471805599453f;
          }
      } else {
        const int k = t_first == 0 ? 1 : 0;
        float* slot = p.warp_slots + ((static_cast<int64_t>(blockIdx.x) * kWarps + warp) * 2 + k) * Cfg::kSlotFloats;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = nt * 8 + 2 * c + j;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
              *reinterpret_cast<float2*>(slot + r * D + 16 * mt + 2 * g) = make_float2(o[mt][nt][j], o[mt][nt][2 + j]);
            if (g == 0) *reinterpret_cast<float2*>(slot + kRows * D + 2 * r) = make_float2(m[nt][j], l[nt][j]);
          }
        if (lane == 0) ctl->part[warp][k] = Part{fu, cur.s, cur.rt, cur.head, cur.item_steps};
      }
    }
    if (!more) break;
    // ---- the steps planned before become the present ones; plan the next
    cur = nxt;
    fc = fn;
    more = advance(nxt, fc.n);
    if (more) fn = plan(nxt);
    else fn.use = fn.issue = 0u;
    fresh = part_ends;
  }
  // a wait that gave up leaves copies in flight: they land before the block may end
  for (; inflight > 0; --inflight) {
    mbar_wait_drain(&ctl->full[warp][stage], phase);
    if (++stage == Cfg::kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }

  // ---- items that several warps of the block share: a warp joins each from the parts in the workspace
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the second kernel may be set up (it waits for this one's end)
  __syncthreads();
  constexpr int kVec = D / 4;                     // 16-byte pieces of a row
  constexpr int kPieces = kRows * kVec / 32;      // a warp's worth of an item
  int at = 0;
  for (int piece0 = 0; at < 2 * kWarps; piece0 += kPieces) {
    while (at < 2 * kWarps && ctl->part[at >> 1][at & 1].steps == 0) ++at;
    if (at >= 2 * kWarps) break;
    // the item's parts: this warp's slot, then the first slots of the warps after it
    const Part it = ctl->part[at >> 1][at & 1];
    const int from = at;
    int last = at;
    for (++at; at < 2 * kWarps; ++at) {
      if (ctl->part[at >> 1][at & 1].steps == 0) continue;
      if (ctl->part[at >> 1][at & 1].item0 != it.item0) break;
      last = at;
    }
    const bool whole = it.item0 >= b_begin && it.item0 + it.steps <= b_end;
    const Seq seq = load_seq(a, it.s);
    const int row0 = it.rt * kRows, n_rows = min(kRows, seq.n_new * group - row0);
    float* slot = p.slots + (static_cast<int64_t>(blockIdx.x) * 2 + (it.item0 >= b_begin ? 1 : 0)) * Cfg::kSlotFloats;
    const float* base = p.warp_slots + (static_cast<int64_t>(blockIdx.x) * kWarps * 2 + from) * Cfg::kSlotFloats;
    // part j: `from` itself, then every second slot (a warp has two)
    const int parts = 1 + (last >> 1) - (from >> 1);
    auto part_at = [&](int j) { return base + (j == 0 ? 0 : 2 * j - (from & 1)) * Cfg::kSlotFloats; };
    for (int piece = (warp + kWarps - piece0 % kWarps) % kWarps; piece < kPieces; piece += kWarps) {
      const int e = piece * 32 + lane, r = e / kVec, d = 4 * (e % kVec);
      // all loads first: a join waits for one of them, not for each
      float2 ml[kWarps];
      float4 x[kWarps];
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        ml[j] = make_float2(-INFINITY, 0.0f);
        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < parts) {
          ml[j] = *reinterpret_cast<const float2*>(part_at(j) + kRows * D + 2 * r);
          x[j] = *reinterpret_cast<const float4*>(part_at(j) + r * D + d);
        }
      }
      float mx = -INFINITY, sum = 0.0f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kWarps; ++j) mx = fmaxf(mx, ml[j].x);
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {
        const float half = ml[j].x == -INFINITY ? 0.0f : ex2(0.5f * (ml[j].x - mx)), f = half * half;
        sum = fmaf(ml[j].y * half, half, sum);
        acc.x = fmaf(x[j].x, f, acc.x);
        acc.y = fmaf(x[j].y, f, acc.y);
        acc.z = fmaf(x[j].z, f, acc.z);
        acc.w = fmaf(x[j].w, f, acc.w);
      }
      if (!whole) {
        *reinterpret_cast<float4*>(slot + r * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(slot + kRows * D + 2 * r) = make_float2(mx, sum);
      } else if (r < n_rows) {
        write_row<D>(p, seq, it.head, group, row0 + r, d, acc, mx, sum);
      }
    }
    if (!whole && it.item0 >= b_begin && threadIdx.x == 0)
      p.desc[blockIdx.x] = make_int4(it.s, it.rt, it.head, static_cast<int>((it.item0 + it.steps - 1) / (quota * kWarps)));
  }
}

// Joins the parts of a row tile that several blocks computed: block b holds its first
// part (the end of b's run), blocks b + 1 .. last the others (the beginnings of theirs).
template <int D, int NT>
__global__ void __launch_bounds__(256) attn_kv8_join_kernel(const AttnParams p) {
  using Cfg = AttnCfg<D, NT>;
  constexpr int kRows = Cfg::kRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the parts are still being computed
  const int4 item = p.desc[blockIdx.x];
  if (item.x < 0) return;
  const Kv8Args& a = p.a;
  const Seq seq = load_seq(a, item.x);
  const int group = a.n_heads / a.n_kv;
  const int row0 = item.y * kRows, n_rows = min(kRows, seq.n_new * group - row0);
  const int first = blockIdx.x, parts = item.w - first + 1;
  const float* base = p.slots;
  auto part = [&](int i) {
    return base + (static_cast<int64_t>(first + i) * 2 + (i == 0 ? 1 : 0)) * Cfg::kSlotFloats;
  };
  constexpr int kVec = D / 4;
  const int lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < kRows * kVec; e += 256) {
    const int r = e / kVec, d = 4 * (e % kVec);
    // the lanes of a row look at its parts' maxima together
    float mx = -INFINITY;
    for (int i = lane % kVec; i < parts; i += kVec) mx = fmaxf(mx, part(i)[kRows * D + 2 * r]);
#pragma unroll
    for (int o = kVec / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    float sum = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = 8;
    for (int i0 = 0; i0 < parts; i0 += kAhead) {
      float2 ml[kAhead];
      float4 x[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        ml[j] = make_float2(-INFINITY, 0.0f);
        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + j < parts) {
          ml[j] = *reinterpret_cast<const float2*>(part(i0 + j) + kRows * D + 2 * r);
          x[j] = *reinterpret_cast<const float4*>(part(i0 + j) + r * D + d);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const float half = ml[j].x == -INFINITY ? 0.0f : ex2(0.5f * (ml[j].x - mx)), f = half * half;
        sum = fmaf(ml[j].y * half, half, sum);
        acc.x = fmaf(x[j].x, f, acc.x);
        acc.y = fmaf(x[j].y, f, acc.y);
        acc.z = fmaf(x[j].z, f, acc.z);
        acc.w = fmaf(x[j].w, f, acc.w);
      }
    }
    if (r < n_rows) write_row<D>(p, seq, item.z, group, row0 + r, d, acc, mx, sum);
  }
}

// rows of a tile, in eights: the fewest of 8, 16, 32 that hold the longest sequence's rows
int tiles_for(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }
int tiles_of(const Kv8Args& a) {
  return tiles_for(a.split_rows > 0 ? a.split_rows - 1 : static_cast<int64_t>(a.max_new) * (a.n_heads / a.n_kv));
}

// Where a call that goes to tcgen05 seems to have short sequences too (prompts next to single tokens), those with no
// more rows than the smallest tile here that holds one token run here, where a long cache is split over the GPU; a
// tile of the other kernel stays with one SM.  This kernel runs after the other one.  512 new tokens of 4000 next
// to 31 single ones of 32000, 64 heads over 8: 461 us, all on tcgen05 1334; a launch with nothing left to do costs 6.
int split_rows_of(const Kv8Args& a) {
  const int group = a.n_heads / a.n_kv;
  if (attn_kv8_long_seqs(a) == a.S || !attn_kv8_tc_fits(a)) return 0;
  return 8 * tiles_for(group) + 1;
}

template <int D, int NT>
cudaError_t launch(AttnParams p, const CUtensorMap& tmK, const CUtensorMap& tmV, void* workspace, cudaStream_t stream) {
  using Cfg = AttnCfg<D, NT>;
  const int blocks = num_sms() * Cfg::kBlocksPerSm;
  const int smem = Cfg::kRingBytes + static_cast<int>(sizeof(AttnCtl)) + (p.a.S + 1) * 4 + 1024;
  static_assert(Cfg::kRingBytes + sizeof(AttnCtl) + (kKv8MaxSeqs + 1) * 4 + 1024 <= 227 * 1024, "shared memory per block");
  p.desc = static_cast<int4*>(workspace);
  p.slots = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 16 * static_cast<size_t>(blocks));
  p.warp_slots = p.slots + static_cast<size_t>(blocks) * 2 * Cfg::kSlotFloats;
  // Where no sequence can have many steps (by the page table's width: the host does not know the lengths), items are padded to a block's warps, so that none is shared between
  // blocks and the second kernel need not be launched.  The padding costs balance: with up to 8 steps a
  // sequence always (a warp then takes one or two steps, or whole items where there are many), with up to 8
  // steps a warp only where every item has a block of its own.
  const int64_t most = (static_cast<int64_t>(p.a.max_pages) * p.a.page + Cfg::kTile - 1) / Cfg::kTile;
  const int64_t rows = static_cast<int64_t>(p.a.max_new) * (p.a.n_heads / p.a.n_kv);
  const int64_t items = p.a.S * ((rows + Cfg::kRows - 1) / Cfg::kRows) * p.a.n_kv;
  p.fixed = most <= kFixedMax || (most <= kFixedMax * Cfg::kWarps && items <= blocks)
                ? static_cast<int>((most + Cfg::kWarps - 1) / Cfg::kWarps * Cfg::kWarps)
                : 0;
  auto kern = attn_kv8_kernel<D, NT>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), 227 * 1024, allowed);
  if (e != cudaSuccess) return e;
  {
    LaunchScope scope(stream, "attn_kv8_kernel");
    kern<<<blocks, Cfg::kThreads, smem, stream>>>(tmK, tmV, p);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess || p.fixed > 0) return e;  // no item is shared
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its launch overlaps the kernel before it
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  LaunchScope scope(stream, "attn_kv8_join_kernel");
  e = cudaLaunchKernelEx(&cfg, attn_kv8_join_kernel<D, NT>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, int NT>
size_t workspace_of() {
  using Cfg = AttnCfg<D, NT>;
  return static_cast<size_t>(num_sms()) * Cfg::kBlocksPerSm * (16 + 2 * Cfg::kSlotFloats * 4 * (1 + Cfg::kWarps));
}

}  // namespace

double attn_kv8_steps(const Kv8Args& args) {
  Kv8Args a = args;
  double tiles = a.S;  // next to the other kernel: at most a tile of each sequence
  if (attn_kv8_tc_fits(a)) {
    a.split_rows = split_rows_of(a);
    if (a.split_rows == 0) return 0.0;
  }
  const int nt = tiles_of(a), rows = 8 * nt, group = a.n_heads / a.n_kv;
  if (a.split_rows == 0) {
    const int64_t most = (static_cast<int64_t>(a.max_new) * group + rows - 1) / rows;
    tiles = std::min(static_cast<double>(a.T) * group / rows + a.S, static_cast<double>(most) * a.S);
  }
  return tiles * a.n_kv * (static_cast<double>(a.max_pages) * a.page / (nt == 4 ? kBox : 2 * kBox) + 1.0);
}

size_t attn_kv8_workspace(const Kv8Args& args) {
  Kv8Args a = args;
  a.split_rows = split_rows_of(a);
  const int nt = tiles_of(a);
  if (a.head_dim == 128) return nt == 1 ? workspace_of<128, 1>() : nt == 2 ? workspace_of<128, 2>() : workspace_of<128, 4>();
  return nt == 1 ? workspace_of<64, 1>() : nt == 2 ? workspace_of<64, 2>() : workspace_of<64, 4>();
}

cudaError_t launch_attn_kv8(const Kv8Args& a, const uint16_t* q, float sm_scale, const uint8_t* k_pages,
                            const uint8_t* v_pages, const uint8_t* k_scales, const uint8_t* v_scales, uint16_t* out,
                            float* lse, void* workspace, cudaStream_t stream) {
  AttnParams p{};
  p.a = a;
  if (attn_kv8_tc_fits(a)) {
    p.a.split_rows = split_rows_of(a);
    const cudaError_t e = launch_attn_kv8_tc(p.a, q, sm_scale, k_pages, v_pages, k_scales, v_scales, out, lse, stream);
    if (e != cudaSuccess || p.a.split_rows == 0) return e;
  }
  p.q = q;
  p.ks = k_scales;
  p.vs = v_scales;
  p.out = out;
  p.lse = lse;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  const uint64_t rows = static_cast<uint64_t>(a.n_pages) * a.n_kv * a.page;
  const CUtensorMapSwizzle sw = a.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  CUtensorMap tmK, tmV;
  cudaError_t e = make_tmap_2d(&tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, k_pages, rows, a.head_dim, a.head_dim, kBox, sw);
  if (e == cudaSuccess) e = make_tmap_2d(&tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, v_pages, rows, a.head_dim, a.head_dim, kBox, sw);
  if (e != cudaSuccess) return e;
  const int nt = tiles_of(p.a);
  if (a.head_dim == 128)
    return nt == 1   ? launch<128, 1>(p, tmK, tmV, workspace, stream)
           : nt == 2 ? launch<128, 2>(p, tmK, tmV, workspace, stream)
                     : launch<128, 4>(p, tmK, tmV, workspace, stream);
  return nt == 1   ? launch<64, 1>(p, tmK, tmV, workspace, stream)
         : nt == 2 ? launch<64, 2>(p, tmK, tmV, workspace, stream)
                   : launch<64, 4>(p, tmK, tmV, workspace, stream);
}

}  // namespace ar
