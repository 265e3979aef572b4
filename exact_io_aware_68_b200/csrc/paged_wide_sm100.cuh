// Attention over a paged key/value cache for sm_100a, many query rows per K/V head: chunks of prompts, drafted
// tokens of wide groups.  Same operation and pools as paged_sm100.cuh.
//
// Bound: the tensor core (4 D flop per row and key against 4 D bytes per key: from about 250 rows on).
// So this is the structure of the training forward (fwd_sm100.cuh): two 128-row query tiles A and B share every
// 128-key block of K and V, tcgen05 MMAs accumulate S and O in TMEM, P goes back through TMEM, and one tile's
// softmax runs while the tensor core works on the other.  What differs:
//  * Rows.  A tile holds floor(128 / g) positions of all g = Hq / Hkv heads that share the K/V head, the heads of
//    a position side by side, so that its rows see nearly the same keys.
//  * Work.  A unit is one 128-key block of one (sequence, K/V head, tile pair).  fa_paged_plan_kernel forms the
//    prefix of the pairs' block counts (causal pairs stop at their last visible key), and every CTA takes an equal,
//    contiguous share of all units.  A pair that several CTAs share is merged from fp32 partials.
//  * Pages.  One TMA box per page and 64-feature panel; a 128-key block is 128 / page of them.  Keys past the
//    sequence's end are not loaded, and their rows of V are zeroed in shared memory (0 * stale would not be 0).
//  * e4m3.  K enters the tensor core as it is: each query row, times a power of two, is split into an e4m3 and an
//    e5m2 part (8 bits fit into 4 + 3, see below), and S is the sum of two 8-bit products.  P needs 16 bits, so V
//    is turned into f16 (exact; NaN stays NaN) by four more warps, in the swizzled layout the MMA reads.  The
//    page's key scale multiplies the finished scores, its value scale the probabilities; where value scales lie far apart
//    (PagedUnit) a block's P and V are bf16, with V times its scale.
// Measured (B200, the whole call): 4 sequences, 512 new tokens against 4097 to 8100 keys, 32/8 heads, D = 128, causal: 187 us in
// bf16 in a short run (1000 TFLOP/s, 0.61 of the measured cuBLAS burst rate; tensor pipe active 55 %, as in the training
// forward: the chain S, softmax, PV of the tiles bounds) and 218 us (850 TFLOP/s) in a long one, where the power cap lowers
// the clock; 3 x 256 new tokens in e4m3 103 us (630 TFLOP/s; tensor pipe 36 %).  A clock trace of the latter shows 4200 cycles
// a unit in the steady state (bf16: 3750) and about 10,000 at every change of segment, where code that has left the
// instruction cache runs: hence the rolled loops there.
// Tried and slower: both tiles on alternating key blocks of one 128-row tile (75 -> 81 us for 64 rows, bf16); V and K both
// converted to f16 (205 us where 8-bit K takes 146); the queries converted by this kernel's warps (4 us a tile).
#pragma once
#include "fwd_sm100.cuh"
#include "paged_sm100.cuh"

namespace fa {

struct WideParams {
  PagedParams p;
  int g;          // query heads per K/V head, <= 128
  int tq;         // positions per tile: floor(128 / g)
  int n_pairs;    // tile pairs per (sequence, K/V head)
  uint8_t* q8;    // e4m3: [2][B, Hq, Nq, D]: the queries' e4m3 and e5m2 parts
  float* q_scale; // [B, Hq, Nq]: what they stand for, times the softmax scale
  int* redo;      // [B, Hkv, n_pairs]: 1 where O is not finite under a causal mask, 2 where the pair has to be computed anew
                  // for it; and one more: nonzero where any has
  uint64_t wait_ns;
  int debug_flags;   // bit 2: the K producer never delivers the first block (exercises the timeout path)
};

// A segment: consecutive blocks of one pair, as much of it as falls into the CTA's share.
struct alignas(16) WideSeg {
  int b, h, pair, t, T;   // t: its first block, T: blocks of the pair
  int L, n, cnt;          // keys and new tokens of the sequence, blocks of the segment (0: the share is done)
  int blocks[2];          // blocks of either tile in it
  int first, pad;         // the CTA's first segment
};

template <int D, bool FP8>
struct WideLayout {
  static constexpr int TILE = 128 * D * 2;         // bytes of one 128-row 16-bit tile
  static constexpr int SUB = 128 * 128;            // one 64-column swizzle panel of a tile
  static constexpr int RAW = 128 * D;              // bytes of one 128-row 8-bit tile
  static constexpr int KTILE = FP8 ? RAW : TILE;
  static constexpr int KST = FP8 ? 4 : (D == 128) ? 3 : 4;
  static constexpr int VST = (D == 128) ? 2 : 4;
  static constexpr int RST = FP8 ? (D == 128 ? 2 : 4) : 0;   // raw V tiles
  static constexpr int SST = 4;                    // scale sets (one per block)
  static constexpr int SET = 80;                   // bytes of one: 8 K scales, 8 V scales / unit of P, the unit, far
  static constexpr int QA_OFF = 0;                 // (e4m3: each query tile is two 8-bit tiles)
  static constexpr int QB_OFF = QA_OFF + TILE;
  static constexpr int K_OFF = QB_OFF + TILE;
  static constexpr int V_OFF = K_OFF + KST * KTILE;
  static constexpr int RAW_OFF = V_OFF + VST * TILE;
  static constexpr int SC_OFF = RAW_OFF + RST * RAW;
  static constexpr int BAR_OFF = SC_OFF + (FP8 ? SST * SET : 0);
  // q_full[2], q_empty[2], k_full, k_empty, v_full, v_empty, raw_full, raw_empty, s_full[2], p_full[2][2], o_fin[2],
  // o_free[2], tail, fin, seg_full, seg_empty, sc_full
  static constexpr int SEGS = 4;                   // segments scheduled ahead
  static constexpr int NBARS = 4 + 2 * KST + 2 * VST + 2 * RST + 2 + 4 + 2 + 2 + 2 + 2 * SEGS + (FP8 ? SST : 0);
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int SEG_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
  static constexpr int BYTES = SEG_OFF + SEGS * int(sizeof(WideSeg));
  __device__ static constexpr int s_col(int x) { return 128 * x; }
  __device__ static constexpr int o_col(int x) { return 256 + D * x; }
  static constexpr int TMEM_COLS = 512;
  // Registers per thread of the warpgroups: softmax (2), producers and MMA issuer, converters.
  static constexpr int THREADS = FP8 ? 512 : 384;
  static constexpr int READERS = FP8 ? 15 : 11;   // warps that read the segments: all but the scheduling one
  static constexpr int LAUNCH_REGS = FP8 ? 128 : 168;
  static constexpr int SOFT_REGS = FP8 ? 152 : 200, IO_REGS = FP8 ? 88 : 104, CVT_REGS = 120;
  static_assert(BYTES <= 232448, "shared memory budget");
  static_assert(2 * SOFT_REGS + IO_REGS + (FP8 ? CVT_REGS : 0) <= THREADS / 128 * LAUNCH_REGS, "register budget");
};

template <int N>
__device__ __forceinline__ void set_regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" :: "n"(N) : "memory"); }
template <int N>
__device__ __forceinline__ void set_regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" :: "n"(N) : "memory"); }

// D[tmem] (+)= A[smem desc] * B[smem desc], 8-bit floating point operands, fp32 accumulate; the form of
// mma_ss_elect.
__device__ __forceinline__ void mma_ss_f8_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|l, 0xffffffff;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// f16x2 to a pair of e4m3 or e5m2 codes (bits 0-15): nearest, saturating, NaN to NaN.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f16x2 t, %1;\n\tcvt.u32.u16 %0, t;\n\t}\n" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_to_e5m2x2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e5m2x2.f16x2 t, %1;\n\tcvt.u32.u16 %0, t;\n\t}\n" : "=r"(r) : "r"(x));
  return r;
}

// 4-D tiled load (no multicast) into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// Blocks of one tile pair (x < 0) or of one of its tiles; kv: the keys that its rows see.
__device__ __forceinline__ int wide_keys(const WideParams& q, int L, int n, int pair, int x) {
  const int i0 = (2 * pair + (x > 0 ? 1 : 0)) * q.tq, i1 = (2 * pair + (x == 0 ? 1 : 2)) * q.tq;
  if (i0 >= n) return 0;
  return q.p.causal ? min(max(L - n + min(n, i1), 0), L) : L;
}

// Queries as two 8-bit parts.  Each row times a power of two that puts its largest element into [2^7, 2^8).  An element's
// 8 significant bits are hi = the nearest e4m3 number and at most 8 units of its last bit, which is 3 significant bits:
// e5m2.  Elements below 2^-9 (2^-17 of the largest) lose bits: at most 2^-14, that is 2^-21 of the largest element.
// A row with an element that is not finite becomes NaN, as its scores are (inf - inf) in any case.  In a kernel
// of its own since by the warps of the main one it took 4 us a tile at each segment's start (latency, cold code).
template <int D>
__device__ __forceinline__ void wide_split_queries(const WideParams& q) {
  constexpr int LPR = D / 8;   // lanes per row
  const int64_t rows = (int64_t)q.p.B * q.p.Hkv * q.p.R;
  const int c = threadIdx.x % LPR;
  for (int64_t row = ((int64_t)(blockIdx.x - 1) * 1024 + threadIdx.x) / LPR; row < (rows + 31) / 32 * 32; row += (int64_t)(gridDim.x - 1) * (1024 / LPR)) {
    const bool real = row < rows;
    const uint4 w = real ? global_load(reinterpret_cast<const uint4*>(q.p.q + row * D) + c) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float mx = 0.f;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = fabsf(__uint_as_float(u[e] << 16)), b = fabsf(__uint_as_float(u[e] & 0xffff0000u));
      mx = max3f(mx, a, b);
      finite = finite && a < INFINITY && b < INFINITY;
    }
#pragma unroll
    for (int z = 1; z < LPR; z <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, z));
    const unsigned all = __ballot_sync(0xffffffffu, finite);
    const unsigned mine = (LPR == 16 ? 0xffffu : 0xffu) << (threadIdx.x % 32 / LPR * LPR);
    const int ex = min(max(int(__float_as_uint(mx) >> 23) - 127, -100), 127);
    const bool scaled = mx > 0.f;
    const float up = (all & mine) != mine ? NAN : scaled ? __uint_as_float(uint32_t(127 + 7 - ex) << 23) : 1.f;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t x = pack_f16x2(__uint_as_float(u[e] << 16) * up, __uint_as_float(u[e] & 0xffff0000u) * up);   // exact down to 2^-17
      const uint32_t h2 = f16x2_to_e4m3x2(x), f2 = e4m3x2_to_f16x2(h2);
      uint32_t rest;   // x - hi
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(x), "r"(f2));
      const uint32_t l2 = f16x2_to_e5m2x2(rest);
      hi[e >> 1] = (e & 1) ? hi[e >> 1] | (h2 << 16) : h2;
      lo[e >> 1] = (e & 1) ? lo[e >> 1] | (l2 << 16) : l2;
    }
    if (!real) continue;
    *reinterpret_cast<uint2*>(q.q8 + row * D + 8 * c) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(q.q8 + (rows + row) * D + 8 * c) = make_uint2(lo[0], lo[1]);
    if (c == 0)
      q.q_scale[row] = fmaxf(q.p.scale_log2 * (scaled ? __uint_as_float(uint32_t(127 - 7 + ex) << 23) : 1.f), kPagedLeastScale);
  }
}

// Prefix of the block counts of all (sequence, tile pair)s, into p.plan, by the first CTA; with e4m3 pools the others
// prepare the queries.
template <int D, bool FP8>
__global__ void __launch_bounds__(1024) fa_paged_plan_kernel(const __grid_constant__ WideParams q) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if constexpr (FP8)
    if (blockIdx.x > 0) {
      wide_split_queries<D>(q);
      return;
    }
  __shared__ int sums[32];
  __shared__ int carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int total = q.p.B * q.n_pairs;
  if (tid == 0) carry = q.p.plan[0] = 0;
  for (int i = tid; i <= total * q.p.Hkv; i += 1024) q.redo[i] = 0;
  __syncthreads();
  for (int base = 0; base < total; base += 1024) {
    const int at = base + tid;
    int v = 0;
    if (at < total) {
      const int b = at / q.n_pairs;
      v = (wide_keys(q, paged_key_len(q.p, b), paged_new_len(q.p, b), at % q.n_pairs, -1) + 127) / 128;
    }
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, s);
      if (lane >= s) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
      int u = sums[lane];
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, u, s);
        if (lane >= s) u += t;
      }
      sums[lane] = u;
    }
    __syncthreads();
    v += carry + (warp > 0 ? sums[warp - 1] : 0);
    if (at < total) q.p.plan[at + 1] = v;
    __syncthreads();
    if (tid == 1023) carry = v;
    __syncthreads();
  }
}

// The largest i in [lo, hi) with f[i * step] * mul <= want; a whole warp, 32 candidates a round.
__device__ __forceinline__ int wide_search(const int* f, int lo, int hi, int step, long long mul, long long want, int lane) {
  while (hi - lo > 1) {
    const int d = (hi - lo + 31) / 32, i = lo + lane * d;
    const bool le = i < hi && f[(int64_t)i * step] * mul <= want;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, le));   // lane 0 always holds
    lo += last * d;
    hi = min(hi, lo + d);
  }
  return lo;
}

// The walk over a CTA's share, by the scheduling warp.
struct WideWalk {
  WideSeg s;
  int left;   // units of the share from this segment on
  __device__ __forceinline__ void fill(const WideParams& q) {
    s.cnt = min(left, s.T - s.t);
#pragma unroll
    for (int x = 0; x < 2; ++x)
      s.blocks[x] = min(max((wide_keys(q, s.L, s.n, s.pair, x) + 127) / 128 - s.t, 0), s.cnt);
  }
  __device__ __forceinline__ void next(const WideParams& q) {
    left -= s.cnt;
    s.cnt = 0;
    s.first = 0;
    if (left <= 0) return;
    s.t = 0;
    const int* f = q.p.plan;
    const int b0 = s.b;
    do {   // pairs with blocks; some are left
      ++s.pair;
      if (s.pair >= q.n_pairs || 2 * s.pair * q.tq >= s.n) {   // the pairs past the last token have none
        s.pair = 0;
        if (++s.h == q.p.Hkv) {
          s.h = 0;
          do ++s.b; while (s.b < q.p.B && f[(int64_t)(s.b + 1) * q.n_pairs] == f[(int64_t)s.b * q.n_pairs]);
          if (s.b >= q.p.B) {   // (only if the lengths changed under the call)
            left = 0;
            return;
          }
          s.n = paged_new_len(q.p, s.b);
        }
      }
      const int64_t at = (int64_t)s.b * q.n_pairs + s.pair;
      s.T = f[at + 1] - f[at];
    } while (s.T == 0);
    if (s.b != b0) s.L = paged_key_len(q.p, s.b);
    fill(q);
  }
};

template <int D, bool FP8>
__global__ void __launch_bounds__((WideLayout<D, FP8>::THREADS), 1)
fa_paged_wide_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q2,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ WideParams q) {
  using L = WideLayout<D, FP8>;
  constexpr int KST = L::KST, VST = L::VST, RST = FP8 ? L::RST : 1;
  const PagedParams& p = q.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;");
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) record_status(kStatusBadSmemAlign);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t* q_full = bars;           // [2]: tile A, tile B
  uint64_t* q_empty = q_full + 2;    // [2]
  uint64_t* k_full = q_empty + 2;
  uint64_t* k_empty = k_full + KST;
  uint64_t* v_full = k_empty + KST;
  uint64_t* v_empty = v_full + VST;
  uint64_t* raw_full = v_empty + VST;
  uint64_t* raw_empty = raw_full + L::RST;
  uint64_t* s_full = raw_empty + L::RST;   // [2]
  uint64_t* p_full = s_full + 2;      // [2][2]: tile, half of the keys
  uint64_t* o_fin = p_full + 4;       // [2]: all PV of the segment done
  uint64_t* o_free = o_fin + 2;       // [2]: the epilogue has read O
  uint64_t* tail = o_free + 2;        // bf16: the V block that holds a sequence's end has landed
  uint64_t* fin = tail + 1;
  uint64_t* seg_full = fin + 1;       // [SEGS]
  uint64_t* seg_empty = seg_full + L::SEGS;
  uint64_t* sc_full = seg_empty + L::SEGS;   // [SST]: e4m3: a block's scales are there
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
  WideSeg* segs = reinterpret_cast<WideSeg*>(smem + L::SEG_OFF);

  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[2 * x], 4);
      mbar_init(&p_full[2 * x + 1], 4);
      mbar_init(&o_fin[x], 1);
      mbar_init(&o_free[x], 4);
    }
    for (int s = 0; s < KST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&v_full[s], FP8 ? 4 : 1);
      mbar_init(&v_empty[s], 1);
    }
    if constexpr (FP8)
      for (int s = 0; s < L::SST; ++s) mbar_init(&sc_full[s], 1);
    for (int s = 0; s < L::RST; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    mbar_init(tail, 1);
    mbar_init(fin, 1);
    for (int i = 0; i < L::SEGS; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], L::READERS);
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{q.wait_ns, abort_flag};
  const int cta = int(blockIdx.x);

  // Segments come from warp 11 by a ring; every other warp reads them in order.
  int seg_at = 0;
  auto read_seg = [&]() {
    WideSeg s;
    const uint32_t at = smem_u32(&segs[seg_at % L::SEGS]);
    asm volatile("ld.shared.v4.s32 {%0,%1,%2,%3}, [%4];" : "=r"(s.b), "=r"(s.h), "=r"(s.pair), "=r"(s.t) : "r"(at) : "memory");
    asm volatile("ld.shared.v4.s32 {%0,%1,%2,%3}, [%4];" : "=r"(s.T), "=r"(s.L), "=r"(s.n), "=r"(s.cnt) : "r"(at + 16) : "memory");
    asm volatile("ld.shared.v4.s32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(s.blocks[0]), "=r"(s.blocks[1]), "=r"(s.first), "=r"(s.pad) : "r"(at + 32) : "memory");
    return s;
  };
  auto wait_seg = [&]() {
    return __all_sync(0xffffffffu, mbar_wait(&seg_full[seg_at % L::SEGS], (seg_at / L::SEGS) & 1, wc));
  };
  auto release_seg = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[seg_at % L::SEGS]);
    ++seg_at;
  };
  auto next_seg = [&](WideSeg& s) -> bool {
    if (!wait_seg()) return false;
    s = read_seg();
    release_seg();
    return s.cnt > 0;
  };
  WideSeg s;

  // Pages of 128 keys from block t on: lane i looks at piece i (a page, or half of a 256-key page).
  const int piece_rows = min(1 << p.page_shift, 128), pieces = 128 / piece_rows;
  auto has_piece = [&](const WideSeg& w, int j, int i) { return i < pieces && (w.t + j) * 128 + i * piece_rows < w.L; };
  auto piece_page = [&](const WideSeg& w, int j, int i) -> int {   // its page (not looked at yet)
    const int key = (w.t + j) * 128 + i * piece_rows;
    const int id = has_piece(w, j, i) ? global_load(p.page_table + (int64_t)w.b * p.max_pages + (key >> p.page_shift)) : 0;
    return id;
  };

  if (warp >= 8 && warp < 12) {
    set_regs_dec<L::IO_REGS>();
    if (warp == 11) {
      // =========================================================== scheduler and producer of the Q tiles
      asm volatile("griddepcontrol.wait;" ::: "memory");   // the plan; everything above overlaps it
      const long long W = (long long)p.plan[p.B * q.n_pairs] * p.Hkv;
      const int sharers = paged_sharers(W, int(gridDim.x));
      WideWalk walk{};
      if (cta < sharers) {
        const long long u0 = paged_share(W, cta, sharers);
        walk.left = int(paged_share(W, cta + 1, sharers) - u0);
        const int b = wide_search(p.plan, 0, p.B, q.n_pairs, p.Hkv, u0, lane);
        const int64_t at = (int64_t)b * q.n_pairs;
        const int base = p.plan[at], sum = p.plan[at + q.n_pairs] - base;
        const long long rem = u0 - (long long)base * p.Hkv;
        const int h = int(rem / sum), v = base + int(rem % sum);
        const int pair = wide_search(p.plan + at, 0, q.n_pairs, 1, 1, v, lane);
        walk.s.b = b;
        walk.s.h = h;
        walk.s.pair = pair;
        walk.s.t = v - p.plan[at + pair];
        walk.s.T = p.plan[at + pair + 1] - p.plan[at + pair];
        walk.s.L = paged_key_len(p, b);
        walk.s.n = paged_new_len(p, b);
        walk.s.first = 1;
        walk.fill(q);
      }
      if (lane == 0) {
        prefetch_tmap(&tm_q);
        if constexpr (FP8) prefetch_tmap(&tm_q2);
        int nq[2] = {0, 0};   // Q tiles delivered, per tile
        bool ok = true;
        for (int i = 0; ok; ++i) {
          const int slot = i % L::SEGS;
          if (i >= L::SEGS && !mbar_wait(&seg_empty[slot], ((i / L::SEGS) - 1) & 1, wc)) break;
          segs[slot] = walk.s;
          mbar_arrive(&seg_full[slot]);
          if (walk.s.cnt == 0) break;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (walk.s.blocks[x] == 0) continue;
            if (nq[x] >= 1 && !mbar_wait(&q_empty[x], (nq[x] - 1) & 1, wc)) { ok = false; break; }
            mbar_arrive_expect_tx(&q_full[x], D * 2 * q.g * q.tq);
            uint8_t* to = smem + (x ? L::QB_OFF : L::QA_OFF);
            const int i0 = (2 * walk.s.pair + x) * q.tq, bh = walk.s.b * p.Hkv + walk.s.h;
            if constexpr (FP8) {
              tma_load_4d(to, &tm_q, &q_full[x], 0, 0, i0, bh);
              tma_load_4d(to + L::RAW, &tm_q2, &q_full[x], 0, 0, i0, bh);
            } else {
#pragma unroll
              for (int c = 0; c < D / 64; ++c) tma_load_4d(to + c * L::SUB, &tm_q, &q_full[x], c * 64, 0, i0, bh);
            }
            ++nq[x];
          }
          if (ok) walk.next(q);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (nq[x] >= 1) mbar_drain(&q_full[x], (nq[x] - 1) & 1, q.wait_ns);
      }
      __syncwarp();
    } else if (warp == 8 || warp == 10) {
      // =========================================================== producers of the K (warp 8) and V (warp 10; e4m3: raw V) rings
      const bool is_k = (warp == 8);
      const int NS = is_k ? KST : FP8 ? RST : VST;
      uint64_t* full = is_k ? k_full : FP8 ? raw_full : v_full;
      uint64_t* empty = is_k ? k_empty : FP8 ? raw_empty : v_empty;
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      uint8_t* ring = smem + (is_k ? L::K_OFF : FP8 ? L::RAW_OFF : L::V_OFF);
      if (lane == 0) prefetch_tmap(map);
      int g = 0, tails = 0;   // blocks delivered so far; those of V in bf16 with a sequence's end
      bool ok = true;
      while (ok && next_seg(s)) {
        const int n_max = s.cnt;
        int next_page = piece_page(s, 0, lane);
        for (int j = 0; j < n_max; ++j, ++g) {
          const int st = g % NS;
          const int page = next_page;
          if (j + 1 < n_max) next_page = piece_page(s, j + 1, lane);   // in flight during the wait below
          const bool mine = has_piece(s, j, lane);
          const unsigned have = __ballot_sync(0xffffffffu, mine);
          const int key0 = (s.t + j) * 128;
          const bool ends = !FP8 && !is_k && key0 + 128 > s.L;
          if (!__all_sync(0xffffffffu, g < NS || mbar_wait(&empty[st], ((g / NS) - 1) & 1, wc))) { ok = false; break; }
          if (is_k && g == 0 && (q.debug_flags & 4)) { ok = false; break; }   // test hook
          uint64_t* bar = ends ? tail : &full[st];
          if (lane == 0) mbar_arrive_expect_tx(bar, __popc(have) * piece_rows * (FP8 ? D : 2 * D));
          __syncwarp();
          if (mine) {
            int from = page;
            if (unsigned(page) >= unsigned(p.n_pages)) {   // outside the pool: the copy fills in zeros
              record_status(kStatusRange);
              from = p.n_pages;
            }
            const int y = (key0 + lane * piece_rows) & ((1 << p.page_shift) - 1);
            if constexpr (FP8) {
              tma_load_4d(ring + st * L::RAW + lane * piece_rows * D, map, bar, 0, y, s.h, from);
            } else {
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(ring + st * L::TILE + c * L::SUB + lane * piece_rows * 128, map, bar, c * 64, y, s.h, from);
            }
          }
          if (ends) {   // rows past the end: zeros, before the block is handed on
            if (!__all_sync(0xffffffffu, mbar_wait(tail, tails & 1, wc))) { ok = false; break; }
            ++tails;
            for (int i = lane; i < (key0 + 128 - s.L) * (D / 8); i += 32) {
              const int row = s.L - key0 + i / (D / 8), c = i % (D / 8);
              *reinterpret_cast<uint4*>(ring + st * L::TILE + (c >> 3) * L::SUB + row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
          }
        }
      }
      if (lane == 0) {   // every copy started here lands before the CTA releases its shared memory
        if (!FP8 && !ok && !is_k) mbar_drain(tail, tails & 1, q.wait_ns);   // a copy of an unfinished tail block, if any
        for (int j = max(0, g - NS); j < g; ++j) mbar_drain(&full[j % NS], (j / NS) & 1, q.wait_ns);
      }
      __syncwarp();
    } else if (warp == 9) {
      // =========================================================== MMA issuer (whole warp, elect.sync)
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc)); };
      constexpr uint32_t kType = FP8 ? (1u << 7) | (1u << 10) : 0u;   // e4m3 (S) or f16 (PV) operands, format 0, instead of bf16 (1)
      constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false) & ~kType;   // Q: K-major, K: K-major
      constexpr uint32_t kIdPV = idesc_bf16(128, D, false, true) & ~kType;     // P: TMEM, V: MN-major
      const uint32_t s0 = smem_u32(smem) >> 4;
      constexpr uint32_t kHi = sdesc_sw128_hi(1024), kKM = sdesc_lbo(16), kMN = sdesc_lbo(L::SUB);
      int gk = 0;                // blocks consumed (K and V alike)
      int nb0 = 0, nb1 = 0;      // blocks of either tile so far: phase of p_full
      int ni0 = 0, ni1 = 0;      // segments with work for either tile so far: phase of q_full, o_free
      bool ok = true;
      while (ok && next_seg(s)) {
        const int n_max = s.cnt;
        auto issue_s = [&](int x, int kst) {   // S_x = Q_x K^T
          const uint32_t q_lo = s0 + uint32_t((L::QA_OFF + x * L::TILE) >> 4) + kKM;
          const uint32_t k_lo = s0 + uint32_t((L::K_OFF + kst * L::KTILE) >> 4) + kKM;
          if constexpr (FP8) {
            // rows of D bytes: the 128-byte swizzle at D = 128, the 64-byte swizzle (layout 4, 8 rows 512 bytes apart) at 64
            constexpr uint32_t kHi8 = D == 128 ? sdesc_sw128_hi(1024) : ((512u >> 4) | (1u << 14) | (4u << 29));
#pragma unroll
            for (int part = 0; part < 2; ++part)   // the queries' e4m3, then their e5m2 part
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_ss_f8_elect(tmem + L::s_col(x), sdesc_join(q_lo + ((part * L::RAW + kk * 32) >> 4), kHi8),
                                sdesc_join(k_lo + ((kk * 32) >> 4), kHi8), kIdS | (part ? 1u << 7 : 0u), part + kk > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * L::SUB + (kk & 3) * 32) >> 4;
              mma_ss_elect(tmem + L::s_col(x), sdesc_join(q_lo + off, kHi), sdesc_join(k_lo + off, kHi), kIdS, kk > 0 ? 1u : 0u);
            }
          }
          mma_commit_elect(&s_full[x]);
        };
        if constexpr (FP8) {
          // Rolled over the tiles and the halves of P, since code that runs once a segment comes from beyond the instruction
          // cache, at a microsecond a stretch (2 x 16 x 4096 prefill 261 -> 224 us).  bf16, with less code in its other warps,
          // loses more by the loops (chunk of 512: 190 -> 214 us).
          // step -1: the first S of either tile; step j: PV(j), then S(j + 1)
          for (int j = -1; ok && j < n_max; ++j) {
            const int vst = (gk + j) % VST, kst1 = (gk + j + 1) % KST;
            if (j >= 0 && !wait(&v_full[vst], ((gk + j) / VST) & 1)) { ok = false; break; }
            uint32_t id_pv = kIdPV;
            if (j >= 0) {   // far: bf16
              uint32_t far;
              const uint32_t at = smem_u32(smem) + L::SC_OFF + (gk + j) % L::SST * L::SET + 68;
              asm volatile("ld.shared.u32 %0, [%1];" : "=r"(far) : "r"(at) : "memory");
              if (far) id_pv |= kType;
            }
            bool have_k = false;   // K_{j+1} resident
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              const int n_x = x ? s.blocks[1] : s.blocks[0], n_i = x ? ni1 : ni0, n_b = x ? nb1 : nb0;
              if (j >= n_x || n_x == 0) continue;
              if (j >= 0) {
                // the first PV of a segment overwrites O: the previous segment's epilogue must have read it
                if (j == 0 && n_i >= 1 && !wait(&o_free[x], (n_i - 1) & 1)) { ok = false; break; }
                const uint32_t v_lo = s0 + uint32_t((L::V_OFF + vst * L::TILE) >> 4) + kMN;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {   // O_x += P_x[keys of half h] V[same keys]
                  if (!wait(&p_full[2 * x + h], (n_b + j) & 1)) { ok = false; break; }
                  tc_fence_after();
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    mma_ts_elect(tmem + L::o_col(x), tmem + L::s_col(x) + 32 * h + k * 8,
                                 sdesc_join(v_lo + (4 * h + k) * (2048 >> 4), kHi), id_pv, (j > 0 || h + k > 0) ? 1u : 0u);
                }
                if (!ok) break;
              } else if (!wait(&q_full[x], n_i & 1)) {
                ok = false;
                break;
              }
              if (j + 1 < n_x) {
                if (!have_k) {
                  if (!wait(&k_full[kst1], ((gk + j + 1) / KST) & 1)) { ok = false; break; }
                  have_k = true;
                }
                tc_fence_after();
                issue_s(x, kst1);
                if (j + 2 == n_x) mma_commit_elect(&q_empty[x]);   // the next segment's Q_x may come now
              } else {
                mma_commit_elect(&o_fin[x]);
              }
            }
            if (!ok) break;
            if (j >= 0) mma_commit_elect(&v_empty[vst]);           // V_j: both tiles' PV issued
            if (j + 1 < n_max) mma_commit_elect(&k_empty[kst1]);   // K_{j+1}: both tiles' S issued
          }
        } else {
          const int n_x[2] = {s.blocks[0], s.blocks[1]}, n_i[2] = {ni0, ni1}, n_b[2] = {nb0, nb1};
          auto issue_pv_half = [&](int x, int vst, int h, uint32_t acc0) {   // O_x += P_x[keys of half h] V[same keys]
            const uint32_t v_lo = s0 + uint32_t((L::V_OFF + vst * L::TILE) >> 4) + kMN;
#pragma unroll
            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
              mma_ts_elect(tmem + L::o_col(x), tmem + L::s_col(x) + kk * 8, sdesc_join(v_lo + kk * (2048 >> 4), kHi), kIdPV,
                           kk > 0 ? 1u : acc0);
          };
          if (!wait(&k_full[gk % KST], (gk / KST) & 1)) { ok = false; break; }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (n_x[x] == 0) continue;
            if (!wait(&q_full[x], n_i[x] & 1)) { ok = false; break; }
            tc_fence_after();
            issue_s(x, gk % KST);
            if (n_x[x] == 1) mma_commit_elect(&q_empty[x]);   // the next segment's Q_x may come now
          }
          if (!ok) break;
          mma_commit_elect(&k_empty[gk % KST]);
          for (int j = 0; ok && j < n_max; ++j) {
            const int vst = (gk + j) % VST, kst1 = (gk + j + 1) % KST;
            if (!wait(&v_full[vst], ((gk + j) / VST) & 1)) { ok = false; break; }
            bool have_k = false;   // K_{j+1} resident
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (j >= n_x[x]) continue;
              // the first PV of a segment overwrites O: the previous segment's epilogue must have read it
              if (j == 0 && n_i[x] >= 1 && !wait(&o_free[x], (n_i[x] - 1) & 1)) { ok = false; break; }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (!wait(&p_full[2 * x + h], (n_b[x] + j) & 1)) { ok = false; break; }
                tc_fence_after();
                issue_pv_half(x, vst, h, j > 0 ? 1u : 0u);
              }
              if (!ok) break;
              if (j + 1 < n_x[x]) {
                if (!have_k) {
                  if (!wait(&k_full[kst1], ((gk + j + 1) / KST) & 1)) { ok = false; break; }
                  tc_fence_after();
                  have_k = true;
                }
                issue_s(x, kst1);
                if (j + 2 == n_x[x]) mma_commit_elect(&q_empty[x]);
              } else {
                mma_commit_elect(&o_fin[x]);
              }
            }
            if (!ok) break;
            mma_commit_elect(&v_empty[vst]);                       // V_j: both tiles' PV issued
            if (j + 1 < n_max) mma_commit_elect(&k_empty[kst1]);   // K_{j+1}: both tiles' S issued
          }
          if (!ok) break;
        }
        gk += n_max;
        nb0 += s.blocks[0];
        nb1 += s.blocks[1];
        ni0 += s.blocks[0] > 0;
        ni1 += s.blocks[1] > 0;
      }
      mma_commit_elect(fin);   // completes when every MMA issued above has finished
      if (lane == 0) mbar_drain(fin, 0, q.wait_ns);
      __syncwarp();
    }
  } else if (FP8 && warp >= 12) {
    // =========================================================== converters: V to f16, or (far) to bf16 times its scale
    set_regs_dec<L::CVT_REGS>();
    const int ct = tid - 384;
    float* scales = reinterpret_cast<float*>(smem + L::SC_OFF);
    int gb = 0;        // blocks so far
    bool ok = true;
    while (ok && next_seg(s)) {
      const int n_max = s.cnt;
      // lanes 8-15 of each warp: V scale of 16-key group lane & 7 (past the end 0), lanes 0-7 of the first K's (1: its scores
      // are masked), looked up one block ahead, their pages two blocks
      auto group_page = [&](int j) -> int {
        const int key = (s.t + j) * 128 + 16 * (lane & 7);
        const bool mine = lane < 16 && (warp == 12 || lane >= 8) && j < n_max && key < s.L;
        return mine ? global_load(p.page_table + (int64_t)s.b * p.max_pages + (key >> p.page_shift)) : -1;
      };
      auto group_scale = [&](int id) -> float {
        if (unsigned(id) >= unsigned(p.n_pages)) return lane < 8 ? 1.f : 0.f;
        return global_load((lane < 8 ? p.k_scale : p.v_scale) + (int64_t)id * p.Hkv + s.h);
      };
      float next_scale = group_scale(group_page(0));
      int next_id = group_page(1);
      PagedUnit vu;   // the segment's units of O, by each warp for itself
      vu.reset();
      float unit = 0.f;   // kPagedPScale / vu.unit
      for (int j = 0; j < n_max; ++j, ++gb) {
        const int key0 = (s.t + j) * 128;
        const int st = gb % RST, dst_st = gb % VST;
        float my_scale = next_scale;
        next_scale = group_scale(next_id);
        next_id = group_page(j + 2);
        const bool value = lane >= 8 && my_scale > 0.f;
        if (__any_sync(0xffffffffu, value && (my_scale > vu.unit || my_scale < vu.least))) {
          const uint32_t bits = __float_as_uint(my_scale);   // (positive floats order as their bits do)
          const uint32_t hi = __reduce_max_sync(0xffffffffu, value ? bits : 0u);
          const uint32_t lo = __reduce_min_sync(0xffffffffu, value ? bits : 0x7f800000u);
          float move;
          vu.meet(__uint_as_float(hi), __uint_as_float(lo), move);
          unit = kPagedPScale / vu.unit;
        }
        if (lane >= 8) my_scale *= unit;
        if (!__all_sync(0xffffffffu, mbar_wait(&raw_full[st], (gb / RST) & 1, wc))) { ok = false; break; }
        constexpr int CPR = D / 16;   // raw 16-byte chunks per key, and chunks per thread
        const uint8_t* raw = smem + L::RAW_OFF + st * L::RAW;
        // (a free stage also means that block gb - VST is done with: its scales, SST blocks back, too)
        if (!__all_sync(0xffffffffu, gb < VST || mbar_wait(&v_empty[dst_st], ((gb / VST) - 1) & 1, wc))) { ok = false; break; }
        if (warp == 12) {
          const float out = lane < 16 ? my_scale : lane == 16 ? vu.unit : __int_as_float(vu.far());
          if (lane < 18) scales[(gb % L::SST) * (L::SET / 4) + lane] = out;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[gb % L::SST]);
        }
        uint8_t* dst = smem + L::V_OFF + dst_st * L::TILE;
        auto convert = [&](int i, auto far_) {
          const int id = i * 128 + ct, row = id / CPR, c = id % CPR;
          const uint4 w = *reinterpret_cast<const uint4*>(raw + id * 16);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[2 * e] = e4m3x2_to_f16x2(u[e]);
            o[2 * e + 1] = e4m3x2_to_f16x2(u[e] >> 16);
          }
          if constexpr (decltype(far_)::value) {
            const float vs = __shfl_sync(0xffffffffu, my_scale, 8 + (row >> 4));   // (a warp's rows are of one group)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = scaled_bf16x2(o[e], vs);
          }
          if (key0 + row >= s.L) {   // past the end: what lies there is nobody's
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0u;
          }
          uint8_t* d = dst + (c >> 2) * L::SUB + row * 128;
          // 16-bit chunks 2c and 2c + 1 of the row; lanes of the second panel store them in the other order, so
          // that 8 lanes meet 8 different banks
          const int z = c >> 2;
          const int ca = ((2 * c + z) & 7) ^ (row & 7), cb = ((2 * c + 1 - z) & 7) ^ (row & 7);
          const uint4 first = make_uint4(o[0], o[1], o[2], o[3]), second = make_uint4(o[4], o[5], o[6], o[7]);
          *reinterpret_cast<uint4*>(d + (ca << 4)) = z ? second : first;
          *reinterpret_cast<uint4*>(d + (cb << 4)) = z ? first : second;
        };
        if (!vu.far()) {
#pragma unroll 4
          for (int i = 0; i < CPR; ++i) convert(i, Int<0>());
        } else {
#pragma unroll 1
          for (int i = 0; i < CPR; ++i) convert(i, Int<1>());
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[st]);
          mbar_arrive(&v_full[dst_st]);
        }
      }
    }
  } else {
    // =========================================================== softmax / epilogue (warps 0-7)
    set_regs_inc<L::SOFT_REGS>();
    const int x = warp >> 2;   // tile
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t s_addr = lane_base + L::s_col(x);
    const uint32_t o_addr = lane_base + L::o_col(x);
    const int ii = r / q.g, jj = r % q.g;
    int nb = 0, ni = 0, gb = 0;   // blocks and segments of this tile, blocks of the CTA so far
    bool ok = true;
    while (ok && wait_seg()) {
      // What the block loop needs of the segment; the rest is read again at its end (registers are short here, and
      // with shared memory taking nearly all of L1 a spilled one is a trip to L2).
      int n, key0, lim, lim_lo;
      float row_scale = 1.f;
      {
        const WideSeg s = read_seg();
        if (s.cnt == 0) break;
        n = x ? s.blocks[1] : s.blocks[0];
        key0 = s.t * 128;
        const int i0 = (2 * s.pair + x) * q.tq, qi = i0 + ii;
        const bool stored = ii < q.tq && qi < p.Nq;
        if (FP8 && stored) row_scale = q.q_scale[((int64_t)(s.b * p.Hkv + s.h) * q.g + jj) * p.Nq + qi];
        lim = stored && qi < s.n ? (p.causal ? max(s.L - s.n + qi + 1, 0) : s.L) : 0;   // keys < lim allowed
        lim_lo = min(p.causal ? s.L - s.n + i0 + 1 : s.L, s.L);                        // the tile's smallest
      }
      const float sl2 = FP8 ? row_scale : p.scale_log2;
      float m_ref = -INFINITY;   // reference max, exp2 domain
      float l = 0.f;
      float vref = kPagedLeastUnit;   // e4m3: O is in units of this / 2^7
      for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[x], (nb + j) & 1, wc))) { ok = false; break; }
        tc_fence_after();
        const int k0 = key0 + j * 128;
        if (k0 + 128 > lim_lo) {   // block straddles a mask edge: its scores are masked in place, 32 columns at a time
          const int keep = lim - k0;
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += 32) {
            uint32_t m[32];
            tmem_ld32(s_addr + c0, m);
            tmem_ld_wait();
            reg_fence32(m);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c0 + c >= keep) m[c] = __float_as_uint(-INFINITY);
            tmem_st32(s_addr + c0, m);
          }
          tmem_st_wait();
        }
        float alpha = 1.f, o_move;
        uint64_t rs2 = f2_make(0.f, 0.f);
        auto move_max = [&](float m_cand) {
          if (m_cand > m_ref + kPagedRescale) {
            alpha = ex2_approx(m_ref - m_cand);
            m_ref = m_cand;
          }
          return m_ref == -INFINITY ? 0.f : -m_ref;
        };
        // P of half h over score columns already read; O already holds PV up to block j - 1
        auto hand_over = [&](int h, const uint32_t (&pk)[32]) {
          tmem_st32(s_addr + 32 * h, pk);
          if (h == 0 && j >= 1 && __any_sync(0xffffffffu, o_move != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t orr[32];
              tmem_ld32(o_addr + c * 32, orr);
              tmem_ld_wait();
              reg_fence32(orr);
#pragma unroll
              for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * o_move);
              tmem_st32(o_addr + c * 32, orr);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * x + h]);
        };
        if constexpr (FP8) {
          // The scores are read twice, 64 at a time (registers and instruction cache are short here).  sc: K's scales
          // of the block's 8 groups of 16 keys, then what P takes of V's, then the units of O and whether scales are far apart.
          const int b = gb + j;
          if (!__all_sync(0xffffffffu, mbar_wait(&sc_full[b % L::SST], (b / L::SST) & 1, wc))) { ok = false; break; }
          const uint32_t sc = smem_u32(smem) + L::SC_OFF + (b % L::SST) * L::SET;
          auto scales4 = [&](int at, float (&f)[4]) {
            asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(sc + 4 * at));
          };
          auto load64 = [&](int h, uint32_t (&sr)[64]) {
            tmem_ld32(s_addr + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
            tmem_ld32(s_addr + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
            tmem_ld_wait();
            reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
            reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          };
          float m_cand = -INFINITY;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t sr[64];
            float ks[4];
            scales4(4 * h, ks);
            load64(h, sr);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
              for (int c = 16 * u; c < 16 * u + 16; c += 4) {
                m0 = max3f(m0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                m1 = max3f(m1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
              }
              m_cand = fmaxf(m_cand, fmaxf(m0, m1) * ks[u]);   // the scores are sr times the group's key scale
            }
          }
          const float neg = move_max(m_cand * sl2);
          const uint64_t negm2 = f2_make(neg, neg);
          o_move = alpha;
          float unit;
          uint32_t far;
          asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=f"(unit), "=r"(far) : "r"(sc + 64));
          if (unit != vref) {
            o_move *= vref / unit;
            vref = unit;
          }
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {   // the MMA takes each half as soon as it is ready
            uint32_t sr[64], pk[32];
            float ks[4], vs[4];
            scales4(4 * h, ks);
            scales4(8 + 4 * h, vs);
            load64(h, sr);
            auto weigh = [&](auto far_) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float kf = fmaf(ks[e >> 3], sl2, kPagedLeastScale), vf = vs[e >> 3];   // 8 pairs: one group
                const uint64_t pp = exp2_pair(sr[2 * e], sr[2 * e + 1], f2_make(kf, kf), negm2);
                rs2 = f2_add(rs2, pp);
                float p0, p1;
                f2_split(decltype(far_)::value ? pp : f2_mul(pp, f2_make(vf, vf)), p0, p1);
                pk[e] = decltype(far_)::value ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
              }
            };
            if (far) weigh(Int<1>()); else weigh(Int<0>());
            hand_over(h, pk);
          }
        } else {
          uint32_t sr[128];
#pragma unroll
          for (int c = 0; c < 128; c += 32) tmem_ld32(s_addr + c, *reinterpret_cast<uint32_t(*)[32]>(&sr[c]));
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 128; c += 32) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&sr[c]));
          float mxv[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // four independent chains
#pragma unroll
          for (int c = 0; c < 128; c += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mxv[u] = max3f(mxv[u], __uint_as_float(sr[c + 2 * u]), __uint_as_float(sr[c + 2 * u + 1]));
          const float neg = move_max(fmaxf(max3f(mxv[0], mxv[1], mxv[2]), mxv[3]) * sl2);
          const uint64_t sl2x2 = f2_make(sl2, sl2), negm2 = f2_make(neg, neg);
          o_move = alpha;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint64_t pp = exp2_pair(sr[64 * h + 2 * e], sr[64 * h + 2 * e + 1], sl2x2, negm2);
              rs2 = f2_add(rs2, pp);
              float p0, p1;
              f2_split(pp, p0, p1);
              pk[e] = pack_bf16x2(p0, p1);
            }
            hand_over(h, pk);
          }
        }
        float rs0, rs1;
        f2_split(rs2, rs0, rs1);
        l = l * alpha + (rs0 + rs1);
      }
      if (!ok) break;

      // ---- epilogue: O / l in bf16 and lse, or the segment's partial
      const WideSeg s = read_seg();
      release_seg();
      gb += s.cnt;
      const int qi = (2 * s.pair + x) * q.tq + ii;
      const bool stored = ii < q.tq && qi < p.Nq;
      const bool whole = s.t == 0 && s.cnt == s.T;
      const int64_t out = ((int64_t)(s.b * p.Hkv + s.h) * q.g + jj) * p.Nq + qi;
      const int64_t slot = (2 * (int64_t)cta + (s.first ? 0 : 1)) * 256 + 128 * x + r;
      if (tid == 0) {
        int2* info = p.info + (s.b * p.Hkv + s.h) * q.n_pairs + s.pair;
        if (s.t + s.cnt == s.T) info->y = whole ? -1 : cta;
        if (s.t == 0) info->x = 2 * cta + (s.first ? 0 : 1);
      }
      if (lim == 0 || n == 0) l = 0.f;
      if (n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&o_fin[x], ni & 1, wc))) { ok = false; break; }
        tc_fence_after();
      }
      float zero = 0.f;   // stays 0 unless O has a value that is not finite
      const float f = l != 0.f ? (FP8 ? vref * (1.f / kPagedPScale) : 1.f) * (whole ? 1.f / l : 1.f) : 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t orr[32];
        if (n > 0) {
          tmem_ld32(o_addr + c * 32, orr);
          tmem_ld_wait();
          reg_fence32(orr);
        }
        if (!stored) continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) zero = fmaf(__uint_as_float(orr[e]), 0.f, zero);
        if (whole) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = l != 0.f ? pack_bf16x2(__uint_as_float(orr[2 * e]) * f, __uint_as_float(orr[2 * e + 1]) * f) : 0u;
          uint4* dst = reinterpret_cast<uint4*>(p.o + out * D + 32 * c);   // (o is 16-byte aligned)
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        } else if (l != 0.f) {
#pragma unroll
          for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * f);
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            st_global_v8(p.part_o + slot * D + 32 * c + e, orr[e], orr[e + 1], orr[e + 2], orr[e + 3], orr[e + 4], orr[e + 5],
                         orr[e + 6], orr[e + 7]);
        }
      }
      // 0 * inf: a value behind a row's causal mask may have reached it
      if (p.causal && stored && l != 0.f && n > 0 && !(zero == 0.f)) q.redo[(s.b * p.Hkv + s.h) * q.n_pairs + s.pair] = 1;
      if (n > 0) {   // O has been read: the next segment's first PV may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[x]);
      }
      if (stored) {
        if (whole)
          p.lse[out] = l != 0.f ? (m_ref + lg2_approx(l)) * kPagedLn2 : -INFINITY;
        else
          p.part_ml[slot] = make_float2(m_ref, l);
      }
      nb += n;
      ni += (n > 0);
    }
  }

  // ---- teardown: every role has drained its asynchronous work
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// One query row by one warp, 32 keys at a time (a lane each for the scores, all lanes for each key's values): for pairs where
// a value of V that is not finite lies behind the mask of some row.  There the tensor core adds 0 * V = NaN to rows
// that do not see its key; here a row reads what it sees and nothing else.  sq: the warp's shared memory for the query.
template <int D>
__device__ __forceinline__ void paged_row(const PagedParams& p, int b, int h, int64_t row, int lim, int lane, float* sq) {
  constexpr int PER = D / 32;
  const bool fp8 = p.k_scale != nullptr;
  float acc[PER];
  __syncwarp();
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    sq[lane * PER + e] = __bfloat162float(p.q[row * D + lane * PER + e]);
    acc[e] = 0.f;
  }
  __syncwarp();
  auto e4m3 = [](uint32_t code) { return __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(code) & 0xffffu))); };
  float m = -INFINITY, l = 0.f;   // l: the lane's part
  for (int j0 = 0; j0 < lim; j0 += 32) {
    const int j = j0 + lane;
    const int id = j < lim ? p.page_table[(int64_t)b * p.max_pages + (j >> p.page_shift)] : -1;
    const bool seen = j < lim && unsigned(id) < unsigned(p.n_pages);   // (a page outside the pool has been reported)
    const int64_t in = (((int64_t)h << p.page_shift) + (j & ((1 << p.page_shift) - 1))) * D;   // element of the key in its page
    float s = 0.f, vs = 1.f;
    if (seen) {
      const uint8_t* k = p.k + uint64_t(id) * p.k_page_bytes;
      if (fp8) {
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint2 w = *reinterpret_cast<const uint2*>(k + in + 8 * c);
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(sq[8 * c + e], e4m3(((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 0xffu), s);
        }
        s *= p.k_scale[(int64_t)id * p.Hkv + h];
        vs = p.v_scale[(int64_t)id * p.Hkv + h];
      } else {
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(k + 2 * in + 16 * c);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(sq[8 * c + e], __uint_as_float((e & 1) ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16), s);
        }
      }
      s *= p.scale_log2;
    }
    float mx = seen ? s : -INFINITY;
#pragma unroll
    for (int z = 16; z > 0; z >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, z));
    mx = fmaxf(mx, m);
    const float base = mx == -INFINITY ? 0.f : mx, a = exp2f(m - base), w = seen ? exp2f(s - base) : 0.f;
    m = mx;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= a;
    const unsigned all = __ballot_sync(0xffffffffu, seen);
#pragma unroll 4
    for (int y = 0; y < 32; ++y) {
      const float wy = __shfl_sync(0xffffffffu, w, y), vy = __shfl_sync(0xffffffffu, vs, y);
      const int iy = __shfl_sync(0xffffffffu, id, y);
      const int64_t at = __shfl_sync(0xffffffffu, in, y) + lane * PER;
      if (!(all >> y & 1)) continue;
      const uint8_t* v = p.v + uint64_t(iy) * p.v_page_bytes;
#pragma unroll
      for (int e = 0; e < PER; ++e)
        acc[e] = fmaf(wy, (fp8 ? e4m3(v[at + e]) : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(v)[at + e])) * vy, acc[e]);
    }
  }
#pragma unroll
  for (int z = 16; z > 0; z >>= 1) l += __shfl_xor_sync(0xffffffffu, l, z);
#pragma unroll
  for (int e = 0; e < PER; ++e) p.o[row * D + lane * PER + e] = __float2bfloat16_rn(l != 0.f ? acc[e] / l : 0.f);
  if (lane == 0) p.lse[row] = l != 0.f ? (m + log2f(l)) * kPagedLn2 : -INFINITY;
}

// Whether a value that is not finite lies among the keys that some row of the pair does not see: new tokens from the pair's first
// position on, up to the end of its last block.  Elsewhere all rows see it, and O stands.  A whole CTA.  (Not inlined: that gave the
// merge more registers and took 1 us of a call of 30.)
template <int D>
__device__ __noinline__ bool wide_hidden_value(const WideParams& q, int b, int h, int pair, int T) {
  const PagedParams& p = q.p;
  const int L = paged_key_len(p, b), lo = max(L - paged_new_len(p, b) + 2 * pair * q.tq + 1, 0), hi = min(L, T * 128);
  const bool fp8 = p.k_scale != nullptr;
  const int cpr = D / (fp8 ? 16 : 8);   // 16-byte chunks of a key
  uint32_t bad = 0;
#pragma unroll 4
  for (int i = int(threadIdx.x); i < (hi - lo) * cpr; i += 256) {
    const int j = lo + i / cpr, id = p.page_table[(int64_t)b * p.max_pages + (j >> p.page_shift)];
    if (unsigned(id) >= unsigned(p.n_pages)) continue;
    const int64_t row = ((int64_t)h << p.page_shift) + (j & ((1 << p.page_shift) - 1));
    const uint4 w = reinterpret_cast<const uint4*>(p.v + uint64_t(id) * p.v_page_bytes)[row * cpr + i % cpr];
    bad |= fp8 ? not_finite<true>(w.x) | not_finite<true>(w.y) | not_finite<true>(w.z) | not_finite<true>(w.w)
               : not_finite<false>(w.x) | not_finite<false>(w.y) | not_finite<false>(w.z) | not_finite<false>(w.w);
  }
  return __syncthreads_or(bad != 0);
}

// Merges the pairs that several CTAs shared and writes the rows of pairs without keys: a row per warp at a time,
// 2 rows a warp (with 8, four CTAs a pair, latency kept it at 20 us on 256 pairs of 2 partials, 38 MB).  Of a pair whose O is not
// finite the first CTA finds out whether it has to be computed anew.
constexpr int kWideMergeCtas = 16;
template <int D>
__global__ void __launch_bounds__(256) fa_paged_wide_combine_kernel(const __grid_constant__ WideParams q) {
  const PagedParams& p = q.p;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x / kWideMergeCtas;
  const unsigned bh = item / q.n_pairs, pair = item % q.n_pairs, b = bh / p.Hkv;
  const int64_t at = (int64_t)b * q.n_pairs + pair;
  const bool has = p.plan[at + 1] > p.plan[at];
  const int2 info = p.info[item];
  if (blockIdx.x % kWideMergeCtas == 0 && q.redo[item] != 0 &&
      wide_hidden_value<D>(q, b, bh % p.Hkv, pair, p.plan[at + 1] - p.plan[at]) && threadIdx.x == 0)
    q.redo[item] = 2, q.redo[p.B * p.Hkv * q.n_pairs] = 1;
  if (has && info.y < 0) return;
  // (a CTA whose wait ran out leaves what the workspace held: then no slot may be taken from it)
  const bool found = has && unsigned(info.x) < 2u * p.n_warps && info.y < p.n_warps;
  const int rows = q.g * q.tq;   // of a tile
  for (int k = (blockIdx.x % kWideMergeCtas) * 8 + warp; k < 2 * rows; k += 8 * kWideMergeCtas) {
    const int x = k >= rows ? 1 : 0, r = k - x * rows;
    const int i = (2 * pair + x) * q.tq + r / q.g;
    if (i >= p.Nq) break;
    PagedMerge<D / 32> a;
    if (found) a.template gather<2>(p, info, 0, 1, 256, 128 * x + r, lane);
    a.store(p, ((int64_t)bh * q.g + r % q.g) * p.Nq + i, lane);
  }
}

// The pairs that have to be computed anew, their rows spread over all warps of the grid.  After the merge, and only under a
// causal mask.
template <int D>
__global__ void __launch_bounds__(256) fa_paged_wide_redo_kernel(const __grid_constant__ WideParams q) {
  const PagedParams& p = q.p;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int items = p.B * p.Hkv * q.n_pairs;
  if (q.redo[items] == 0) return;
  __shared__ float sq[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = int(gridDim.x) * 8, me = warp * int(gridDim.x) + int(blockIdx.x);
  const int rows = q.g * q.tq;   // of a tile
  int turn = 0;                  // the warp that takes the next pair's first row
  for (int base = 0; base < items; base += 32)
    for (unsigned flags = __ballot_sync(0xffffffffu, base + lane < items && q.redo[base + lane] == 2); flags != 0; flags &= flags - 1) {
      const int item = base + __ffs(flags) - 1;
      const int bh = item / q.n_pairs, pair = item % q.n_pairs, b = bh / p.Hkv;
      const int L = paged_key_len(p, b), n = paged_new_len(p, b);
      for (int k = me >= turn ? me - turn : me - turn + warps; k < 2 * rows; k += warps) {
        const int i = (2 * pair + k / rows) * q.tq + k % rows / q.g;
        if (i >= p.Nq) break;
        const int lim = i < n ? min(max(L - n + i + 1, 0), L) : 0;
        paged_row<D>(p, b, bh % p.Hkv, ((int64_t)bh * q.g + k % rows % q.g) * p.Nq + i, lim, lane, sq[warp]);
      }
      turn = (turn + 2 * rows) % warps;
    }
}

}  // namespace fa
