// Attention over a paged key/value cache for sm_100a: Nq new query rows per head against keys and
// values kept in pages of a common pool, query heads in groups that share one K/V head.
//
// Pool: [n_pages, Hkv, page, D], bf16 or e4m3 (one fp32 scale per page and head); sequence b holds
// L = key_lens[b] keys, key j in page page_table[b][j / page], row j % page.  The n = new_lens[b]
// queries stand at positions L - n .. L - 1; causal keeps key j <= L - n + i.  The R = (Hq / Hkv) Nq
// query rows of one K/V head are contiguous in q [B, Hq, Nq, D] and form tiles of 8, 16, 24 (32) rows; many
// rows take the tensor-memory path of paged_wide_sm100.cuh.
//
// Mathematics (the online softmax of the other kernels): s = tau q.k, running reference max m and
// sum l, O = sum 2^(s' - m) v with s' = s log2 e; partials of one row over disjoint keys merge by
// m* = max m_i, O = sum 2^(m_i - m*) O_i / sum 2^(m_i - m*) l_i.  With e4m3 pages k = c * ks, where
// ks is constant over a page, so ks multiplies the finished dot product and vs the probability (or V, see PagedUnit).
//
// Bound: HBM.  A key and its value are 4 D bytes (2 D in e4m3) for 4 D flop per row: at most 32
// flop per byte for 16 rows.  Each SM gets 23 bytes a cycle of the measured copy rate, i.e. 16 keys
// of bf16 at D = 128 every 350 cycles.  What has to be hidden is latency (copy, ldmatrix, a chain of MMAs,
// the exponentials), so the design is many independent warps with few registers:
//  * Both products are transposed, S^T = K Q^T and O^T = V^T P^T (m16n8k16: 16 keys or 16 features by 8
//    query rows), so that 8 rows fill the MMA; the other way round half of a 16-row tile, of
//    the accumulators and of the MMAs would be padding.  K comes by ldmatrix, V by ldmatrix.trans, P^T
//    turns from accumulator into operand by movmatrix.
//  * Every warp works alone: it walks its own contiguous share of all (sequence, head, key tile)s and
//    loads its tiles into a ring of its own (cp.async), with no barrier between warps.  Shares are equal to one tile
//    whatever the lengths are, nothing depends on the longest sequence, and the workspace (two partials per
//    warp) depends on the device alone.  A row tile that several warps shared is merged by
//    fa_paged_combine_kernel.
//  * 12 warps of 168 registers for 8 rows, 8 warps of 255 beyond, with rings of two tiles of 8 KB: what spills least.  Shared
//    memory is taken from L1, and where it takes nearly all of it a spilled register is a trip to L2: a third tile
//    costs 20 rows of D = 128 48.2 against 45.3 us in bf16, and gains nothing elsewhere (16 rows 58.2 against 57.7).
//    Tiles of 4 KB where an e4m3 tile's scores would not fit into the registers beside O: 32 rows of D = 64 39.4 -> 33.0 us (34.8
//    since scales may lie far apart), 24 of D = 128 49.3 -> 45.2 us (44; 16 rows, where they fit, 48 -> 56 us).
// Measured (B200, the whole call, 32/8 heads, D = 128): 64 sequences of 100 to 4000 keys, one query each, 90 us in bf16
// (6.0 TB/s of K and V, 91 % of the copy rate) and 57 us in e4m3 (4.7 TB/s; there the warps' own latency bounds:
// issue slots 47 % used, waits on memory rare); 16 heads x 65,536 keys, 8 queries, 91 us (5.9 TB/s); 8 x 32,768 keys
// e4m3, 64/8 heads, 93 us (5.8 TB/s).  About 10 us of a call are launch, look-ups, first loads and the merge.
// Tried and slower: tiles of 2 KB with 14 to 16 warps (57 -> 60 us e4m3), a loop over 16-key groups in place of unrolled
// tiles (57 -> 58 us), a 16-row tile with untransposed products (102 us e4m3), S by 8-bit MMAs with queries of two 8-bit parts
// (56 -> 59 us; 20 rows, D = 64: 28 -> 36 us, registers spill).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "sm100.cuh"

namespace fa {

enum : int { kStatusRange = 6 };   // a page number, length or position outside the cache

constexpr int kPagedMaxB = 4096;   // the prefix of the tile counts sits in shared memory
constexpr float kPagedRescale = 8.0f;   // the reference max moves only when a tile exceeds it by 2^8
constexpr float kPagedPScale = 128.0f;  // e4m3: probabilities enter the f16 MMA times 2^7 (at most 2^15)
constexpr float kPagedLeastUnit = 6.0185311e-36f;   // 2^-117, the least scale that the append gives
constexpr float kPagedFarUnit = 1.0995116e12f;      // 2^40

// Value scales of one row tile's stretch of keys, e4m3.  O is kept in units of `unit` / 2^7, and P enters the f16 product as
// p s 2^7 / unit, at most 2^15 where s <= unit.  But f16 ends at 2^-24: with the largest scale so far as the unit, a page 2^21
// below it loses bits and one 2^32 below it everything, also in rows that do not see the loud page, or see nothing but
// zeros in it.  So f16 is for scales within 2^8 of one another (it then loses 2^-24 of a page's own unit).  From the first scale
// on that lies further away the stretch is `far`: P enters as bf16 without the scale, V as bf16 times its scale (exact where
// that is a power of two), in units that leave room at both ends, 2^40 (O: up to 2^128, full precision down to 2^-93).
// That takes 2 to 3 times as long in the narrow kernels (64 ragged sequences 56 -> 159 us) and as long as ever in the wide one;
// to be ready for it costs calls that never meet it 1 to 2 % (32 rows of D = 64 33.0 -> 34.9 us, whole prompts 220 -> 228).
struct PagedUnit {
  float unit, least;   // least: of the scales so far; 0: far
  __device__ __forceinline__ void reset() {
    unit = kPagedLeastUnit;
    least = INFINITY;
  }
  __device__ __forceinline__ bool far() const { return least == 0.f; }
  // hi, lo: the largest and least scale of more pages.  True where the unit changed; O times `move` is what it was.
  __device__ __forceinline__ bool meet(float hi, float lo, float& move) {
    if ((hi <= unit && lo >= least) || far()) return false;
    const float was = unit;
    unit = fmaxf(unit, hi);
    least = fminf(least, lo);
    if (unit > 256.f * least) {
      unit = kPagedFarUnit;
      least = 0.f;
    }
    move = was / unit;
    return unit != was;
  }
};
constexpr float kPagedLeastScale = 1.4e-45f;   // 2^-149: a score scale that underflows to 0 makes NaN of a masked score, -inf
constexpr float kPagedLn2 = 0.69314718055994530942f;

struct PagedParams {
  const __nv_bfloat16* q;      // [B, Hq, Nq, D]
  const uint8_t* k;            // pool of keys
  const uint8_t* v;
  const float* k_scale;        // [n_pages, Hkv] (e4m3)
  const float* v_scale;
  __nv_bfloat16* o;            // [B, Hq, Nq, D]
  float* lse;                  // [B, Hq, Nq]
  float* part_o;               // [2 * warps][row tile][D] fp32, unnormalised
  float2* part_ml;             // [2 * warps][row tile]: m (log2 domain), l
  int* plan;                   // [B + 1]: prefix of the sequences' key tiles
  int2* info;                  // [B, Hkv, row_tiles]: slot of the first partial; warp of the last, or -1: no partials
  const int32_t* page_table;   // [B, max_pages]
  const int32_t* key_lens;     // [B]
  const int32_t* new_lens;     // [B] or null
  uint32_t k_page_bytes, v_page_bytes;   // from one page to the next
  int B, Hkv, Nq, R, row_tiles;         // R = rows per K/V head
  int n_pages, page_shift, max_pages;
  int n_warps;                 // of the whole grid (wide path: CTAs): how many hold partials
  int causal;
  float scale_log2;
};

// A plain load.  Not __ldg: these kernels start while the one before them on the stream may still write what they read
// (they wait for it first), and the read-only path wants data that is constant for a kernel's whole life.
template <typename T>
__device__ __forceinline__ T global_load(const T* p) { return *p; }

template <int OFF>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {   // 16 bytes from src + OFF
  asm volatile("cp.async.cg.shared.global [%0], [%1 + %2], 16;" :: "r"(dst), "l"(src), "n"(OFF) : "memory");
}
template <int OFF>
__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool valid) {   // zeros if not valid
  asm volatile("cp.async.cg.shared.global [%0], [%1 + %3], 16, %2;" :: "r"(dst), "l"(src), "r"(valid ? 16 : 0), "n"(OFF) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// c += a b, m16n8k16; bf16 or f16 operands, fp32 accumulator
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c = a b
template <bool F16>
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// two e4m3 codes (the low 16 bits of w) as f16x2: exact, NaN stays NaN
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}\n" : "=r"(r) : "r"(w));
  return r;
}
// the transpose of an 8 x 8 matrix of 16-bit elements, one row pair per lane
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// two f16 times s as bf16x2
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t w, float s) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_bf16x2(f.x * s, f.y * s);
}

// Nonzero where one of the values in w (two bf16 or four e4m3) is not finite.
template <bool FP8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  if constexpr (FP8) return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return (((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u);
}

// Keys of sequence b, clamped to what its row of the page table can hold; new tokens clamped to Nq.
__device__ __forceinline__ int paged_key_len(const PagedParams& p, int b) {
  const int L = p.key_lens[b];
  const long long cap = (long long)p.max_pages << p.page_shift;
  if (L < 0 || L > cap) record_status(kStatusRange);
  return L < 0 ? 0 : int(L > cap ? cap : L);
}
__device__ __forceinline__ int paged_new_len(const PagedParams& p, int b) {
  if (p.new_lens == nullptr) return p.Nq;
  const int n = p.new_lens[b];
  if (n < 0 || n > p.Nq) record_status(kStatusRange);
  return min(max(n, 0), p.Nq);
}

// How many warps share W tiles: no share is empty, so every partial between the first and the last warp of a
// row tile exists.
__device__ __forceinline__ int paged_sharers(long long W, int n_warps) { return int(W < n_warps ? W : n_warps); }
// First tile of sharer i of n < 2^15: floor(W i / n), by 32-bit divisions where W fits.
__device__ __forceinline__ long long paged_share(long long W, int i, int n) {
  if (W >> 32) return W * i / n;
  const unsigned q = unsigned(W) / unsigned(n), r = unsigned(W) % unsigned(n);
  return (long long)q * i + r * unsigned(i) / unsigned(n);
}

template <int D, bool FP8, int NG>
struct PagedLayout {
  static constexpr int ROWB = FP8 ? D : 2 * D;         // bytes of one key
  static constexpr int TILE = FP8 && (NG == 4 || (NG == 3 && D == 128)) ? 2048 : 4096;   // bytes of a tile's K, and of its V
  static constexpr int KT = TILE / ROWB;               // keys per tile: 16, 32 or 64
  static constexpr int GROUPS = KT / 16;               // 16-key groups: each inside one page
  static constexpr int CPR = ROWB / 16;                // 16-byte chunks per key
  static constexpr int WARPS = NG == 1 ? 12 : 8;
  static constexpr int STAGES = 2;
  static constexpr int STAGE = 2 * TILE + (FP8 ? 128 : 0);   // K, V, and the groups' scales
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int bytes(int B) { return RING + (B + 1) * 4; }
  // Byte offset of chunk c of row r, XOR-swizzled so that the 8 rows of an ldmatrix at one chunk
  // fall into different banks.
  static __device__ __forceinline__ int at(int r, int c) {
    if constexpr (ROWB == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return r * ROWB + ((c ^ (r & 7)) << 4);
  }
};

template <int N>
struct Int {
  static constexpr int value = N;
};

// Where a warp stands in the list of (sequence, head and row tile, key tile)s.
struct PagedPos {
  int b, h, rt, t;   // sequence, K/V head, row tile, key tile
  int T, L;          // key tiles and keys of sequence b
};

template <int D, bool FP8, int NG>
__global__ void __launch_bounds__(32 * PagedLayout<D, FP8, NG>::WARPS, 1) fa_paged_split_kernel(const PagedParams p) {
  using Lt = PagedLayout<D, FP8, NG>;
  constexpr int KT = Lt::KT, G = Lt::GROUPS, RT = 8 * NG, WARPS = Lt::WARPS, STAGES = Lt::STAGES, C = D / 16;
  extern __shared__ __align__(1024) uint8_t smem[];
  int* off = reinterpret_cast<int*>(smem + Lt::RING);   // [B + 1]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // a programmatic dependent launch: the kernel before it on the stream has to be complete from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- prefix of the sequences' key tiles: every thread sums a run of sequences, then the runs are scanned
  {
    __shared__ int runs[WARPS];
    const int per = (p.B + 32 * WARPS - 1) / (32 * WARPS);
    int sum = 0;
    for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
      const int T = paged_new_len(p, b) > 0 ? (paged_key_len(p, b) + KT - 1) / KT : 0;
      sum += T;
      off[b + 1] = sum;
    }
    int incl = sum;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += u;
    }
    if (lane == 31) runs[warp] = incl;
    __syncthreads();
    int base = incl - sum;
    for (int w = 0; w < warp; ++w) base += runs[w];
    for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) off[b + 1] += base;
    if (tid == 0) off[0] = 0;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = tid; b <= p.B; b += 32 * WARPS) p.plan[b] = off[b];
  }

  const int HR = p.Hkv * p.row_tiles;
  const long long W = (long long)off[p.B] * HR;
  // shares: warps of different SMs first, so that few tiles still spread over the whole device
  const int me = warp * int(gridDim.x) + int(blockIdx.x);
  const int sharers = paged_sharers(W, p.n_warps);
  if (me >= sharers) return;
  const long long w0 = paged_share(W, me, sharers), w1 = paged_share(W, me + 1, sharers);

  PagedPos ld;
  {
    const int want = (W >> 32) ? int(w0 / HR) : int(unsigned(w0) / unsigned(HR));   // the sequence with off[b] <= want < off[b + 1]
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (off[mid] <= want) lo = mid; else hi = mid;
    }
    ld.b = lo;
    ld.T = off[lo + 1] - off[lo];
    const long long rem = w0 - (long long)off[lo] * HR;
    const int hr = (rem >> 32) ? int(rem / ld.T) : int(unsigned(rem) / unsigned(ld.T));
    ld.t = int(rem - (long long)hr * ld.T);
    ld.h = hr / p.row_tiles;
    ld.rt = hr % p.row_tiles;
    ld.L = paged_key_len(p, lo);
  }
  PagedPos cp = ld;
  auto advance = [&](PagedPos& x) {
    if (++x.t < x.T) return;
    x.t = 0;
    if (++x.rt < p.row_tiles) return;
    x.rt = 0;
    if (++x.h < p.Hkv) return;
    x.h = 0;
    do ++x.b; while (x.b < p.B && off[x.b + 1] == off[x.b]);
    if (x.b < p.B) {
      x.T = off[x.b + 1] - off[x.b];
      x.L = paged_key_len(p, x.b);
    }
  };

  const uint32_t ring = smem_u32(smem) + warp * STAGES * Lt::STAGE;
  const int page_mask = (1 << p.page_shift) - 1;
  int ids[G];   // pages of the groups of the tile that is loaded next
  auto look_up = [&]() {
#pragma unroll
    for (int x = 0; x < G; ++x) {
      const int key = ld.t * KT + 16 * x;
      ids[x] = key < ld.L ? global_load(p.page_table + (int64_t)ld.b * p.max_pages + (key >> p.page_shift)) : 0;
    }
  };
  // A lane copies chunk c of keys r0, r0 + RPI, ... of each group.  RPI is a power of two and r0 below it, so the swizzle
  // of key i RPI + r0 is that of r0 with the bits of i RPI flipped in.
  constexpr int RPI = 32 / Lt::CPR;   // keys per warp-wide copy
  const int c0 = lane % Lt::CPR, r0 = lane / Lt::CPR;
  const uint32_t lane_at = uint32_t(Lt::at(r0, c0)), lane_from = uint32_t(r0 * Lt::ROWB + c0 * 16);
  auto load = [&](int stage) {
    const uint32_t dst = ring + stage * Lt::STAGE;
#pragma unroll
    for (int x = 0; x < G; ++x) {
      const int key = ld.t * KT + 16 * x;
      const bool ok = unsigned(ids[x]) < unsigned(p.n_pages);
      if (!ok) record_status(kStatusRange);
      const unsigned page = ok ? ids[x] : 0;
      const unsigned in = ((unsigned(ld.h) << p.page_shift) + (key & page_mask)) * Lt::ROWB + lane_from;   // within the page
      const uint8_t* ks = p.k + (uint64_t(page) * p.k_page_bytes + in);
      const uint8_t* vs = p.v + (uint64_t(page) * p.v_page_bytes + in);
      const int left = ok ? ld.L - key : 0;
      auto copy = [&](auto all) {
        auto one = [&](auto i_) {
          constexpr int i = decltype(i_)::value;
          if constexpr (i < 16 / RPI) {
            constexpr int row = 16 * i * RPI / 16;
            // (at(r0, c0) has its swizzle in bits 4-6)
            const uint32_t at = Lt::ROWB == 64 ? lane_at + row * 64 : (lane_at ^ ((row & 7) << 4)) + row * Lt::ROWB;
            const uint32_t to = dst + 16 * x * Lt::ROWB + at;
            if constexpr (decltype(all)::value) {
              cp_async16<row * Lt::ROWB>(to, ks);
              cp_async16<row * Lt::ROWB>(to + Lt::TILE, vs);
            } else {
              cp_async16_if<row * Lt::ROWB>(to, ks, row + r0 < left);
              cp_async16_if<row * Lt::ROWB>(to + Lt::TILE, vs, row + r0 < left);
            }
          }
        };
        one(Int<0>()); one(Int<1>()); one(Int<2>()); one(Int<3>()); one(Int<4>()); one(Int<5>()); one(Int<6>()); one(Int<7>());
      };
      if (left >= 16) copy(Int<1>()); else copy(Int<0>());   // past the end: zeros
      if constexpr (FP8) {
        if (lane < 2)
          cp_async4(dst + 2 * Lt::TILE + 8 * x + 4 * lane, (lane == 0 ? p.k_scale : p.v_scale) + (uint64_t(page) * p.Hkv + ld.h),
                    left > 0);
      }
    }
  };

  long long at_load = w0;
  look_up();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    if (at_load < w1) {
      load(s);
      advance(ld);
      if (++at_load < w1) look_up();
    }
    cp_async_commit();
  }

  // Fragments: lane = 4 g + t4.  As operand column a lane holds query row g of each group of 8, as
  // accumulator columns the rows 2 t4 and 2 t4 + 1; accumulator rows are keys (or features) g and g + 8.
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t qf[NG][C][2];
  float o[NG][C][4];
  float m[NG][2], l[NG][2], sc[NG][2];   // rows 2 t4 + i; sc: score scale in the log2 domain
  int lim[NG][2], limg[NG], lim_lo;      // keys < lim allowed; limg: of row g; lim_lo: the smallest that is not zero
  PagedUnit vu;                          // e4m3: the units of O
  vu.reset();
  float unit = 0.f;                      // kPagedPScale / vu.unit
  int stage = 0;
  bool fresh = true;
  long long seg = w0;                    // first tile of the running segment
  for (long long w = w0; w < w1; ++w) {
    if (fresh) {
      // ---- queries and limits of this row tile
      fresh = false;
      seg = w;
      const int h = cp.h, rt = cp.rt;
      const int n = paged_new_len(p, cp.b);
      const __nv_bfloat16* qb = p.q + ((int64_t)(cp.b * p.Hkv + h) * p.R + rt * RT) * D;
      lim_lo = cp.L;
#pragma unroll
      for (int ng = 0; ng < NG; ++ng) {
        const int row = rt * RT + 8 * ng + g, qi = row % p.Nq;
        const bool real = row < p.R;
        limg[ng] = real && qi < n ? (p.causal ? max(min(cp.L, cp.L - n + qi + 1), 0) : cp.L) : 0;
        if (limg[ng] > 0) lim_lo = min(lim_lo, limg[ng]);   // a row without keys is dropped at the end instead
        float rs = p.scale_log2;
        if constexpr (FP8) {
          // f16 queries: each row times a power of two that puts its largest element into [2^14, 2^15)
          const uint2* src = reinterpret_cast<const uint2*>(qb + (int64_t)(8 * ng + g) * D);
          uint2 w2[C];
          float mx = 0.f;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            w2[c] = real ? src[c * 4 + t4] : make_uint2(0u, 0u);
            mx = max3f(mx, fabsf(__uint_as_float(w2[c].x << 16)), fabsf(__uint_as_float(w2[c].x & 0xffff0000u)));
            mx = max3f(mx, fabsf(__uint_as_float(w2[c].y << 16)), fabsf(__uint_as_float(w2[c].y & 0xffff0000u)));
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const int e = min(max(int(__float_as_uint(mx) >> 23) - 127, -100), 127);
          const bool scaled = mx > 0.f && mx < INFINITY;
          const float up = scaled ? __uint_as_float(uint32_t(127 + 14 - e) << 23) : 1.f;    // 2^(14 - e)
          rs = fmaxf(rs * (scaled ? __uint_as_float(uint32_t(127 - 14 + e) << 23) : 1.f), kPagedLeastScale);
#pragma unroll
          for (int c = 0; c < C; ++c) {
            qf[ng][c][0] = pack_f16x2(__uint_as_float(w2[c].x << 16) * up, __uint_as_float(w2[c].x & 0xffff0000u) * up);
            qf[ng][c][1] = pack_f16x2(__uint_as_float(w2[c].y << 16) * up, __uint_as_float(w2[c].y & 0xffff0000u) * up);
          }
        } else {
          const uint32_t* src = reinterpret_cast<const uint32_t*>(qb + (int64_t)(8 * ng + g) * D);
#pragma unroll
          for (int c = 0; c < C; ++c) {
            qf[ng][c][0] = real ? src[c * 8 + t4] : 0u;
            qf[ng][c][1] = real ? src[c * 8 + 4 + t4] : 0u;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lim[ng][i] = __shfl_sync(0xffffffffu, limg[ng], 4 * (2 * t4 + i));
          sc[ng][i] = FP8 ? __shfl_sync(0xffffffffu, rs, 4 * (2 * t4 + i)) : rs;
          m[ng][i] = -INFINITY;
          l[ng][i] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[ng][c][e] = 0.f;
      }
      lim_lo = __reduce_min_sync(0xffffffffu, lim_lo);
      vu.reset();
      unit = kPagedPScale / vu.unit;
    }

    // ---- the next tile of the list goes into the stage that the previous iteration emptied
    cp_async_wait<STAGES - 2>();
    __syncwarp();
    {
      const int into = stage == 0 ? STAGES - 1 : stage - 1;
      if (at_load < w1) {
        load(into);
        advance(ld);
        if (++at_load < w1) look_up();
      }
      cp_async_commit();
    }
    const uint32_t kt = ring + stage * Lt::STAGE, vt = kt + Lt::TILE;
    const int k0 = cp.t * KT;

    // ---- S^T = K Q^T: per 16 keys, two chains of MMAs over the features
    float s[G][NG][4];
#pragma unroll
    for (int x = 0; x < G; ++x) {
      float s2[NG][4];
      constexpr int BATCH = FP8 || NG > 1 ? 4 : 8;   // chunks loaded ahead of their MMAs
#pragma unroll
      for (int c0 = 0; c0 < Lt::CPR; c0 += BATCH) {
        uint32_t r[BATCH / 2][4];   // keys 0-7 and 8-15 at chunk c, keys 0-7 and 8-15 at chunk c + 1
#pragma unroll
        for (int y = 0; y < BATCH / 2; ++y)
          ldsm4(r[y], kt + Lt::at(16 * x + (lane & 15), c0 + 2 * y + (lane >> 4)));
#pragma unroll
        for (int y = 0; y < BATCH / 2; ++y) {
          if constexpr (FP8) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t a0 = e4m3x2_to_f16x2(r[y][2 * z]), a2 = e4m3x2_to_f16x2(r[y][2 * z] >> 16);
              const uint32_t a1 = e4m3x2_to_f16x2(r[y][2 * z + 1]), a3 = e4m3x2_to_f16x2(r[y][2 * z + 1] >> 16);
              const int c = c0 + 2 * y + z;
#pragma unroll
              for (int ng = 0; ng < NG; ++ng) {
                if (c < 2)
                  mma16816_first<true>(z == 0 ? s[x][ng] : s2[ng], a0, a1, a2, a3, qf[ng][c][0], qf[ng][c][1]);
                else
                  mma16816<true>(z == 0 ? s[x][ng] : s2[ng], a0, a1, a2, a3, qf[ng][c][0], qf[ng][c][1]);
              }
            }
          } else {
            const int c = c0 / 2 + y;
#pragma unroll
            for (int ng = 0; ng < NG; ++ng) {
              if (c < 2)
                mma16816_first<false>((y & 1) == 0 ? s[x][ng] : s2[ng], r[y][0], r[y][1], r[y][2], r[y][3], qf[ng][c][0], qf[ng][c][1]);
              else
                mma16816<false>((y & 1) == 0 ? s[x][ng] : s2[ng], r[y][0], r[y][1], r[y][2], r[y][3], qf[ng][c][0], qf[ng][c][1]);
            }
          }
        }
      }
#pragma unroll
      for (int ng = 0; ng < NG; ++ng)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[x][ng][e] += s2[ng][e];
    }
    float vsc[G];
    if constexpr (FP8) {
#pragma unroll
      for (int x = 0; x < G; ++x) {
        float ks;
        asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(ks), "=f"(vsc[x]) : "r"(kt + 2 * Lt::TILE + 8 * x));
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][ng][e] *= ks;
      }
    }
    if (k0 + KT > lim_lo) {
#pragma unroll
      for (int x = 0; x < G; ++x)
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k0 + 16 * x + g + 8 * (e >> 1) >= lim[ng][e & 1]) s[x][ng][e] = -INFINITY;
    }

    // ---- online softmax.  The reference max of a row moves only when a score passes it by 2^8; whether any
    // does is one vote, and only then the rows' maxima are formed across the lanes.  o is rescaled by alpha
    // (and, e4m3, by the value scale's move), l by alpha.
    float alpha[NG][2], vmove = 1.f;
    bool over = false;
#pragma unroll
    for (int ng = 0; ng < NG; ++ng)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = s[0][ng][i];
#pragma unroll
        for (int x = 0; x < G; ++x) mx = max3f(mx, s[x][ng][i], s[x][ng][2 + i]);
        alpha[ng][i] = mx * sc[ng][i];   // the lane's own maximum, for now
        over |= alpha[ng][i] > m[ng][i] + kPagedRescale;
      }
    if constexpr (FP8) {
      float hi = 0.f, lo = INFINITY;   // (groups past the end have scale 0)
#pragma unroll
      for (int x = 0; x < G; ++x) {
        hi = fmaxf(hi, vsc[x]);
        lo = vsc[x] > 0.f ? fminf(lo, vsc[x]) : lo;
      }
      if (vu.meet(hi, lo, vmove)) {   // the same in every lane
        unit = kPagedPScale / vu.unit;
        over = true;
      }
#pragma unroll
      for (int x = 0; x < G; ++x) vsc[x] *= unit;
    }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int ng = 0; ng < NG; ++ng) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = alpha[ng][i];
#pragma unroll
          for (int z = 4; z < 32; z <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, z));
          alpha[ng][i] = 1.f;
          if (mx > m[ng][i] + kPagedRescale) {
            alpha[ng][i] = ex2_approx(m[ng][i] - mx);
            m[ng][i] = mx;
          }
          l[ng][i] *= alpha[ng][i];
          alpha[ng][i] *= vmove;
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[ng][c][e] *= alpha[ng][e & 1];
      }
    }
    // P^T as operand columns; 16-bit parts: f16 (e4m3, times the page's value scale; bf16 where scales lie far apart), else
    // bf16 in two parts for up to 8 rows: the product is not what bounds the kernel, and P then has 16 bits
    constexpr bool LOW = !FP8 && NG == 1;
    uint32_t pf[G][NG][2], pl[LOW ? G : 1][2];
    const bool far = FP8 && vu.far();
#pragma unroll
    for (int ng = 0; ng < NG; ++ng) {
      const float n0 = m[ng][0] == -INFINITY ? 0.f : -m[ng][0], n1 = m[ng][1] == -INFINITY ? 0.f : -m[ng][1];
#pragma unroll
      for (int x = 0; x < G; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float p0 = ex2_approx(fmaf(s[x][ng][2 * y], sc[ng][0], n0)), p1 = ex2_approx(fmaf(s[x][ng][2 * y + 1], sc[ng][1], n1));
          l[ng][0] += p0;
          l[ng][1] += p1;
          if constexpr (FP8) {
            pf[x][ng][y] = movmatrix_trans(far ? pack_bf16x2(p0, p1) : pack_f16x2(p0 * vsc[x], p1 * vsc[x]));
          } else {
            const uint32_t hi = pack_bf16x2(p0, p1);
            pf[x][ng][y] = movmatrix_trans(hi);
            if constexpr (LOW)
              pl[x][y] = movmatrix_trans(pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u)));
          }
        }
    }

    // ---- O^T += V^T P^T.  A value that is not finite must not reach a row that does not see its key (0 * inf):
    // where rows see different keys of the tile and such a value is there, it is taken out of the
    // product and its effect is added to the rows that do see it.  That, and scales far apart, in a loop of little code.
    bool careful = false;
    if (lim_lo < min(cp.L, k0 + KT)) {
      uint32_t bad = 0;
#pragma unroll
      for (int x = 0; x < Lt::TILE / 512; ++x) {
        uint32_t q4[4];
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(q4[0]), "=r"(q4[1]), "=r"(q4[2]), "=r"(q4[3])
                     : "r"(vt + 16 * (32 * x + lane)));
#pragma unroll
        for (int e = 0; e < 4; ++e) bad |= not_finite<FP8>(q4[e]);
      }
      careful = __any_sync(0xffffffffu, bad != 0);
    }
    const int vrow = (lane & 7) + ((lane >> 4) << 3), vchunk = (lane >> 3) & 1;
    // operand rows: the 16 features of a block, in order (bf16) or the even then the odd ones (e4m3)
    auto values = [&](const uint32_t (&r)[4], int z, uint32_t (&a)[4]) {
      if constexpr (FP8) {   // r[z], r[2 + z]: keys 0-7 and 8-15 of chunk z
        a[0] = e4m3x2_to_f16x2(__byte_perm(r[z], 0, 0x4420));
        a[1] = e4m3x2_to_f16x2(__byte_perm(r[z], 0, 0x4431));
        a[2] = e4m3x2_to_f16x2(__byte_perm(r[2 + z], 0, 0x4420));
        a[3] = e4m3x2_to_f16x2(__byte_perm(r[2 + z], 0, 0x4431));
      } else {               // keys 0-7 at chunks 0 and 1, keys 8-15 at chunks 0 and 1
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = r[e];
      }
    };
    constexpr int PER = FP8 ? 2 : 1;   // feature blocks per ldmatrix
    if (!careful && !far) {
#pragma unroll
      for (int x = 0; x < G; ++x) {
        constexpr int BATCH = C / PER < 4 ? C / PER : 4;
#pragma unroll
        for (int c0 = 0; c0 < C / PER; c0 += BATCH) {
          uint32_t r[BATCH][4];
#pragma unroll
          for (int y = 0; y < BATCH; ++y) ldsm4_trans(r[y], vt + Lt::at(16 * x + vrow, 2 * (c0 + y) + vchunk));
#pragma unroll
          for (int y = 0; y < BATCH; ++y)
#pragma unroll
            for (int z = 0; z < PER; ++z) {
              uint32_t a[4];
              values(r[y], z, a);
              const int c = PER * (c0 + y) + z;
#pragma unroll
              for (int ng = 0; ng < NG; ++ng) mma16816<FP8>(o[ng][c], a[0], a[1], a[2], a[3], pf[x][ng][0], pf[x][ng][1]);
              if constexpr (LOW) mma16816<false>(o[0][c], a[0], a[1], a[2], a[3], pl[x][0], pl[x][1]);
            }
        }
      }
    } else {
      constexpr uint32_t kOne = FP8 ? 0x3c00u : 0x3f80u, kExp = FP8 ? 0x7c00u : 0x7f80u;   // 1, and the exponent's bits
#pragma unroll 1
      for (int x = 0; x < G; ++x) {
        uint32_t see[NG][2], px[NG][2], plx[2] = {0u, 0u};   // see: 1 where row g sees the key
        float vx = 0.f;                                      // the group's value scale in units of O
        if constexpr (FP8) {
#pragma unroll
          for (int z = 0; z < G; ++z)
            if (z == x) vx = vsc[z];
        }
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int key = k0 + 16 * x + 8 * y + 2 * t4;
            see[ng][y] = (key < limg[ng] ? kOne : 0u) | (key + 1 < limg[ng] ? kOne << 16 : 0u);
#pragma unroll
            for (int z = 0; z < G; ++z)
              if (z == x) {
                px[ng][y] = pf[z][ng][y];
                if constexpr (LOW) plx[y] = pl[z][y];
              }
          }
#pragma unroll
        for (int cc = 0; cc < C / PER; ++cc) {
          uint32_t r[4];
          ldsm4_trans(r, vt + Lt::at(16 * x + vrow, 2 * cc + vchunk));
#pragma unroll
          for (int z = 0; z < PER; ++z) {
            uint32_t a[4], up[4], dn[4];
            values(r, z, a);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t keep = 0;
              up[e] = dn[e] = 0;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t v = (a[e] >> (16 * q)) & 0xffffu;
                const bool special = (v & kExp) == kExp, nan = special && (v & ~kExp & 0x7fffu) != 0;
                if (!special || !careful) keep |= 0xffffu << (16 * q);
                if (careful && (nan || (special && !(v & 0x8000u)))) up[e] |= kOne << (16 * q);
                if (careful && (nan || (special && (v & 0x8000u)))) dn[e] |= kOne << (16 * q);
              }
              a[e] &= keep;
            }
            uint32_t b[4];   // far: the values in bf16, and no f16 product
            if constexpr (FP8) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                b[e] = far ? scaled_bf16x2(a[e], vx) : 0u;
                a[e] = far ? 0u : a[e];
              }
            }
            const int c = PER * cc + z;
#pragma unroll
            for (int ng = 0; ng < NG; ++ng) {
              float cu[4] = {0.f, 0.f, 0.f, 0.f}, cd[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816<FP8>(o[ng][c], a[0], a[1], a[2], a[3], far ? 0u : px[ng][0], far ? 0u : px[ng][1]);
              if constexpr (FP8) mma16816<false>(o[ng][c], b[0], b[1], b[2], b[3], far ? px[ng][0] : 0u, far ? px[ng][1] : 0u);
              if constexpr (LOW) mma16816<false>(o[0][c], a[0], a[1], a[2], a[3], plx[0], plx[1]);
              mma16816<FP8>(cu, up[0], up[1], up[2], up[3], see[ng][0], see[ng][1]);
              mma16816<FP8>(cd, dn[0], dn[1], dn[2], dn[3], see[ng][0], see[ng][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (cu[e] > 0.f) o[ng][c][e] += INFINITY;
                if (cd[e] > 0.f) o[ng][c][e] -= INFINITY;
              }
            }
          }
        }
      }
    }
    __syncwarp();

    // ---- end of the segment: this row tile's last key tile, or this warp's last
    if (cp.t + 1 == cp.T || w + 1 == w1) {
      const bool whole = cp.t + 1 == cp.T && w - seg + 1 == cp.T;
      const int h = cp.h, rt = cp.rt;
      if (lane == 0) {
        int2* info = p.info + (cp.b * p.Hkv + h) * p.row_tiles + rt;
        if (cp.t + 1 == cp.T) info->y = whole ? -1 : me;
        if (cp.t - int(w - seg) == 0) info->x = 2 * me + (seg == w0 ? 0 : 1);
      }
#pragma unroll
      for (int ng = 0; ng < NG; ++ng)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float lr = l[ng][i];
#pragma unroll
          for (int z = 4; z < 32; z <<= 1) lr += __shfl_xor_sync(0xffffffffu, lr, z);
          const int row = 8 * ng + 2 * t4 + i;
          if (rt * RT + row >= p.R) continue;
          const bool dead = lim[ng][i] == 0;
          if (dead) lr = 0.f;
          const float f = (FP8 ? vu.unit * (1.f / kPagedPScale) : 1.f) * (whole ? (lr != 0.f ? 1.f / lr : 0.f) : 1.f);
          const int64_t out = (int64_t)(cp.b * p.Hkv + h) * p.R + rt * RT + row;
          const int64_t slot = (2 * (int64_t)me + (seg == w0 ? 0 : 1)) * RT + row;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float a = dead ? 0.f : o[ng][c][i] * f, b = dead ? 0.f : o[ng][c][2 + i] * f;
            if constexpr (FP8) {
              const int at = 16 * c + 2 * g;
              if (whole)
                *reinterpret_cast<uint32_t*>(p.o + out * D + at) = pack_bf16x2(a, b);
              else
                *reinterpret_cast<float2*>(p.part_o + slot * D + at) = make_float2(a, b);
            } else {
              const int at = 16 * c + g;
              if (whole) {
                p.o[out * D + at] = __float2bfloat16_rn(a);
                p.o[out * D + at + 8] = __float2bfloat16_rn(b);
              } else {
                p.part_o[slot * D + at] = a;
                p.part_o[slot * D + at + 8] = b;
              }
            }
          }
          if (g == 0) {
            if (whole)
              p.lse[out] = lr != 0.f ? (m[ng][i] + lg2_approx(lr)) * kPagedLn2 : -INFINITY;
            else
              p.part_ml[slot] = make_float2(m[ng][i], lr);
          }
        }
      fresh = true;
    }
    advance(cp);
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
}

// Running merge of partials: m, l and a lane's features of O.
template <int PER>
struct PagedMerge {
  float acc[PER], m, l;
  __device__ __forceinline__ PagedMerge() : m(-INFINITY), l(0.f) {
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  }
  // N partials at once: their maximum first, then all weights side by side.  l1 = 0: no key seen there (m1 may be -inf)
  template <int N>
  __device__ __forceinline__ void add(const float (&m1)[N], const float (&l1)[N], const float (&x)[N][PER]) {
    float mx = m;
#pragma unroll
    for (int u = 0; u < N; ++u) mx = l1[u] != 0.f ? fmaxf(mx, m1[u]) : mx;
    const float base = mx == -INFINITY ? 0.f : mx;
    const float a = ex2_approx(m - base);
    m = mx;
    l *= a;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= a;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const bool seen = l1[u] != 0.f;
      const float c = ex2_approx(m1[u] - base);
      l += seen ? l1[u] * c : 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] += seen ? x[u][e] * c : 0.f;
    }
  }
  // partials sub, sub + step, ... of one row, N in flight; the first partial may be its warp's (CTA's) second slot,
  // the others are the first ones of theirs
  template <int N>
  __device__ __forceinline__ void gather(const PagedParams& p, int2 info, int sub, int step, int rows, int srow, int lane) {
    const int first = info.x >> 1;
    for (int w0 = first + sub; w0 <= info.y; w0 += N * step) {
      float m1[N], l1[N], x[N][PER];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int w = w0 + u * step;
        m1[u] = l1[u] = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) x[u][e] = 0.f;
        if (w > info.y) continue;
        const int64_t slot = (int64_t)(w == first ? info.x : 2 * w) * rows + srow;
        const float2 ml = p.part_ml[slot];
        m1[u] = ml.x;
        l1[u] = ml.y;
        const float* from = p.part_o + slot * (32 * PER) + lane * PER;
        if constexpr (PER == 4) {
          const float4 f = *reinterpret_cast<const float4*>(from);
          x[u][0] = f.x; x[u][1] = f.y; x[u][2] = f.z; x[u][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(from);
          x[u][0] = f.x; x[u][1] = f.y;
        }
      }
      add<N>(m1, l1, x);
    }
  }
  __device__ __forceinline__ void store(const PagedParams& p, int64_t row, int lane) const {
    const float inv = l != 0.f ? 1.f / l : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * (32 * PER) + lane * PER);
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0) p.lse[row] = l != 0.f ? (m + lg2_approx(l)) * kPagedLn2 : -INFINITY;
  }
};

// Merges the partials of query rows that several warps made, WPR warps of a CTA per row, N partials in flight per warp.  Rows of a row
// tile that one warp had whole are done already.  Also writes the rows of sequences without keys or
// without new tokens: O = 0, lse = -inf.
template <int D, int WPR, int N>
__global__ void __launch_bounds__(256) fa_paged_combine_kernel(const PagedParams p, const int tile_rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int PER = D / 32, RPC = 8 / WPR;   // features per lane, rows per CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  const unsigned row = blockIdx.x * RPC + warp / WPR;   // of [B, Hkv, R]; B Hq Nq < 2^31
  const bool real = row < unsigned(p.B) * p.Hkv * p.R;
  const unsigned bh = real ? row / p.R : 0, r = row % p.R, b = bh / p.Hkv;
  const bool has = p.plan[b + 1] > p.plan[b];
  const int2 info = p.info[(int64_t)bh * p.row_tiles + r / tile_rows];
  const bool whole = has && info.y < 0;
  PagedMerge<PER> a;
  if (real && has && !whole) a.template gather<N>(p, info, sub, WPR, tile_rows, r % tile_rows, lane);
  if constexpr (WPR > 1) {
    __shared__ float sm[8], sl[8], so[8][D];
    if (lane == 0) {
      sm[warp] = a.m;
      sl[warp] = a.l;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) so[warp][lane * PER + e] = a.acc[e];
    __syncthreads();
    if (sub != 0) return;
    float m1[WPR - 1], l1[WPR - 1], x[WPR - 1][PER];
#pragma unroll
    for (int y = 1; y < WPR; ++y) {
      m1[y - 1] = sm[warp + y];
      l1[y - 1] = sl[warp + y];
#pragma unroll
      for (int e = 0; e < PER; ++e) x[y - 1][e] = so[warp + y][lane * PER + e];
    }
    a.template add<WPR - 1>(m1, l1, x);
  }
  if (real && !whole) a.store(p, row, lane);
}

}  // namespace fa
