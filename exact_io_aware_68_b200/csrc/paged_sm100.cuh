// Attention over a paged key/value cache for sm_100a: Nq new query rows per head against keys and
// values kept in pages of a common pool, query heads in groups that share one K/V head.
//
// Pool: [n_pages, Hkv, page, D], bf16 or e4m3 (one fp32 scale per page and head); sequence b holds
// L = key_lens[b] keys, key j in page page_table[b][j / page], row j % page.  The n = new_lens[b]
// queries stand at positions L - n .. L - 1; causal keeps key j <= L - n + i.  The R = (Hq / Hkv) Nq
// query rows of one K/V head are contiguous in q [B, Hq, Nq, D] and form tiles of 8 or 16 rows.
//
// Mathematics (the online softmax of the other kernels): s = tau q.k, running reference max m and
// sum l, O = sum 2^(s' - m) v with s' = s log2 e; partials of one row over disjoint keys merge by
// m* = max m_i, O = sum 2^(m_i - m*) O_i / sum 2^(m_i - m*) l_i.  With e4m3 pages k = c * ks, where
// ks is constant over a page, so ks multiplies the finished dot product and vs the probability.
//
// Bound: HBM.  A key and its value are 4 D bytes (2 D in e4m3) for 4 D flop per row: at most 16
// flop per byte for 16 rows.  Each SM gets 23 bytes a cycle of the measured copy rate, i.e. a
// 16-key tile of bf16 at D = 128 every 350 cycles, in which one warp's m16n8k16 MMAs take 64.
// The MMA shape with 16 rows wastes nothing that is short, and needs no exchange between warps, so
// every warp works alone: it walks its own contiguous share of all (sequence, head, key tile)s,
// loads tiles of 4 KB of K and 4 KB of V into a ring of its own (cp.async, 3 deep: 16 KB in flight
// per warp, 128 KB per SM) and multiplies them out of shared memory.  Shares are equal to one tile whatever
// the lengths are, nothing depends on the longest sequence, and the workspace (two partials per
// warp) depends on the device alone.  A row tile that several warps shared is merged by
// fa_paged_combine_kernel.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "sm100.cuh"

namespace fa {

enum : int { kStatusRange = 6 };   // a page number, length or position outside the cache

constexpr int kPagedWarps = 8;
constexpr int kPagedStages = 3;
constexpr int kPagedMaxB = 4096;   // the prefix of the tile counts sits in shared memory
constexpr float kPagedRescale = 8.0f;   // the reference max moves only when a tile exceeds it by 2^8
constexpr float kPagedPScale = 128.0f;  // e4m3: probabilities enter the f16 MMA times 2^7 (at most 2^15)
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
  const int32_t* page_table;   // [B, max_pages]
  const int32_t* key_lens;     // [B]
  const int32_t* new_lens;     // [B] or null
  int64_t k_page_bytes, v_page_bytes;   // from one page to the next
  int B, Hkv, Nq, R, row_tiles;         // R = rows per K/V head
  int n_pages, page_shift, max_pages;
  int n_warps;                 // of the whole grid
  int causal;
  float scale_log2;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {   // 16 bytes, zeros if not valid
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
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
// two e4m3 codes (the low 16 bits of w) as f16x2: exact, NaN stays NaN
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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

template <int D, bool FP8>
struct PagedLayout {
  static constexpr int ROWB = FP8 ? D : 2 * D;         // bytes of one key
  static constexpr int KT = 4096 / ROWB;               // keys per tile: 16, 32 or 64
  static constexpr int GROUPS = KT / 16;               // 16-key groups: each inside one page
  static constexpr int CPR = ROWB / 16;                // 16-byte chunks per key
  static constexpr int STAGE = 2 * 4096 + (FP8 ? 128 : 0);   // K, V, and the groups' scales
  static constexpr int RING = kPagedWarps * kPagedStages * STAGE;
  static constexpr int bytes(int B) { return RING + (B + 1) * 4; }
  // Byte offset of chunk c of row r, XOR-swizzled so that the 8 rows of an ldmatrix at one chunk
  // fall into different banks.
  static __device__ __forceinline__ int at(int r, int c) {
    if constexpr (ROWB == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return r * ROWB + ((c ^ (r & 7)) << 4);
  }
};

// Where a warp stands in the list of (sequence, head and row tile, key tile)s.
struct PagedPos {
  int b, hr, t;   // sequence, head * row_tiles + row tile, key tile
  int T, L;       // key tiles and keys of sequence b
};

template <int D, bool FP8, bool R16>
__global__ void __launch_bounds__(32 * kPagedWarps, 1) fa_paged_split_kernel(const PagedParams p) {
  using Lt = PagedLayout<D, FP8>;
  constexpr int KT = Lt::KT, G = Lt::GROUPS, NT = KT / 8, RT = R16 ? 16 : 8;
  extern __shared__ __align__(1024) uint8_t smem[];
  int* off = reinterpret_cast<int*>(smem + Lt::RING);   // [B + 1]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- prefix of the sequences' key tiles: every thread sums a run of sequences, then the runs are scanned
  {
    __shared__ int runs[32 * kPagedWarps];
    const int per = (p.B + 32 * kPagedWarps - 1) / (32 * kPagedWarps);
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
      for (int b = tid; b <= p.B; b += 32 * kPagedWarps) p.plan[b] = off[b];
  }

  const int HR = p.Hkv * p.row_tiles;
  const long long W = (long long)off[p.B] * HR;
  // shares: warps of different SMs first, so that few tiles still spread over the whole device
  const int me = warp * int(gridDim.x) + int(blockIdx.x);
  const int sharers = paged_sharers(W, p.n_warps);
  if (me >= sharers) return;
  const long long w0 = W * me / sharers, w1 = W * (me + 1) / sharers;

  PagedPos ld;
  {
    const int want = int(w0 / HR);   // the sequence with off[b] <= want < off[b + 1]
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (off[mid] <= want) lo = mid; else hi = mid;
    }
    ld.b = lo;
    ld.T = off[lo + 1] - off[lo];
    const long long rem = w0 - (long long)off[lo] * HR;
    ld.hr = int(rem / ld.T);
    ld.t = int(rem % ld.T);
    ld.L = paged_key_len(p, lo);
  }
  PagedPos cp = ld;
  auto advance = [&](PagedPos& x) {
    if (++x.t < x.T) return;
    x.t = 0;
    if (++x.hr < HR) return;
    x.hr = 0;
    do ++x.b; while (x.b < p.B && off[x.b + 1] == off[x.b]);
    if (x.b < p.B) {
      x.T = off[x.b + 1] - off[x.b];
      x.L = paged_key_len(p, x.b);
    }
  };

  const uint32_t ring = smem_u32(smem) + warp * kPagedStages * Lt::STAGE;
  const int page_mask = (1 << p.page_shift) - 1;
  int ids[G];   // pages of the groups of the tile that is loaded next
  auto look_up = [&]() {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int key = ld.t * KT + 16 * g;
      ids[g] = key < ld.L ? __ldg(p.page_table + (int64_t)ld.b * p.max_pages + (key >> p.page_shift)) : 0;
    }
  };
  auto load = [&](int stage) {
    const uint32_t dst = ring + stage * Lt::STAGE;
    const int h = ld.hr / p.row_tiles;
    constexpr int RPI = 32 / Lt::CPR;   // keys per warp-wide copy
    const int c = lane % Lt::CPR, r0 = lane / Lt::CPR;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int key = ld.t * KT + 16 * g;
      const bool ok = unsigned(ids[g]) < unsigned(p.n_pages);
      if (!ok) record_status(kStatusRange);
      const int64_t page = ok ? ids[g] : 0;
      const int64_t in = ((int64_t)h << p.page_shift) + (key & page_mask);
      const uint8_t* ks = p.k + page * p.k_page_bytes + (in + r0) * Lt::ROWB + c * 16;
      const uint8_t* vs = p.v + page * p.v_page_bytes + (in + r0) * Lt::ROWB + c * 16;
      const int left = ok ? ld.L - key - r0 : 0;
#pragma unroll
      for (int i = 0; i < 16 / RPI; ++i) {
        const int at = Lt::at(16 * g + i * RPI + r0, c);
        cp_async16(dst + at, ks + i * RPI * Lt::ROWB, i * RPI < left);
        cp_async16(dst + 4096 + at, vs + i * RPI * Lt::ROWB, i * RPI < left);
      }
      if constexpr (FP8) {
        if (lane < 2) cp_async4(dst + 8192 + 8 * g + 4 * lane, (lane == 0 ? p.k_scale : p.v_scale) + page * p.Hkv + h, ok && key < ld.L);
      }
    }
  };

  long long at_load = w0;
  look_up();
#pragma unroll
  for (int s = 0; s < kPagedStages - 1; ++s) {
    if (at_load < w1) {
      load(s);
      advance(ld);
      if (++at_load < w1) look_up();
    }
    cp_async_commit();
  }

  const int g = lane >> 2, t4 = lane & 3;
  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2], sc[2];   // rows g and g + 8; sc: score scale in the log2 domain
  int lim[2], lim_lo;        // keys < lim allowed; lim_lo: the smallest that is not zero
  float vref = 0.f;          // e4m3: the largest value scale so far, O is in units of it
  int stage = 0;
  bool fresh = true;
  long long seg = w0;        // first tile of the running segment
  for (long long w = w0; w < w1; ++w) {
    if (fresh) {
      // ---- queries and limits of this row tile
      fresh = false;
      seg = w;
      const int h = cp.hr / p.row_tiles, rt = cp.hr % p.row_tiles;
      const int n = paged_new_len(p, cp.b);
      const __nv_bfloat16* qb = p.q + ((int64_t)(cp.b * p.Hkv + h) * p.R + rt * RT) * D;
      lim_lo = cp.L;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = rt * RT + g + 8 * i, qi = row % p.Nq;
        const bool real = (R16 || i == 0) && row < p.R;
        lim[i] = real && qi < n ? (p.causal ? max(min(cp.L, cp.L - n + qi + 1), 0) : cp.L) : 0;
        if (lim[i] > 0) lim_lo = min(lim_lo, lim[i]);   // a row without keys is dropped at the end instead
        sc[i] = p.scale_log2;
        m[i] = -INFINITY;
        l[i] = 0.f;
        const uint2* src = reinterpret_cast<const uint2*>(qb + (int64_t)(g + 8 * i) * D);
        const uint32_t* src1 = reinterpret_cast<const uint32_t*>(src);
        if constexpr (FP8) {
          // f16 queries: each row times a power of two that puts its largest element into [2^14, 2^15)
          uint2 w2[D / 16];
          float mx = 0.f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            w2[c] = real ? src[c * 4 + t4] : make_uint2(0u, 0u);
            mx = max3f(mx, fabsf(__uint_as_float(w2[c].x << 16)), fabsf(__uint_as_float(w2[c].x & 0xffff0000u)));
            mx = max3f(mx, fabsf(__uint_as_float(w2[c].y << 16)), fabsf(__uint_as_float(w2[c].y & 0xffff0000u)));
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const int e = min(max(int(__float_as_uint(mx) >> 23) - 127, -100), 127);
          const bool scaled = mx > 0.f && mx < INFINITY;
          const float up = scaled ? __uint_as_float(uint32_t(127 + 14 - e) << 23) : 1.f;    // 2^(14 - e)
          sc[i] *= scaled ? __uint_as_float(uint32_t(127 - 14 + e) << 23) : 1.f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            qf[c][i] = pack_f16x2(__uint_as_float(w2[c].x << 16) * up, __uint_as_float(w2[c].x & 0xffff0000u) * up);
            qf[c][2 + i] = pack_f16x2(__uint_as_float(w2[c].y << 16) * up, __uint_as_float(w2[c].y & 0xffff0000u) * up);
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            qf[c][i] = real ? src1[c * 8 + t4] : 0u;
            qf[c][2 + i] = real ? src1[c * 8 + 4 + t4] : 0u;
          }
        }
      }
      lim_lo = __reduce_min_sync(0xffffffffu, lim_lo);
      vref = 6.0185311e-36f;   // 2^-117
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    }

    // ---- the next tile of the list goes into the stage that the previous iteration emptied
    cp_async_wait<kPagedStages - 2>();
    __syncwarp();
    {
      const int into = stage == 0 ? kPagedStages - 1 : stage - 1;
      if (at_load < w1) {
        load(into);
        advance(ld);
        if (++at_load < w1) look_up();
      }
      cp_async_commit();
    }
    const uint32_t kt = ring + stage * Lt::STAGE, vt = kt + 4096;

    // ---- S = Q K^T
    float s[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
    const int lrow = (lane & 7) + ((lane >> 4) << 3), lchunk = (lane >> 3) & 1;
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      if constexpr (FP8) {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {   // two chunks of 16 features
          uint32_t r[4];
          ldsm4(r, kt + Lt::at(8 * j + lrow, c + lchunk));
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int cc = c + (x & 1);
            mma16816<true>(s[j + (x >> 1)], qf[cc][0], qf[cc][1], qf[cc][2], qf[cc][3], e4m3x2_to_f16x2(r[x]),
                           e4m3x2_to_f16x2(r[x] >> 16));
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t r[4];
          ldsm4(r, kt + Lt::at(8 * j + lrow, 2 * c + lchunk));
          mma16816<false>(s[j], qf[c][0], qf[c][1], qf[c][2], qf[c][3], r[0], r[1]);
          mma16816<false>(s[j + 1], qf[c][0], qf[c][1], qf[c][2], qf[c][3], r[2], r[3]);
        }
      }
    }
    float vsc[G];
    if constexpr (FP8) {
      float ks[G];
#pragma unroll
      for (int x = 0; x < G; ++x)
        asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(ks[x]), "=f"(vsc[x]) : "r"(kt + 8192 + 8 * x));
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < (R16 ? 4 : 2); ++e) s[j][e] *= ks[j >> 1];
    }
    const int k0 = cp.t * KT;
    if (k0 + KT > lim_lo) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < (R16 ? 4 : 2); ++e)
          if (k0 + 8 * j + 2 * t4 + (e & 1) >= lim[e >> 1]) s[j][e] = -INFINITY;
    }

    // ---- online softmax: o is rescaled by alpha (and, e4m3, by the value scale's move), l by alpha
    float alpha[2] = {1.f, 1.f}, neg[2] = {0.f, 0.f}, vmove = 1.f;
    bool moved = false;
#pragma unroll
    for (int i = 0; i < (R16 ? 2 : 1); ++i) {
      float mx = s[0][2 * i];
#pragma unroll
      for (int j = 0; j < NT; ++j) mx = max3f(mx, s[j][2 * i], s[j][2 * i + 1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      mx *= sc[i];
      if (mx > m[i] + kPagedRescale) {
        alpha[i] = ex2_approx(m[i] - mx);
        m[i] = mx;
        moved = true;
      }
      neg[i] = m[i] == -INFINITY ? 0.f : -m[i];
    }
    if constexpr (FP8) {
      float vmax = vref;
#pragma unroll
      for (int x = 0; x < G; ++x) vmax = fmaxf(vmax, vsc[x]);
      if (vmax > vref) {   // the same in every lane
        vmove = vref / vmax;
        vref = vmax;
        moved = true;
      }
      const float unit = kPagedPScale / vref;
#pragma unroll
      for (int x = 0; x < G; ++x) vsc[x] *= unit;
    }
    if (__any_sync(0xffffffffu, moved)) {
      const float a0 = alpha[0] * vmove, a1 = alpha[R16 ? 1 : 0] * vmove;
      l[0] *= alpha[0];
      l[1] *= alpha[1];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        o[c][0] *= a0;
        o[c][1] *= a0;
        o[c][2] *= a1;
        o[c][3] *= a1;
      }
    }
    uint32_t pf[G][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < (R16 ? 2 : 1); ++i) {
        float p0 = ex2_approx(fmaf(s[j][2 * i], sc[i], neg[i])), p1 = ex2_approx(fmaf(s[j][2 * i + 1], sc[i], neg[i]));
        l[i] += p0 + p1;
        if constexpr (FP8) {
          pf[j >> 1][2 * (j & 1) + i] = pack_f16x2(p0 * vsc[j >> 1], p1 * vsc[j >> 1]);
        } else {
          const uint32_t hi = pack_bf16x2(p0, p1);
          pf[j >> 1][2 * (j & 1) + i] = hi;
          // 8 rows: the MMA's other 8 rows take what rounding P to bf16 leaves, so that P has 16 bits
          if constexpr (!R16)
            pf[j >> 1][2 * (j & 1) + 1] =
                pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
        }
      }
      if constexpr (FP8 && !R16) pf[j >> 1][2 * (j & 1) + 1] = 0u;
    }

    // ---- O += P V.  A value that is not finite must not reach a row that does not see its key (0 * inf):
    // where rows see different keys of the tile and such a value is there, it is taken out of the
    // product and its effect is added to the rows that do see it.
    bool careful = false;
    if (lim_lo < min(cp.L, k0 + KT)) {
      uint32_t bad = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        uint32_t q4[4];
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(q4[0]), "=r"(q4[1]), "=r"(q4[2]), "=r"(q4[3])
                     : "r"(vt + 16 * (32 * x + lane)));
#pragma unroll
        for (int e = 0; e < 4; ++e) bad |= not_finite<FP8>(q4[e]);
      }
      careful = __any_sync(0xffffffffu, bad != 0);
    }
    const int vrow = lane & 15, vchunk = lane >> 4;
    if (!careful) {
#pragma unroll
      for (int x = 0; x < G; ++x)
#pragma unroll
        for (int c = 0; c < Lt::CPR; c += 2) {
          uint32_t r[4];
          ldsm4_trans(r, vt + Lt::at(16 * x + vrow, c + vchunk));
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if constexpr (FP8) {
              mma16816<true>(o[2 * (c + y)], pf[x][0], pf[x][1], pf[x][2], pf[x][3],
                             e4m3x2_to_f16x2(__byte_perm(r[2 * y], 0, 0x4420)), e4m3x2_to_f16x2(__byte_perm(r[2 * y + 1], 0, 0x4420)));
              mma16816<true>(o[2 * (c + y) + 1], pf[x][0], pf[x][1], pf[x][2], pf[x][3],
                             e4m3x2_to_f16x2(__byte_perm(r[2 * y], 0, 0x4431)), e4m3x2_to_f16x2(__byte_perm(r[2 * y + 1], 0, 0x4431)));
            } else {
              mma16816<false>(o[c + y], pf[x][0], pf[x][1], pf[x][2], pf[x][3], r[2 * y], r[2 * y + 1]);
            }
          }
        }
    } else {
      // a = 1 where the row sees the key; 16-bit one in the operands' type
      constexpr uint32_t kOne = FP8 ? 0x3c00u : 0x3f80u;
#pragma unroll
      for (int x = 0; x < G; ++x) {
        uint32_t see[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = k0 + 16 * x + 8 * (e >> 1) + 2 * t4;
          see[e] = (R16 || (e & 1) == 0) ? (key < lim[e & 1] ? kOne : 0u) | (key + 1 < lim[e & 1] ? kOne << 16 : 0u) : 0u;
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t r[4];
          ldsm4_trans(r, vt + Lt::at(16 * x + vrow, FP8 ? (c >> 1) : c));   // its two upper matrices repeat the lower: vrow < 16
          uint32_t b[2], up[2], dn[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t w = FP8 ? e4m3x2_to_f16x2(__byte_perm(r[y], 0, (c & 1) ? 0x4431 : 0x4420)) : r[y];
            constexpr uint32_t kExp = FP8 ? 0x7c00u : 0x7f80u;
            uint32_t u = 0, d = 0, keep = 0;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t a = (w >> (16 * z)) & 0xffffu;
              const bool inf_or_nan = (a & kExp) == kExp, nan = inf_or_nan && (a & ~kExp & 0x7fffu) != 0;
              if (!inf_or_nan) keep |= 0xffffu << (16 * z);
              if (nan || (inf_or_nan && !(a & 0x8000u))) u |= kOne << (16 * z);
              if (nan || (inf_or_nan && (a & 0x8000u))) d |= kOne << (16 * z);
            }
            b[y] = w & keep;
            up[y] = u;
            dn[y] = d;
          }
          float cu[4] = {0.f, 0.f, 0.f, 0.f}, cd[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816<FP8>(o[c], pf[x][0], pf[x][1], pf[x][2], pf[x][3], b[0], b[1]);
          mma16816<FP8>(cu, see[0], see[1], see[2], see[3], up[0], up[1]);
          mma16816<FP8>(cd, see[0], see[1], see[2], see[3], dn[0], dn[1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (cu[e] > 0.f) o[c][e] += INFINITY;
            if (cd[e] > 0.f) o[c][e] -= INFINITY;
          }
        }
      }
    }
    __syncwarp();

    // ---- end of the segment: this row tile's last key tile, or this warp's last
    if (cp.t + 1 == cp.T || w + 1 == w1) {
      const bool whole = cp.t + 1 == cp.T && w - seg + 1 == cp.T;
      const int h = cp.hr / p.row_tiles, rt = cp.hr % p.row_tiles;
#pragma unroll
      for (int i = 0; i < (R16 ? 2 : 1); ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const int row = g + 8 * i;
        if (rt * RT + row >= p.R) continue;
        const bool dead = lim[i] == 0;
        if (dead) l[i] = 0.f;
        const float f = (FP8 ? vref * (1.f / kPagedPScale) : 1.f) * (whole ? (l[i] != 0.f ? 1.f / l[i] : 0.f) : 1.f);
        const int64_t out = (int64_t)(cp.b * p.Hkv + h) * p.R + rt * RT + row;
        const int64_t slot = (2 * (int64_t)me + (seg == w0 ? 0 : 1)) * RT + row;
        // fragment columns -> features: bf16 pairs 8c + 2 t4; e4m3 quads 16c + 4 t4 (even and odd tiles interleaved)
#pragma unroll
        for (int c = 0; c < D / 8; c += 2) {
          float x[4];   // o[c] pair, o[c + 1] pair
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float val = o[c + (e >> 1)][2 * i + (e & 1)];
            if constexpr (!R16) val += o[c + (e >> 1)][2 + (e & 1)];
            x[e] = dead ? 0.f : val * f;
          }
          if constexpr (FP8) {
            const int at = 8 * c + 4 * t4;
            if (whole)
              *reinterpret_cast<uint2*>(p.o + out * D + at) = make_uint2(pack_bf16x2(x[0], x[2]), pack_bf16x2(x[1], x[3]));
            else
              *reinterpret_cast<float4*>(p.part_o + slot * D + at) = make_float4(x[0], x[2], x[1], x[3]);
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int at = 8 * (c + y) + 2 * t4;
              if (whole)
                *reinterpret_cast<uint32_t*>(p.o + out * D + at) = pack_bf16x2(x[2 * y], x[2 * y + 1]);
              else
                *reinterpret_cast<float2*>(p.part_o + slot * D + at) = make_float2(x[2 * y], x[2 * y + 1]);
            }
          }
        }
        if (t4 == 0) {
          if (whole)
            p.lse[out] = l[i] != 0.f ? (m[i] + lg2_approx(l[i])) * kPagedLn2 : -INFINITY;
          else
            p.part_ml[slot] = make_float2(m[i], l[i]);
        }
      }
      fresh = true;
    }
    advance(cp);
    stage = stage == kPagedStages - 1 ? 0 : stage + 1;
  }
}

// Merges the partials of one query row that several warps made; one warp (WPR = 1) or one CTA of
// WPR warps per row.  Rows of a row tile that one warp had whole are done already.  Also writes the rows of
// sequences without keys or without new tokens: O = 0, lse = -inf.
template <int D, int RT, int WPR>
__global__ void __launch_bounds__(256) fa_paged_combine_kernel(const PagedParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = WPR == 1 ? (long long)blockIdx.x * 8 + warp : (long long)blockIdx.x;   // of [B, Hkv, R]
  if (row >= (long long)p.B * p.Hkv * p.R) return;
  const int r = int(row % p.R), h = int(row / p.R % p.Hkv), b = int(row / p.R / p.Hkv);
  constexpr int PER = D / 32;
  const int T = p.plan[b + 1] - p.plan[b], HR = p.Hkv * p.row_tiles;
  const long long W = (long long)p.plan[p.B] * HR;
  float acc[PER], ms = -INFINITY, ls = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  if (T > 0) {
    const long long first = (long long)p.plan[b] * HR + (long long)(h * p.row_tiles + r / RT) * T;
    const int sharers = paged_sharers(W, p.n_warps);
    const int w_first = int(((first + 1) * sharers - 1) / W), w_last = int(((first + T) * sharers - 1) / W);
    if (w_first == w_last) return;
    const int sub = WPR == 1 ? 0 : warp;
    for (int w = w_first + sub; w <= w_last; w += WPR) {
      const long long starts = W * w / sharers;
      const int64_t slot = (2 * (int64_t)w + (starts >= first ? 0 : 1)) * RT + r % RT;
      const float2 ml = p.part_ml[slot];
      float x[PER];
#pragma unroll
      for (int e = 0; e < PER; ++e) x[e] = p.part_o[slot * D + lane * PER + e];
      if (ml.y == 0.f) continue;   // no key seen there (its m may be -inf)
      const float mn = fmaxf(ms, ml.x);
      const float a = ms == -INFINITY ? 0.f : ex2_approx(ms - mn), c = ex2_approx(ml.x - mn);
      ls = ls * a + ml.y * c;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = acc[e] * a + x[e] * c;
      ms = mn;
    }
  }
  if constexpr (WPR > 1) {
    __shared__ float sm[WPR], sl[WPR], so[WPR][D];
    if (lane == 0) {
      sm[warp] = ms;
      sl[warp] = ls;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) so[warp][lane * PER + e] = acc[e];
    __syncthreads();
    if (warp != 0) return;
    for (int x = 1; x < WPR; ++x) {
      if (sl[x] == 0.f) continue;
      const float mn = fmaxf(ms, sm[x]);
      const float a = ms == -INFINITY ? 0.f : ex2_approx(ms - mn), c = ex2_approx(sm[x] - mn);
      ls = ls * a + sl[x] * c;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = acc[e] * a + so[x][lane * PER + e] * c;
      ms = mn;
    }
  }
  const float inv = ls != 0.f ? 1.f / ls : 0.f;
  uint32_t out[PER / 2];
#pragma unroll
  for (int e = 0; e < PER / 2; ++e) out[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + lane * PER);
#pragma unroll
  for (int e = 0; e < PER / 2; ++e) dst[e] = out[e];
  if (lane == 0) p.lse[row] = ls != 0.f ? (ms + lg2_approx(ls)) * kPagedLn2 : -INFINITY;
}

}  // namespace fa
