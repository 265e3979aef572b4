// Appending keys and values to a paged cache for sm_100a, with the position rotation on the way.
//
// The n = new_lens[b] new tokens of sequence b take the positions key_lens[b] - n .. key_lens[b] - 1;
// position j lies in page page_table[b][j / page], row j % page, of the pools [n_pages, Hkv, page, d].
// Keys (and the queries, which go to an array of their own) are rotated on the way: a pair (x, y) at
// position j becomes (x cos - y sin, y cos + x sin) with the cosines and sines of row j of two fp32
// tables, pairs (i, i + rot / 2) or (2 i, 2 i + 1).  The products are rounded before they are added
// (no fma), so that the result is the same wherever it is computed in fp32 this way.
//
// e4m3 pools hold one fp32 scale per page and head.  A page's scale becomes s' = max(s, 2^e), where
// 2^e is the smallest power of two with |x| <= 448 * 2^e over the page's new (finite) values and s the
// scale of the tokens it held before (none: 2^e alone).  Where s' > s those are re-rounded by s / s',
// which only moves their exponents when s is a power of two too.  Infinities saturate, NaN stays.
//
// Bound: HBM, every value read and written once (a launch's latency for single tokens).  A thread
// takes 16 features of a token (two 16-byte loads: the two halves of its pairs) and walks over heads
// of that token, so that one read of the tables serves up to 8 heads.
// Measured (B200, 32/8 heads, d = 128): 8 prompts of up to 2048 tokens 62 us in bf16 (6.0 TB/s, 92 % of the copy rate) and
// 67 us in e4m3 (5.1 TB/s: its pages wait for the scale, one load after another); 64 single tokens 2.4 and 3.0 us.
#pragma once
#include <cuda_bf16.h>
#include "paged_sm100.cuh"

namespace fa {

struct AppendParams {
  const __nv_bfloat16* x[3];   // q, k, v: [B, H, Nq, d] with the strides below; q may be null
  int64_t sb[3], sh[3], sn[3]; // strides in elements: batch, head, token
  __nv_bfloat16* q_out;        // [B, Hq, Nq, d] contiguous
  uint8_t* pool[2];            // k, v
  int64_t page_bytes[2];
  float* scale[2];             // [n_pages, Hkv] (e4m3)
  const int32_t* page_table;   // [B, max_pages]
  const int32_t* key_lens;     // [B], after the append
  const int32_t* new_lens;     // [B] or null
  const float* cos;            // [max_pos, rot / 2]; null: no rotation
  const float* sin;
  int B, Hq, Hkv, Nq, d, rot, interleaved, max_pos;   // Hq = 0 without q
  int n_pages, page_shift, max_pages;
  int heads_per_thread;
  int row_blocks_x;            // token blocks of the row role
  int row_blocks;              // all of its blocks (e4m3: the pages' units follow)
  int touched;                 // e4m3: most pages that a sequence's new tokens can touch
};

// Position and state of new token i of sequence b; pos < 0: no such token, or one outside the cache.
__device__ __forceinline__ int append_position(const AppendParams& p, int b, int i) {
  const int L = p.key_lens[b], n = p.new_lens == nullptr ? p.Nq : p.new_lens[b];
  const long long cap = (long long)p.max_pages << p.page_shift;
  if (n < 0 || n > p.Nq || L < n || L > cap || (p.cos != nullptr && L > p.max_pos && n > 0)) record_status(kStatusRange);
  if (i >= n || i >= p.Nq) return -1;
  const long long pos = (long long)L - n + i;
  if (pos < 0 || pos >= cap || (p.cos != nullptr && pos >= p.max_pos)) return -1;
  return int(pos);
}

struct Pair16 {   // 16 features of one token: two chunks of 8
  uint4 a, b;
};
// Chunks (of 8 features) that lane `p` of a row takes, and whether they are rotated together.
__device__ __forceinline__ bool append_chunks(const AppendParams& p, int lane, int& ca, int& cb) {
  const int turned = p.cos == nullptr ? 0 : p.rot / 16;
  if (lane >= turned || p.interleaved) {
    ca = 2 * lane;   // (beyond the rotated pairs both pairings leave whole chunk pairs: rot is a multiple of 16)
    cb = ca + 1;
  } else {
    ca = lane;
    cb = lane + turned;
  }
  return lane < turned;
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(u[e] << 16);
    x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void load8(const float* src, float (&x)[8]) {
  const float4 a = global_load(reinterpret_cast<const float4*>(src)), b = global_load(reinterpret_cast<const float4*>(src) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = u;
}
__device__ __forceinline__ void turn16(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8], bool interleaved) {
  if (!interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) turn(a[e], b[e], c[e], s[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      turn(a[2 * e], a[2 * e + 1], c[e], s[e]);
      turn(b[2 * e], b[2 * e + 1], c[4 + e], s[4 + e]);
    }
  }
}

// The row role: rotated queries, and for bf16 pools keys and values.  POOL: keys and values too.
template <bool POOL>
__device__ __forceinline__ void append_rows(const AppendParams& p, int block) {
  const int lpr = p.d / 16;   // threads per row
  const int lane = threadIdx.x % lpr;
  const long long tok = (long long)(block % p.row_blocks_x) * (blockDim.x / lpr) + threadIdx.x / lpr;
  if (tok >= (long long)p.B * p.Nq) return;
  const int b = int(tok / p.Nq), i = int(tok % p.Nq);
  const int pos = append_position(p, b, i);
  int ca, cb;
  const bool turned = append_chunks(p, lane, ca, cb);
  float c[8], s[8];
  if (turned && pos >= 0) {
    load8(p.cos + (int64_t)pos * (p.rot / 2) + 8 * lane, c);
    load8(p.sin + (int64_t)pos * (p.rot / 2) + 8 * lane, s);
  }
  int64_t page = -1;
  if (POOL && pos >= 0) {
    page = global_load(p.page_table + (int64_t)b * p.max_pages + (pos >> p.page_shift));
    if (page < 0 || page >= p.n_pages) {
      record_status(kStatusRange);
      page = -1;
    }
  }
  const int heads = p.Hq + (POOL ? 2 * p.Hkv : 0);
  const int h0 = (block / p.row_blocks_x) * p.heads_per_thread, h1 = min(heads, h0 + p.heads_per_thread);
  constexpr int U = 4;   // heads in flight
  for (int hb = h0; hb < h1; hb += U) {
    Pair16 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hh = hb + u;
      if (hh >= h1 || pos < 0) continue;
      const int which = hh < p.Hq ? 0 : hh < p.Hq + p.Hkv ? 1 : 2;
      const int h = which == 0 ? hh : which == 1 ? hh - p.Hq : hh - p.Hq - p.Hkv;
      const uint4* src = reinterpret_cast<const uint4*>(p.x[which] + b * p.sb[which] + h * p.sh[which] + i * p.sn[which]);
      w[u].a = global_load(src + ca);
      w[u].b = global_load(src + cb);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hh = hb + u;
      if (hh >= h1) continue;
      const int which = hh < p.Hq ? 0 : hh < p.Hq + p.Hkv ? 1 : 2;
      if (pos < 0) w[u].a = w[u].b = make_uint4(0u, 0u, 0u, 0u);   // no token: the query row is zero
      if (which < 2 && turned && pos >= 0) {
        float x[8], y[8];
        unpack8(w[u].a, x);
        unpack8(w[u].b, y);
        turn16(x, y, c, s, p.interleaved != 0);
        w[u].a = pack8(x);
        w[u].b = pack8(y);
      }
      uint4* dst;
      if (which == 0) {
        dst = reinterpret_cast<uint4*>(p.q_out + (((int64_t)b * p.Hq + hh) * p.Nq + i) * p.d);
      } else {
        if (page < 0) continue;
        const int h = which == 1 ? hh - p.Hq : hh - p.Hq - p.Hkv;
        const int64_t row = ((int64_t)h << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        dst = reinterpret_cast<uint4*>(p.pool[which - 1] + page * p.page_bytes[which - 1] + row * (p.d * 2));
      }
      dst[ca] = w[u].a;
      dst[cb] = w[u].b;
    }
  }
}

__global__ void __launch_bounds__(128) fa_kv_append_kernel(const __grid_constant__ AppendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // (a programmatic dependent launch)
  append_rows<true>(p, int(blockIdx.x));
}

// ----------------------------------------------------------------------------- e4m3 pages
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8]) {   // nearest, saturating; NaN stays NaN
  uint32_t r[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}\n"
        : "=r"(r[e]) : "f"(x[4 * e]), "f"(x[4 * e + 1]), "f"(x[4 * e + 2]), "f"(x[4 * e + 3]));
  return make_uint2(r[0], r[1]);
}
// The smallest power of two s with amax <= 448 s, at least 2^-117.  448 = 1.75 * 2^8.
__device__ __forceinline__ float e4m3_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = int(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(uint32_t(max(e, -117) + 127) << 23);
}

// One CTA of THREADS per (sequence, touched page, head, key or value): its new rows stay in registers
// (at most 4 per thread) between the search for the scale and the rounding, as the bf16 they came in: rotating
// them twice costs less than the registers of the results.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 768 / THREADS : 1) fa_kv_append_e4m3_kernel(const __grid_constant__ AppendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (int(blockIdx.x) < p.row_blocks) {
    append_rows<false>(p, int(blockIdx.x));
    return;
  }
  long long unit = (long long)blockIdx.x - p.row_blocks;
  const int kv = int(unit & 1);
  unit >>= 1;
  const int h = int(unit % p.Hkv);
  unit /= p.Hkv;
  const int tp = int(unit % p.touched), b = int(unit / p.touched);
  const int L = p.key_lens[b], n = p.new_lens == nullptr ? p.Nq : p.new_lens[b];
  const int page_size = 1 << p.page_shift;
  const long long cap = (long long)p.max_pages << p.page_shift;
  if (n < 0 || n > p.Nq || L < n || L > cap || (p.cos != nullptr && L > p.max_pos && n > 0)) {
    record_status(kStatusRange);
    return;
  }
  if (n == 0) return;
  const int start = L - n, pg = (start >> p.page_shift) + tp;
  const long long base = (long long)pg << p.page_shift;
  if (base >= L) return;
  const int lo = int(base > start ? base : start), hi = int(base + page_size < L ? base + page_size : L);
  const int64_t page = global_load(p.page_table + (int64_t)b * p.max_pages + pg);   // (in flight with the rows)
  const int old = lo - int(base), m = hi - lo;

  const int lpr = p.d / 16, lane = int(threadIdx.x) % lpr, r0 = int(threadIdx.x) / lpr, rpp = THREADS / lpr;
  int ca, cb;
  const bool turned = append_chunks(p, lane, ca, cb) && kv == 0;
  const __nv_bfloat16* src = p.x[1 + kv] + b * p.sb[1 + kv] + h * p.sh[1 + kv] + (int64_t)(lo - start) * p.sn[1 + kv];
  uint4 wa[4], wb[4];
  float amax = 0.f;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = r0 + u * rpp;
    if (r >= m) continue;
    const uint4* row = reinterpret_cast<const uint4*>(src + r * p.sn[1 + kv]);
    wa[u] = global_load(row + ca);
    wb[u] = global_load(row + cb);
  }
  if (page < 0 || page >= p.n_pages) {
    record_status(kStatusRange);
    return;
  }
  float* scale = p.scale[kv] + page * p.Hkv + h;
  uint8_t* dst = p.pool[kv] + page * p.page_bytes[kv] + ((int64_t)h << p.page_shift) * p.d;
  const float before = old > 0 ? *scale : 0.f;
  // row u of this thread, rotated
  auto row_of = [&](int u, float (&x)[8], float (&y)[8]) {
    unpack8(wa[u], x);
    unpack8(wb[u], y);
    if (turned) {
      float c[8], s[8];
      load8(p.cos + (int64_t)(lo + r0 + u * rpp) * (p.rot / 2) + 8 * lane, c);
      load8(p.sin + (int64_t)(lo + r0 + u * rpp) * (p.rot / 2) + 8 * lane, s);
      turn16(x, y, c, s, p.interleaved != 0);
    }
  };
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (r0 + u * rpp >= m) continue;
    float x[8], y[8];
    row_of(u, x, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float ax = fabsf(x[e]), ay = fabsf(y[e]);
      if (ax < INFINITY) amax = fmaxf(amax, ax);
      if (ay < INFINITY) amax = fmaxf(amax, ay);
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
  if constexpr (THREADS > 32) {
    __shared__ float part[THREADS / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, part[w]);
  }
  const float after = fmaxf(e4m3_scale(amax), before);

  if (old > 0 && after > before) {   // re-round what the page held
    const float ratio = before / after;
    for (int c = int(threadIdx.x); c < old * p.d / 8; c += THREADS) {
      uint2 w = *reinterpret_cast<const uint2*>(dst + 8 * c);
      float z[8];
      const uint32_t u[4] = {w.x, w.x >> 16, w.y, w.y >> 16};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t two = e4m3x2_to_f16x2(u[e]);
        z[2 * e] = __half2float(__ushort_as_half((unsigned short)(two & 0xffffu))) * ratio;
        z[2 * e + 1] = __half2float(__ushort_as_half((unsigned short)(two >> 16))) * ratio;
      }
      *reinterpret_cast<uint2*>(dst + 8 * c) = pack8_e4m3(z);
    }
  }
  // x / after.  after is a power of two, and the product with its inverse exact, unless the caller's own scale was not:
  // then divide.  (A select between the two pays for both: 64 divisions a thread.)
  const bool pow2 = (__float_as_uint(after) & 0x7fffffu) == 0;
  const float inv = 1.f / after;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = r0 + u * rpp;
    if (r >= m) continue;
    float x[8], y[8];
    row_of(u, x, y);
    if (!pow2) {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int z = 0; z < 8; ++z)
          if (z == e) {
            x[z] = __fdiv_rn(x[z], after);
            y[z] = __fdiv_rn(y[z], after);
          }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= inv;
        y[e] *= inv;
      }
    }
    uint8_t* row = dst + (int64_t)(old + r) * p.d;
    *reinterpret_cast<uint2*>(row + 8 * ca) = pack8_e4m3(x);
    *reinterpret_cast<uint2*>(row + 8 * cb) = pack8_e4m3(y);
  }
  if (threadIdx.x == 0 && after != before) *scale = after;
}

}  // namespace fa
