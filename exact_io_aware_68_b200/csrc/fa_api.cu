// The C ABI declared in include/fa.h: argument validation, TMA descriptor encoding and the
// kernel launches.  The kernels live in the headers included below; this is the library's
// single translation unit.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <mutex>

#include "../../include/fa.h"
#include "bwd_dq_sm100.cuh"
#include "bwd_sm100.cuh"
#include "decode_sm100.cuh"
#include "fwd256_sm100.cuh"
#include "fwd_sm100.cuh"
#include "kv_append.cuh"
#include "paged_sm100.cuh"
#include "paged_wide_sm100.cuh"
#include "simt_f32.cuh"

namespace {

thread_local char g_err[512] = "";

fa_status fail(fa_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

uint64_t default_wait_ns() {
  const char* e = std::getenv("FA_WAIT_LIMIT_MS");
  if (e != nullptr) {
    const long long ms = std::atoll(e);
    if (ms > 0) return uint64_t(ms) * 1000000ull;
  }
  return 2000000000ull;
}
std::atomic<uint64_t> g_wait_ns{default_wait_ns()};
std::atomic<int> g_debug_flags{0};

// cuTensorMapEncodeTiled from the driver, fetched through the runtime (no -lcuda needed).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 3-D view {d, N, B*H} of a bf16 [B,H,N,d] tensor, loaded as 64 x box_rows x 1 boxes with the
// 128-byte swizzle; rows past N (the ragged last tile) read as zeros.
fa_status make_tile_map(CUtensorMap* map, const void* ptr, int BH, int N, int d, const char* name,
                        unsigned box_rows = 128) {
  auto fn = encode_fn();
  if (fn == nullptr) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(N), cuuint64_t(BH)};
  const cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(N) * cuuint64_t(d) * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with CUresult %d", name, int(r));
  return FA_OK;
}

// 3-D view {d, N, B*H} of the fp32 dQ accumulator for the backward's TMA bulk reductions:
// boxes of (features per dQ warp) x (queries per round), no swizzle; rows past N are not written.
fa_status make_dq_map(CUtensorMap* map, const void* ptr, int BH, int N, int d, unsigned box_x, unsigned box_y) {
  auto fn = encode_fn();
  if (fn == nullptr) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(N), cuuint64_t(BH)};
  const cuuint64_t strides[2] = {cuuint64_t(d) * 4, cuuint64_t(N) * cuuint64_t(d) * 4};
  const cuuint32_t box[3] = {box_x, box_y, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled(dQ accumulator) failed with CUresult %d", int(r));
  return FA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Which head dimensions an entry point takes.
enum class Dims { kBf16, kBf16Fwd, kF32 };

fa_status check_common(int B, int H, int N, int d, float scale, float dropout_p, Dims dims) {
  if (B < 1 || H < 1 || N < 1) return fail(FA_ERR_INVALID_ARG, "B, H and N must be >= 1 (got %d, %d, %d)", B, H, N);
  if (int64_t(B) * H > 65535) return fail(FA_ERR_UNSUPPORTED, "B*H = %lld exceeds 65535", (long long)B * H);
  if (int64_t(N) > (int64_t(1) << 30)) return fail(FA_ERR_UNSUPPORTED, "N = %d is too large", N);
  if (dims == Dims::kBf16 && d != 64 && d != 128)
    return fail(FA_ERR_UNSUPPORTED, "head dimension d = %d: this bf16 entry point supports d in {64, 128}", d);
  if (dims == Dims::kBf16Fwd && d != 64 && d != 128 && d != 256)
    return fail(FA_ERR_UNSUPPORTED, "head dimension d = %d: the bf16 forward supports d in {64, 128, 256}", d);
  if (dims == Dims::kF32 && (d < 1 || d > 128))
    return fail(FA_ERR_UNSUPPORTED, "head dimension d = %d: fp32 supports 1 <= d <= 128", d);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!(dropout_p >= 0.f) || !(dropout_p < 1.f)) return fail(FA_ERR_INVALID_ARG, "dropout_p must be in [0, 1)");
  return FA_OK;
}

#define FA_CHECK_PTR(p)                                                                      \
  do {                                                                                       \
    if ((p) == nullptr) return fail(FA_ERR_INVALID_ARG, "%s is NULL", #p);                   \
    if (!aligned16(p)) return fail(FA_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p);     \
  } while (0)

// The same for arrays that are only read 4 bytes at a time.
#define FA_CHECK_WORDS(p)                                                                                      \
  do {                                                                                                         \
    if ((p) == nullptr) return fail(FA_ERR_INVALID_ARG, "%s is NULL", #p);                                     \
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return fail(FA_ERR_INVALID_ARG, "%s is not 4-byte aligned", #p); \
  } while (0)

fa_status launch_status(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return FA_OK;
}

// The 15-bit dropout threshold: a column is kept when its 15-bit draw is >= this value.
uint32_t drop_threshold(float p) {
  const double t = std::floor(double(p) * 32768.0);
  return uint32_t(t > 32767.0 ? 32767.0 : t);
}

struct Workspace {
  float* dq_acc;
  float* dvec;
  unsigned int* work_ctr;
};
size_t ws_dq_bytes(int B, int H, int N, int d) {
  return (size_t(B) * H * N * d * 4 + 255) & ~size_t(255);
}
size_t ws_d_bytes(int B, int H, int N) { return (size_t(B) * H * N * 4 + 255) & ~size_t(255); }
// fp32 dQ accumulator, D, and 256 bytes for the main kernel's item counter
size_t ws_total_bytes(int B, int H, int N, int d) { return ws_dq_bytes(B, H, N, d) + ws_d_bytes(B, H, N) + 256; }
fa_status check_workspace(void* ws, size_t bytes, int B, int H, int N, int d, Workspace* out) {
  if (ws == nullptr) return fail(FA_ERR_INVALID_ARG, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(FA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  const size_t need = ws_total_bytes(B, H, N, d);
  if (bytes < need) return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", bytes, need);
  out->dq_acc = static_cast<float*>(ws);
  out->dvec = reinterpret_cast<float*>(static_cast<char*>(ws) + ws_dq_bytes(B, H, N, d));
  out->work_ctr =
      reinterpret_cast<unsigned int*>(static_cast<char*>(ws) + ws_dq_bytes(B, H, N, d) + ws_d_bytes(B, H, N));
  return FA_OK;
}

// Number of SMs of the current device (queried once per device).
fa_status sm_count(int* out) {
  static std::atomic<int> cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev >= 0 && dev < 64 && cache[dev].load() > 0) {
    *out = cache[dev].load();
    return FA_OK;
  }
  int n = 0;
  e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess || n <= 0) return fail(FA_ERR_CUDA, "cudaDeviceGetAttribute(SM count): %s", cudaGetErrorString(e));
  if (dev >= 0 && dev < 64) cache[dev].store(n);
  *out = n;
  return FA_OK;
}

// L2 size of the current device in bytes (queried once per device).
fa_status l2_bytes(size_t* out) {
  static std::atomic<long long> cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev >= 0 && dev < 64 && cache[dev].load() > 0) {
    *out = size_t(cache[dev].load());
    return FA_OK;
  }
  int n = 0;
  e = cudaDeviceGetAttribute(&n, cudaDevAttrL2CacheSize, dev);
  if (e != cudaSuccess || n <= 0) return fail(FA_ERR_CUDA, "cudaDeviceGetAttribute(L2 size): %s", cudaGetErrorString(e));
  if (dev >= 0 && dev < 64) cache[dev].store(n);
  *out = size_t(n);
  return FA_OK;
}

template <typename K>
fa_status set_smem(K kernel, int bytes) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  return FA_OK;
}

// The same, asked of the runtime once per device and kernel (`done`: a bit per device).
template <typename K>
fa_status set_smem_once(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 && (done.load() >> dev & 1)) return FA_OK;
  const fa_status st = set_smem(kernel, bytes);
  if (st == FA_OK && dev >= 0 && dev < 64) done.fetch_or(uint64_t(1) << dev);
  return st;
}

// The warp-specialised kernels re-split their registers per warpgroup with setmaxnreg; the split
// adds up to `regs` registers per thread at launch.  A build whose kernel was given fewer
// registers would leave a setmaxnreg.inc waiting forever, so it is refused before the launch.
template <typename K>
fa_status check_launch_regs(K kernel, int regs, const char* name) {
  cudaFuncAttributes a{};
  const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaFuncGetAttributes(%s): %s", name, cudaGetErrorString(e));
  if (a.numRegs < regs)
    return fail(FA_ERR_INTERNAL, "%s was built with %d registers per thread; its register split needs %d", name,
                a.numRegs, regs);
  return FA_OK;
}

template <int D, bool DROPOUT>
fa_status launch_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const fa::FwdParams& p,
                     cudaStream_t s) {
  using L = fa::FwdLayout<D>;
  fa_status st = set_smem(fa::fa_fwd_sm100_kernel<D, DROPOUT>, L::BYTES);
  if (st != FA_OK) return st;
  if ((st = check_launch_regs(fa::fa_fwd_sm100_kernel<D, DROPOUT>, fa::kFwdLaunchRegs, "fa_fwd kernel")) != FA_OK)
    return st;
  // persistent: one CTA per SM (or fewer when there are fewer work items)
  const long long items = (long long)p.n_pairs * p.B * p.H;
  int sms = 0;
  if ((st = sm_count(&sms)) != FA_OK) return st;
  const dim3 grid(unsigned(items < sms ? items : sms));
  fa::fa_fwd_sm100_kernel<D, DROPOUT><<<grid, fa::kFwdThreads, L::BYTES, s>>>(mq, mk, mv, p);
  return launch_status("fa_fwd kernel launch");
}

template <int D, bool DROPOUT, bool DQ>
fa_status launch_bwd_main(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo,
                          fa::BwdParams p, cudaStream_t s) {
  using L = fa::BwdLayout<D, DROPOUT>;
  CUtensorMap mdq;
  fa_status st0 = make_dq_map(&mdq, p.dq_acc, p.B * p.H, p.N, D, L::FPW, L::QPR);
  if (st0 != FA_OK) return st0;
  fa_status st = set_smem(fa::fa_bwd_sm100_kernel<D, DROPOUT, DQ>, L::BYTES);
  if (st != FA_OK) return st;
  if ((st = check_launch_regs(fa::fa_bwd_sm100_kernel<D, DROPOUT, DQ>, fa::kBwdLaunchRegs, "fa_bwd main kernel")) !=
      FA_OK)
    return st;
  int sms = 0;
  if ((st = sm_count(&sms)) != FA_OK) return st;
  // Items (head, key tile) are taken in a linear launch order. Head-major order keeps the CTAs
  // in flight on a few heads, so their Q and dO stay in L2, but each head's heaviest causal key
  // tile starts only when the head does. That tail is about 2 * SMs / (B*H*n_tiles) of the run.
  // While there are at most 20 items per SM, the order is instead: groups of heads one after
  // another, key-tile-major inside each group. Every head's first key tile (the most query
  // tiles when causal) then starts with its group, and the one-tile items form each group's tail.
  // A group holds at most 16 heads, and its Q, dO and fp32 dQ accumulator (8*N*d bytes a head)
  // fit in 32 MB of L2. Measured on the headline causal 2x16x4096x128: head-major 352 us,
  // key-tile-major over all 32 heads 332-340 us (2.6x the algorithmic DRAM bytes), groups of 8
  // heads 330 us. 64k-token sequences keep head-major (the other order was 9 % slower). The group
  // size comes from the device's L2 size (fa_bwd_head_group).
  p.kt_major = int64_t(p.B) * p.H * p.n_tiles <= 20 * int64_t(sms) ? 1 : 0;
  size_t l2 = 0;
  if ((st = l2_bytes(&l2)) != FA_OK) return st;
  p.head_group = fa_bwd_head_group(p.N, D, l2);
  // persistent: one CTA per SM (or fewer when there are fewer items), each walking items
  // c, c + G, c + 2G, ... of the launch order
  const long long items = (long long)p.B * p.H * p.n_tiles;
  const dim3 grid(unsigned(items < sms ? items : sms));
  fa::fa_bwd_sm100_kernel<D, DROPOUT, DQ><<<grid, fa::kBwdThreads, L::BYTES, s>>>(mq, mk, mv, mdo, mdq, p);
  return launch_status("fa_bwd main kernel launch");
}

template <int D, bool DROPOUT>
fa_status launch_dq_pass(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo,
                         const fa::DqParams& p, dim3 grid, cudaStream_t s) {
  using L = fa::DqLayout<D>;
  const fa_status st = set_smem(fa::fa_bwd_dq_pass_kernel<D, DROPOUT>, L::BYTES);
  if (st != FA_OK) return st;
  fa::fa_bwd_dq_pass_kernel<D, DROPOUT><<<grid, 256, L::BYTES, s>>>(mq, mk, mv, mdo, p);
  return launch_status("fa_bwd_split dQ kernel launch");
}

fa::BwdParams bwd_params(int B, int H, int N, float scale, int causal, const int32_t* key_lens, float dropout_p,
                         uint64_t seed, const Workspace& w) {
  fa::BwdParams p{};
  p.lse = nullptr;
  p.dvec = w.dvec;
  p.dq_acc = w.dq_acc;
  p.work_ctr = w.work_ctr;
  p.key_lens = key_lens;
  p.B = B;
  p.H = H;
  p.N = N;
  p.n_tiles = (N + 127) / 128;
  p.causal = causal ? 1 : 0;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.dropout = dropout_p > 0.f ? 1 : 0;
  p.drop_thr = drop_threshold(dropout_p);
  p.drop_scale = dropout_p > 0.f ? 1.f / (1.f - dropout_p) : 1.f;
  p.seed = seed;
  p.wait_ns = g_wait_ns.load();
  p.debug_flags = g_debug_flags.load();
  return p;
}

// Key-range split of the decode kernel.  Its shared memory holds one CTA per SM, so a grid of
// BH * n CTAs runs in ceil(BH * n / sms) waves, each as long as one split's keys.  n minimises
// waves * (chunk + 256): the 256 stands for a split's fixed cost (Q load, pipeline fill, partial
// write) in keys.  Chunks are whole 128-key blocks of at least 512 keys; n <= 4 * sms.  With no SM
// count (sms <= 0) the split is the finest one, n = ceil(Nkv / 512), which bounds the workspace of
// every device.  Host arithmetic only.
struct DecodeSplit {
  int chunk, n_split;
};
DecodeSplit decode_split(int BH, int Nkv, int sms) {
  auto chunk_for = [&](long long n) {
    long long c = (Nkv + n - 1) / n;
    c = (c + 127) / 128 * 128;
    return c < 512 ? 512LL : c;
  };
  const long long finest = (Nkv + 511) / 512;
  if (sms <= 0) {
    const long long c = chunk_for(finest);
    return DecodeSplit{int(c), int((Nkv + c - 1) / c)};
  }
  const long long top = std::min<long long>(finest, 4LL * sms);
  DecodeSplit best{0, 0};
  long long best_cost = -1;
  for (long long n = 1; n <= top; ++n) {
    const long long c = chunk_for(n);
    const long long splits = (Nkv + c - 1) / c;
    const long long waves = (BH * splits + sms - 1) / sms;
    const long long cost = waves * (c + 256);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = DecodeSplit{int(c), int(splits)};
    }
  }
  return best;
}
// SM count of the current device for the decode split, or 0 with no visible device (the CUDA error
// that the query leaves is cleared, and the library's error message is left alone).
int decode_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  return n;
}
size_t decode_o_bytes(int BH, int n_split, int Nq, int d) {
  return (size_t(BH) * n_split * Nq * d * 4 + 255) & ~size_t(255);
}
// Two partials per split (one per key half of the split kernel's tile).
size_t decode_ws_bytes(int BH, int Nq, int Nkv, int d, int sms) {
  const DecodeSplit sp = decode_split(BH, Nkv, sms);
  const int n_part = 2 * sp.n_split;
  return decode_o_bytes(BH, n_part, Nq, d) + ((size_t(BH) * n_part * Nq * 2 * 4 + 255) & ~size_t(255));
}

template <int D>
fa_status launch_decode(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const fa::DecodeParams& p,
                        cudaStream_t s) {
  using L = fa::DecodeLayout<D>;
  fa_status st = set_smem(fa::fa_decode_split_kernel<D>, L::BYTES);
  if (st != FA_OK) return st;
  fa::fa_decode_split_kernel<D><<<dim3(p.n_split, p.B * p.H), 192, L::BYTES, s>>>(mq, mk, mv, p);
  if ((st = launch_status("fa_fwd_decode split kernel launch")) != FA_OK) return st;
  // The combine is a programmatic dependent launch: it may be scheduled while the split kernel
  // runs and waits (griddepcontrol.wait) until that grid has completed and its writes are visible,
  // so the second launch adds no gap of its own.
  const unsigned rows = unsigned(p.B * p.H * p.Nq);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fa::fa_decode_combine_kernel<D>, p);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "fa_fwd_decode combine kernel launch: %s", cudaGetErrorString(e));
  return launch_status("fa_fwd_decode combine kernel launch");
}

// The d = 256 forward (fwd256_sm100.cuh): one query tile per CTA, 64-key blocks, persistent grid.
fa_status fwd256(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, float scale,
                 int causal, const int32_t* key_lens, float dropout_p, uint64_t seed, cudaStream_t s) {
  using L = fa::Fwd256Layout;
  CUtensorMap mq, mk, mv;
  fa_status st;
  if ((st = make_tile_map(&mq, q, B * H, N, 256, "q")) != FA_OK) return st;
  if ((st = make_tile_map(&mk, k, B * H, N, 256, "k", 64)) != FA_OK) return st;
  if ((st = make_tile_map(&mv, v, B * H, N, 256, "v", 64)) != FA_OK) return st;
  fa::Fwd256Params p{};
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.key_lens = key_lens;
  p.B = B;
  p.H = H;
  p.N = N;
  p.n_qtiles = (N + 127) / 128;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.dropout = dropout_p > 0.f ? 1 : 0;
  p.drop_thr = drop_threshold(dropout_p);
  p.drop_scale = dropout_p > 0.f ? 1.f / (1.f - dropout_p) : 1.f;
  p.seed = seed;
  p.wait_ns = g_wait_ns.load();
  int sms = 0;
  if ((st = sm_count(&sms)) != FA_OK) return st;
  const long long items = (long long)p.n_qtiles * B * H;
  const dim3 grid(unsigned(items < sms ? items : sms));
  if (p.dropout) {
    if ((st = set_smem(fa::fa_fwd256_sm100_kernel<true>, L::BYTES)) != FA_OK) return st;
    fa::fa_fwd256_sm100_kernel<true><<<grid, 256, L::BYTES, s>>>(mq, mk, mv, p);
  } else {
    if ((st = set_smem(fa::fa_fwd256_sm100_kernel<false>, L::BYTES)) != FA_OK) return st;
    fa::fa_fwd256_sm100_kernel<false><<<grid, 256, L::BYTES, s>>>(mq, mk, mv, p);
  }
  return launch_status("fa_fwd (d = 256) kernel launch");
}

// ----------------------------------------------------------------------------- paged cache
// What the append and the attention check alike; d = 64 or 128 keeps a row a whole number of threads
// and of swizzled chunks, a page of 16 keys or more keeps an MMA's 16 keys inside one page.
fa_status check_paged(int B, int Hq, int Hkv, int Nq, int d, int n_pages, int page_size, int max_pages,
                      int64_t k_page_stride, int64_t v_page_stride) {
  if (B < 1 || Hkv < 1 || Nq < 1 || n_pages < 1 || max_pages < 1)
    return fail(FA_ERR_INVALID_ARG, "B, Hkv, Nq, n_pages and max_pages must be >= 1 (got %d, %d, %d, %d, %d)", B, Hkv, Nq,
                n_pages, max_pages);
  if (Hq < 1 || Hq % Hkv != 0) return fail(FA_ERR_INVALID_ARG, "Hq = %d must be a positive multiple of Hkv = %d", Hq, Hkv);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d = %d: the paged cache supports d in {64, 128}", d);
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
    return fail(FA_ERR_UNSUPPORTED, "page_size = %d: 16, 32, 64, 128 or 256", page_size);
  if (B > fa::kPagedMaxB) return fail(FA_ERR_UNSUPPORTED, "B = %d exceeds %d", B, fa::kPagedMaxB);
  if (int64_t(B) * Hq > 65535) return fail(FA_ERR_UNSUPPORTED, "B*Hq = %lld exceeds 65535", (long long)B * Hq);
  if (Nq > (1 << 20)) return fail(FA_ERR_UNSUPPORTED, "Nq = %d is too large", Nq);
  if (int64_t(B) * max_pages * page_size >= (int64_t(1) << 31))
    return fail(FA_ERR_UNSUPPORTED, "B * max_pages * page_size = %lld must be below 2^31", (long long)B * max_pages * page_size);
  const int64_t page = int64_t(Hkv) * page_size * d;
  for (const int64_t s : {k_page_stride, v_page_stride})
    if (s < page || s % 16 != 0)
      return fail(FA_ERR_INVALID_ARG, "page stride %lld must be a multiple of 16, at least Hkv * page_size * d = %lld",
                  (long long)s, (long long)page);
  for (const int64_t s : {k_page_stride, v_page_stride})
    if (s >= (int64_t(1) << 31)) return fail(FA_ERR_UNSUPPORTED, "page stride %lld must be below 2^31", (long long)s);
  return FA_OK;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// How fa_fwd_paged cuts its rows, by sizes alone (host arithmetic).  R = (Hq / Hkv) Nq query rows share a K/V head:
//  * up to 24 rows (32 at d = 64), or what the wide kernel's plan cannot index: tiles of 8, 16, 24 (32) consecutive
//    rows, independent warps (paged_sm100.cuh);
//  * more: pairs of 128-row tiles on the tensor memory path (paged_wide_sm100.cuh).
struct PagedShape {
  bool wide;
  int rows;        // of a tile (wide: of a pair: 256)
  int tq;          // rows, or positions, per tile
  int tiles;       // tiles (pairs) per (sequence, K/V head)
  int64_t plan;    // entries of the plan
  int R;           // rows per K/V head
};
PagedShape paged_shape(int B, int Hq, int Hkv, int Nq, int d, int64_t max_keys) {
  const int g = Hq / Hkv, R = g * Nq;
  PagedShape s{};
  s.R = R;
  if (R > (d == 64 ? 32 : 24) && g <= 128) {
    s.tq = 128 / g;
    s.tiles = (Nq + 2 * s.tq - 1) / (2 * s.tq);
    s.rows = 256;
    s.plan = int64_t(B) * s.tiles + 1;
    s.wide = s.plan * ((max_keys + 127) / 128) < (int64_t(1) << 31);
    if (s.wide) return s;
  }
  s.wide = false;
  s.rows = s.tq = R <= 8 ? 8 : R <= 16 ? 16 : R <= 24 || d == 128 ? 24 : 32;
  s.tiles = (R + s.rows - 1) / s.rows;
  s.plan = B + 1;
  return s;
}
// The grids of the split and of the wide kernel: one CTA per SM; with no device a bound for any.
int paged_ctas(int sms) { return sms <= 0 || sms > 512 ? 512 : sms; }
constexpr int kPagedMostWarps = 16;
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
// The workspace: partial O, partial (m, l), plan, info; wide: redo, and for e4m3 pools the queries in 8 bits, their scales.
struct PagedSpace {
  size_t ml, plan, info, redo, q8, q_scale, total;   // byte offsets
};
PagedSpace paged_space(int B, int Hkv, const PagedShape& s, int d, int sms) {
  const size_t rows = size_t(paged_ctas(sms)) * (s.wide ? 1 : kPagedMostWarps) * 2 * s.rows;
  PagedSpace w;
  w.ml = up256(rows * d * 4);
  w.plan = w.ml + up256(rows * 8);
  w.info = w.plan + up256(size_t(s.plan) * 4);
  w.redo = w.info + up256(size_t(B) * Hkv * s.tiles * 8);
  w.q8 = w.redo + (s.wide ? up256((size_t(B) * Hkv * s.tiles + 1) * 4) : 0);
  w.q_scale = w.q8 + (s.wide ? up256(size_t(B) * Hkv * s.R * d * 2) : 0);
  w.total = w.q_scale + (s.wide ? up256(size_t(B) * Hkv * s.R * 4) : 0);
  return w;
}

// Launch as a programmatic dependent of the kernel before it on the stream: the kernel may be
// scheduled early and waits (griddepcontrol.wait) until that grid has completed.
template <typename... P>
fa_status launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, unsigned smem, cudaStream_t s, const char* what,
                           P... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p...);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return launch_status(what);
}

// Warps per row: 8 while that makes at most 4 CTAs per SM (few rows, many partials each), 4 while it makes at most 16,
// else 1.  Partials in flight per warp: 8, but with 4 warps and at most 8 partials a row on average 2, since idle slots
// cost (64 ragged sequences with 8 instead of 2: 93.3 against 90 us; 5 drafted tokens with 2 instead of 8: 29.8 against
// 28.2 us; 1 x 1000 keys with 4 instead of 8: 9.7 against 8.9 us).
template <int D>
fa_status launch_paged_combine(const fa::PagedParams& p, int tile_rows, int sms, cudaStream_t s) {
  const long long rows = (long long)p.B * p.Hkv * p.R;
  const char* what = "fa_fwd_paged combine kernel launch";
  auto launch = [&](void (*kernel)(fa::PagedParams, int), long long ctas) {
    return launch_dependent<fa::PagedParams, int>(kernel, unsigned(ctas), 256, 0, s, what, p, tile_rows);
  };
  if (rows <= 4LL * sms) return launch(fa::fa_paged_combine_kernel<D, 8, 8>, rows);
  if (rows > 32LL * sms) return launch(fa::fa_paged_combine_kernel<D, 1, 4>, (rows + 7) / 8);
  const bool many = (long long)p.n_warps > 8LL * p.B * p.Hkv * p.row_tiles;
  return launch(many ? fa::fa_paged_combine_kernel<D, 4, 8> : fa::fa_paged_combine_kernel<D, 4, 2>, (rows + 1) / 2);
}

template <int D, bool FP8, int NG>
fa_status launch_paged(fa::WideParams q, int sms, cudaStream_t s) {
  using Lt = fa::PagedLayout<D, FP8, NG>;
  static_assert(Lt::WARPS <= kPagedMostWarps && Lt::bytes(fa::kPagedMaxB) <= 232448, "workspace, shared memory");
  const int ctas = paged_ctas(sms);
  q.p.n_warps = ctas * Lt::WARPS;
  static std::atomic<uint64_t> smem_set{0};
  fa_status st = set_smem_once(fa::fa_paged_split_kernel<D, FP8, NG>, Lt::bytes(fa::kPagedMaxB), smem_set);
  if (st != FA_OK) return st;
  st = launch_dependent<fa::PagedParams>(fa::fa_paged_split_kernel<D, FP8, NG>, unsigned(ctas), 32 * Lt::WARPS,
                                         unsigned(Lt::bytes(q.p.B)), s, "fa_fwd_paged split kernel launch", q.p);
  if (st != FA_OK) return st;
  return launch_paged_combine<D>(q.p, 8 * NG, sms, s);
}

// Pool of pages as {d, page_size, Hkv, n_pages}, loaded page by page (at most 128 rows): 64 features with the
// 128-byte swizzle in bf16; in e4m3 whole rows, K swizzled by their length for the MMA, V not (it is converted).
fa_status make_pool_map(CUtensorMap* map, const void* ptr, bool fp8, bool is_k, int d, int page_size, int Hkv, int n_pages,
                        int64_t page_bytes, const char* name) {
  auto fn = encode_fn();
  if (fn == nullptr) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
  const cuuint64_t row = cuuint64_t(d) * (fp8 ? 1 : 2);
  const cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(page_size), cuuint64_t(Hkv), cuuint64_t(n_pages)};
  const cuuint64_t strides[3] = {row, row * page_size, cuuint64_t(page_bytes)};
  const cuuint32_t box[4] = {cuuint32_t(fp8 ? d : 64), cuuint32_t(page_size < 128 ? page_size : 128), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr),
                        dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        fp8 && !is_k ? CU_TENSOR_MAP_SWIZZLE_NONE : fp8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with CUresult %d", name, int(r));
  return FA_OK;
}
// Queries as {d, heads of a group, Nq, B * Hkv}: a box is 64 features (8 bits: all of them) of all the group's heads
// at tq positions.
fa_status make_group_map(CUtensorMap* map, const void* ptr, bool bits8, int d, int g, int Nq, int BH, int tq) {
  auto fn = encode_fn();
  if (fn == nullptr) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
  const cuuint64_t row = cuuint64_t(d) * (bits8 ? 1 : 2);
  const cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(g), cuuint64_t(Nq), cuuint64_t(BH)};
  const cuuint64_t strides[3] = {row * Nq, row, row * Nq * g};
  const cuuint32_t box[4] = {cuuint32_t(bits8 ? d : 64), cuuint32_t(g), cuuint32_t(tq), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, bits8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr),
                        dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        bits8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled(q) failed with CUresult %d", int(r));
  return FA_OK;
}

template <int D, bool FP8>
fa_status launch_paged_wide(fa::WideParams q, int page_size, int sms, cudaStream_t s) {
  using L = fa::WideLayout<D, FP8>;
  q.p.n_warps = paged_ctas(sms);
  CUtensorMap mq, mq2, mk, mv;
  fa_status st;
  const fa::PagedParams& p = q.p;
  const int64_t rows = int64_t(p.B) * p.Hkv * p.R;
  const void* q1 = FP8 ? static_cast<const void*>(q.q8) : p.q;
  const void* q2 = FP8 ? static_cast<const void*>(q.q8 + rows * D) : p.q;   // (bf16: not used)
  if ((st = make_group_map(&mq, q1, FP8, D, q.g, p.Nq, p.B * p.Hkv, q.tq)) != FA_OK) return st;
  if ((st = make_group_map(&mq2, q2, FP8, D, q.g, p.Nq, p.B * p.Hkv, q.tq)) != FA_OK) return st;
  if ((st = make_pool_map(&mk, p.k, FP8, true, D, page_size, p.Hkv, p.n_pages, p.k_page_bytes, "k_cache")) != FA_OK) return st;
  if ((st = make_pool_map(&mv, p.v, FP8, false, D, page_size, p.Hkv, p.n_pages, p.v_page_bytes, "v_cache")) != FA_OK) return st;
  auto kernel = fa::fa_paged_wide_kernel<D, FP8>;
  if ((st = set_smem(kernel, L::BYTES)) != FA_OK) return st;
  if ((st = check_launch_regs(kernel, L::LAUNCH_REGS, "fa_fwd_paged wide kernel")) != FA_OK) return st;
  // one CTA plans; e4m3: the others, at most two per SM, prepare the queries, D / 8 threads a row
  const int64_t split = FP8 ? std::min<int64_t>((rows + 8191 / D) / (8192 / D), 2 * sms) : 0;
  st = launch_dependent<fa::WideParams>(fa::fa_paged_plan_kernel<D, FP8>, unsigned(1 + split), 1024, 0, s,
                                        "fa_fwd_paged plan kernel launch", q);
  if (st != FA_OK) return st;
  st = launch_dependent<CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, fa::WideParams>(
      kernel, unsigned(paged_ctas(sms)), unsigned(L::THREADS), unsigned(L::BYTES), s, "fa_fwd_paged wide kernel launch", mq, mq2, mk, mv, q);
  if (st != FA_OK) return st;
  // pairs < 2^27: B Hq Nq < 2^31, and all but the last pair of a head have more than 126 rows
  const unsigned pairs = unsigned(p.B) * p.Hkv * q.n_pairs;
  st = launch_dependent<fa::WideParams>(fa::fa_paged_wide_combine_kernel<D>, pairs * fa::kWideMergeCtas, 256, 0, s,
                                        "fa_fwd_paged combine kernel launch", q);
  if (st != FA_OK || !p.causal || p.Nq == 1) return st;
  return launch_dependent<fa::WideParams>(fa::fa_paged_wide_redo_kernel<D>, unsigned(2 * sms), 256, 0, s, "fa_fwd_paged redo kernel launch", q);
}

template <int D>
fa_status launch_paged_rows(const fa::WideParams& q, bool fp8, int rows, int sms, cudaStream_t s) {
  if constexpr (D == 64)
    if (rows == 32) return fp8 ? launch_paged<D, true, 4>(q, sms, s) : launch_paged<D, false, 4>(q, sms, s);
  if (rows == 24) return fp8 ? launch_paged<D, true, 3>(q, sms, s) : launch_paged<D, false, 3>(q, sms, s);
  if (rows == 16) return fp8 ? launch_paged<D, true, 2>(q, sms, s) : launch_paged<D, false, 2>(q, sms, s);
  return fp8 ? launch_paged<D, true, 1>(q, sms, s) : launch_paged<D, false, 1>(q, sms, s);
}

fa_status run_paged(bool fp8, const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                    const float* v_scale, void* o, float* lse, int64_t k_page_stride, int64_t v_page_stride,
                    const int32_t* page_table, const int32_t* key_lens, const int32_t* new_lens, int B, int Hq, int Hkv,
                    int Nq, int d, int n_pages, int page_size, int max_pages, float scale, int causal, void* workspace,
                    size_t workspace_bytes, cudaStream_t s) {
  fa_status st = check_paged(B, Hq, Hkv, Nq, d, n_pages, page_size, max_pages, k_page_stride, v_page_stride);
  if (st != FA_OK) return st;
  if (int64_t(B) * Hq * Nq >= (int64_t(1) << 31))
    return fail(FA_ERR_UNSUPPORTED, "B * Hq * Nq = %lld must be below 2^31", (long long)B * Hq * Nq);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  FA_CHECK_PTR(q);
  FA_CHECK_PTR(k_cache);
  FA_CHECK_PTR(v_cache);
  FA_CHECK_PTR(o);
  FA_CHECK_PTR(lse);
  FA_CHECK_WORDS(page_table);
  FA_CHECK_WORDS(key_lens);
  if (new_lens != nullptr) FA_CHECK_WORDS(new_lens);
  // (rows of q are read again after others' o is there, where a pair is computed anew)
  const uint64_t at_q = reinterpret_cast<uintptr_t>(q), at_o = reinterpret_cast<uintptr_t>(o), bytes = uint64_t(B) * Hq * Nq * d * 2;
  if ((at_o > at_q ? at_o - at_q : at_q - at_o) < bytes) return fail(FA_ERR_INVALID_ARG, "o overlaps q");
  if (fp8) {
    FA_CHECK_WORDS(k_scale);
    FA_CHECK_WORDS(v_scale);
  }
  if (workspace == nullptr) return fail(FA_ERR_INVALID_ARG, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(FA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  int sms = 0;
  const PagedShape shape = paged_shape(B, Hq, Hkv, Nq, d, int64_t(max_pages) * page_size);
  const size_t least = paged_space(B, Hkv, shape, d, 1).total;   // refused without a device too
  if (workspace_bytes < least) return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, needs more than %zu", workspace_bytes, least);
  if ((st = sm_count(&sms)) != FA_OK) return st;
  const PagedSpace space = paged_space(B, Hkv, shape, d, sms);
  if (workspace_bytes < space.total)
    return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", workspace_bytes, space.total);
  fa::WideParams q4{};
  fa::PagedParams& p = q4.p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const uint8_t*>(k_cache);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + space.ml);
  p.plan = reinterpret_cast<int*>(ws + space.plan);
  p.info = reinterpret_cast<int2*>(ws + space.info);
  p.page_table = page_table;
  p.key_lens = key_lens;
  p.new_lens = new_lens;
  p.k_page_bytes = uint32_t(k_page_stride * (fp8 ? 1 : 2));
  p.v_page_bytes = uint32_t(v_page_stride * (fp8 ? 1 : 2));
  p.B = B;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.R = Hq / Hkv * Nq;
  p.row_tiles = shape.tiles;
  p.n_pages = n_pages;
  p.page_shift = log2_of(page_size);
  p.max_pages = max_pages;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  q4.g = Hq / Hkv;
  q4.tq = shape.tq;
  q4.n_pairs = shape.tiles;
  q4.redo = reinterpret_cast<int*>(ws + space.redo);
  q4.q8 = reinterpret_cast<uint8_t*>(ws + space.q8);
  q4.q_scale = reinterpret_cast<float*>(ws + space.q_scale);
  q4.wait_ns = g_wait_ns.load();
  q4.debug_flags = g_debug_flags.load();
  if (shape.wide) {
    if (d == 64) return fp8 ? launch_paged_wide<64, true>(q4, page_size, sms, s) : launch_paged_wide<64, false>(q4, page_size, sms, s);
    return fp8 ? launch_paged_wide<128, true>(q4, page_size, sms, s) : launch_paged_wide<128, false>(q4, page_size, sms, s);
  }
  return d == 64 ? launch_paged_rows<64>(q4, fp8, shape.rows, sms, s) : launch_paged_rows<128>(q4, fp8, shape.rows, sms, s);
}

// Bytes from the first element to the end of the last of a bf16 array [B, H, N, d] with element strides st (batch, head, token).
uint64_t span_of(int B, int H, int N, int d, const int64_t* st) {
  return 2 * (uint64_t(B - 1) * st[0] + uint64_t(H - 1) * st[1] + uint64_t(N - 1) * st[2] + d);
}
bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < na : x - y < nb;
}

fa_status run_append(bool fp8, const void* q, const void* k, const void* v, const int64_t* strides, void* q_out,
                     void* k_cache, void* v_cache, float* k_scale, float* v_scale, int64_t k_page_stride,
                     int64_t v_page_stride, const int32_t* page_table, const int32_t* key_lens, const int32_t* new_lens,
                     const float* rope_cos, const float* rope_sin, int max_pos, int rot_dim, int interleaved, int B, int Hq,
                     int Hkv, int Nq, int d, int n_pages, int page_size, int max_pages, cudaStream_t s) {
  fa_status st = check_paged(B, q == nullptr ? Hkv : Hq, Hkv, Nq, d, n_pages, page_size, max_pages, k_page_stride, v_page_stride);
  if (st != FA_OK) return st;
  FA_CHECK_PTR(k);
  FA_CHECK_PTR(v);
  if (q != nullptr) {
    FA_CHECK_PTR(q);
    FA_CHECK_PTR(q_out);
  }
  FA_CHECK_PTR(k_cache);
  FA_CHECK_PTR(v_cache);
  if (fp8) {
    FA_CHECK_WORDS(k_scale);
    FA_CHECK_WORDS(v_scale);
  }
  FA_CHECK_WORDS(page_table);
  FA_CHECK_WORDS(key_lens);
  if (new_lens != nullptr) FA_CHECK_WORDS(new_lens);
  if (strides == nullptr) return fail(FA_ERR_INVALID_ARG, "strides is NULL");
  for (int i = q == nullptr ? 3 : 0; i < 9; ++i)
    if (strides[i] < 0 || strides[i] % 8 != 0)
      return fail(FA_ERR_INVALID_ARG, "strides[%d] = %lld must be a multiple of 8, >= 0", i, (long long)strides[i]);
  if ((rope_cos == nullptr) != (rope_sin == nullptr)) return fail(FA_ERR_INVALID_ARG, "rope_cos and rope_sin go together");
  if (rope_cos != nullptr) {
    FA_CHECK_PTR(rope_cos);
    FA_CHECK_PTR(rope_sin);
    if (rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0)
      return fail(FA_ERR_UNSUPPORTED, "rot_dim = %d: a multiple of 16, at most d = %d", rot_dim, d);
    if (max_pos < 1) return fail(FA_ERR_INVALID_ARG, "max_pos = %d must be >= 1", max_pos);
  }
  if (q != nullptr) {   // a thread writes a query row where it read it; elsewhere another thread may not have read yet
    const uint64_t out = 2 * uint64_t(B) * Hq * Nq * d;
    const bool contiguous = (B == 1 || strides[0] == int64_t(Hq) * Nq * d) && (Hq == 1 || strides[1] == int64_t(Nq) * d) &&
                            (Nq == 1 || strides[2] == d);
    if (!(q_out == q && contiguous) && overlap(q_out, out, q, span_of(B, Hq, Nq, d, strides)))
      return fail(FA_ERR_INVALID_ARG, "q_out overlaps q");
    if (overlap(q_out, out, k, span_of(B, Hkv, Nq, d, strides + 3)) || overlap(q_out, out, v, span_of(B, Hkv, Nq, d, strides + 6)))
      return fail(FA_ERR_INVALID_ARG, "q_out overlaps k or v");
  }
  fa::AppendParams p{};
  const void* x[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    p.x[i] = static_cast<const __nv_bfloat16*>(x[i]);
    p.sb[i] = strides[3 * i];
    p.sh[i] = strides[3 * i + 1];
    p.sn[i] = strides[3 * i + 2];
  }
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.pool[0] = static_cast<uint8_t*>(k_cache);
  p.pool[1] = static_cast<uint8_t*>(v_cache);
  p.page_bytes[0] = k_page_stride * (fp8 ? 1 : 2);
  p.page_bytes[1] = v_page_stride * (fp8 ? 1 : 2);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.page_table = page_table;
  p.key_lens = key_lens;
  p.new_lens = new_lens;
  p.cos = rope_cos;
  p.sin = rope_sin;
  p.B = B;
  p.Hq = q == nullptr ? 0 : Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.d = d;
  p.rot = rope_cos == nullptr ? 0 : rot_dim;
  p.interleaved = interleaved ? 1 : 0;
  p.max_pos = max_pos;
  p.n_pages = n_pages;
  p.page_shift = log2_of(page_size);
  p.max_pages = max_pages;
  int sms = 0;
  if ((st = sm_count(&sms)) != FA_OK) return st;
  const int heads = p.Hq + (fp8 ? 0 : 2 * Hkv);
  const int64_t tokens = int64_t(B) * Nq;
  // the row role's blocks hold `threads` threads of d / 16 per token; a thread takes up to 8 heads of its token
  // as long as that leaves about 2048 threads per SM
  auto rows = [&](int threads) -> int64_t {
    const int per = threads / (d / 16);
    const int64_t x = (tokens + per - 1) / per;
    p.heads_per_thread = 1;
    while (p.heads_per_thread < 8 && tokens * (d / 16) * heads / (2 * p.heads_per_thread) >= int64_t(sms) * 2048) p.heads_per_thread *= 2;
    const int64_t blocks = heads == 0 ? 0 : x * ((heads + p.heads_per_thread - 1) / p.heads_per_thread);
    p.row_blocks_x = int(x);
    p.row_blocks = int(blocks);
    return blocks;
  };
  if (!fp8) {
    if (rows(128) >= (int64_t(1) << 31)) return fail(FA_ERR_UNSUPPORTED, "B * Nq = %lld tokens are too many", (long long)tokens);
    return launch_dependent<fa::AppendParams>(fa::fa_kv_append_kernel, unsigned(p.row_blocks), 128, 0, s, "fa_kv_append kernel launch", p);
  }
  p.touched = (Nq + page_size - 2) / page_size + 1;
  const int most = Nq < page_size ? Nq : page_size;   // new rows of one page
  const int lpr = d / 16;
  int threads = 32;
  while (threads / lpr * 4 < most) threads *= 2;
  const int64_t blocks = rows(threads) + int64_t(B) * p.touched * Hkv * 2;
  if (blocks >= (int64_t(1) << 31)) return fail(FA_ERR_UNSUPPORTED, "too many pages to append to (%lld)", (long long)blocks);
  const unsigned grid = unsigned(blocks);
  const char* what = "fa_kv_append_e4m3 kernel launch";
  auto kernel = threads == 32    ? fa::fa_kv_append_e4m3_kernel<32>
                : threads == 64  ? fa::fa_kv_append_e4m3_kernel<64>
                : threads == 128 ? fa::fa_kv_append_e4m3_kernel<128>
                : threads == 256 ? fa::fa_kv_append_e4m3_kernel<256>
                                 : fa::fa_kv_append_e4m3_kernel<512>;
  return launch_dependent<fa::AppendParams>(kernel, grid, unsigned(threads), 0, s, what, p);
}

unsigned grid_for(uint64_t work, unsigned per_block) {
  const uint64_t g = (work + per_block - 1) / per_block;
  return unsigned(g < 1 ? 1 : (g > (1u << 30) ? (1u << 30) : g));
}

}  // namespace

extern "C" {

int fa_bwd_head_group(int N, int d, size_t l2_bytes) {
  // Q, dO (bf16) and the fp32 dQ accumulator of one head: 8 * N * d bytes.  A group fills about a
  // quarter of L2, rounded to the nearest whole head (measured best on the 126 MB B200: groups of 8
  // heads at N = 4096, d = 128), 1..16 heads.
  if (N < 1 || d < 1) return 1;
  const uint64_t per_head = 8ull * uint64_t(N) * uint64_t(d);
  const uint64_t g = (uint64_t(l2_bytes) / 4 + per_head / 2) / per_head;
  return int(g < 1 ? 1 : (g > 16 ? 16 : g));
}

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
                 float scale, int causal, const int32_t* key_lens, float dropout_p, uint64_t seed, cudaStream_t stream) {
  fa_status st = check_common(B, H, N, d, scale, dropout_p, Dims::kBf16Fwd);
  if (st != FA_OK) return st;
  FA_CHECK_PTR(q);
  FA_CHECK_PTR(k);
  FA_CHECK_PTR(v);
  FA_CHECK_PTR(o);
  FA_CHECK_PTR(lse);
  if (d == 256) return fwd256(q, k, v, o, lse, B, H, N, scale, causal, key_lens, dropout_p, seed, stream);
  CUtensorMap mq, mk, mv;
  if ((st = make_tile_map(&mq, q, B * H, N, d, "q")) != FA_OK) return st;
  if ((st = make_tile_map(&mk, k, B * H, N, d, "k")) != FA_OK) return st;
  if ((st = make_tile_map(&mv, v, B * H, N, d, "v")) != FA_OK) return st;
  fa::FwdParams p{};
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.key_lens = key_lens;
  p.B = B;
  p.H = H;
  p.N = N;
  p.n_qtiles = (N + 127) / 128;
  p.n_pairs = (p.n_qtiles + 1) / 2;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.dropout = dropout_p > 0.f ? 1 : 0;
  p.drop_thr = drop_threshold(dropout_p);
  p.drop_scale = dropout_p > 0.f ? 1.f / (1.f - dropout_p) : 1.f;
  p.seed = seed;
  p.wait_ns = g_wait_ns.load();
  p.debug_flags = g_debug_flags.load();
  p.o_align32 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0 ? 1 : 0;
  cudaStream_t s = stream;
  if (d == 64) return p.dropout ? launch_fwd<64, true>(mq, mk, mv, p, s) : launch_fwd<64, false>(mq, mk, mv, p, s);
  return p.dropout ? launch_fwd<128, true>(mq, mk, mv, p, s) : launch_fwd<128, false>(mq, mk, mv, p, s);
}

fa_status fa_fwd_f32(const float* q, const float* k, const float* v, float* o, float* lse, int B, int H, int N, int d,
                     float scale, int causal, const int32_t* key_lens, float dropout_p, uint64_t seed, cudaStream_t stream) {
  fa_status st = check_common(B, H, N, d, scale, dropout_p, Dims::kF32);
  if (st != FA_OK) return st;
  FA_CHECK_PTR(q);
  FA_CHECK_PTR(k);
  FA_CHECK_PTR(v);
  FA_CHECK_PTR(o);
  FA_CHECK_PTR(lse);
  fa::F32Params p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.lse = lse;
  p.key_lens = key_lens;
  p.B = B;
  p.H = H;
  p.N = N;
  p.d = d;
  p.causal = causal ? 1 : 0;
  p.scale = scale;
  p.dropout = dropout_p > 0.f ? 1 : 0;
  p.drop_thr = drop_threshold(dropout_p);
  p.drop_scale = dropout_p > 0.f ? 1.f / (1.f - dropout_p) : 1.f;
  p.seed = seed;
  cudaStream_t s = stream;
  const dim3 grid((N + 63) / 64, B * H);   // 64 query rows per CTA
  if (d <= 32)
    fa::fa_fwd_f32_kernel<32><<<grid, 128, 0, s>>>(p);
  else if (d <= 64)
    fa::fa_fwd_f32_kernel<64><<<grid, 128, 0, s>>>(p);
  else if (d <= 96)
    fa::fa_fwd_f32_kernel<96><<<grid, 128, 0, s>>>(p);
  else
    fa::fa_fwd_f32_kernel<128><<<grid, 128, 0, s>>>(p);
  return launch_status("fa_fwd_f32 kernel launch");
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1 || d < 1) return 0;
  return ws_total_bytes(B, H, N, d);
}

fa_status fa_bwd_prep(const void* o, const void* dO, int B, int H, int N, int d, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
  fa_status st = check_common(B, H, N, d, 1.f, 0.f, Dims::kBf16);
  if (st != FA_OK) return st;
  FA_CHECK_PTR(o);
  FA_CHECK_PTR(dO);
  Workspace w;
  if ((st = check_workspace(workspace, workspace_bytes, B, H, N, d, &w)) != FA_OK) return st;
  fa::BwdParams p = bwd_params(B, H, N, 1.f, 0, nullptr, 0.f, 0, w);
  p.o = static_cast<const __nv_bfloat16*>(o);
  p.dO = static_cast<const __nv_bfloat16*>(dO);
  cudaStream_t s = stream;
  const uint64_t threads = uint64_t(B) * H * N * (d / 8);
  if (d == 64)
    fa::fa_bwd_prep_kernel<64><<<grid_for(threads, 256), 256, 0, s>>>(p);
  else
    fa::fa_bwd_prep_kernel<128><<<grid_for(threads, 256), 256, 0, s>>>(p);
  return launch_status("fa_bwd_prep kernel launch");
}

fa_status fa_bwd_main(const void* q, const void* k, const void* v, const float* lse, const void* dO, void* dk, void* dv,
                      int B, int H, int N, int d, float scale, int causal, const int32_t* key_lens, float dropout_p,
                      uint64_t seed, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  fa_status st = check_common(B, H, N, d, scale, dropout_p, Dims::kBf16);
  if (st != FA_OK) return st;
  FA_CHECK_PTR(q);
  FA_CHECK_PTR(k);
  FA_CHECK_PTR(v);
  FA_CHECK_PTR(lse);
  FA_CHECK_PTR(dO);
  FA_CHECK_PTR(dk);
  FA_CHECK_PTR(dv);
  Workspace w;
  if ((st = check_workspace(workspace, workspace_bytes, B, H, N, d, &w)) != FA_OK) return st;
  CUtensorMap mq, mk, mv, mdo;
  if ((st = make_tile_map(&mq, q, B * H, N, d, "q")) != FA_OK) return st;
  if ((st = make_tile_map(&mk, k, B * H, N, d, "k")) != FA_OK) return st;
  if ((st = make_tile_map(&mv, v, B * H, N, d, "v")) != FA_OK) return st;
  if ((st = make_tile_map(&mdo, dO, B * H, N, d, "dO")) != FA_OK) return st;
  fa::BwdParams p = bwd_params(B, H, N, scale, causal, key_lens, dropout_p, seed, w);
  p.lse = lse;
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.out_align32 = ((reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv)) & 31u) == 0 ? 1 : 0;
  cudaStream_t s = stream;
  if (d == 64)
    return p.dropout ? launch_bwd_main<64, true, true>(mq, mk, mv, mdo, p, s)
                     : launch_bwd_main<64, false, true>(mq, mk, mv, mdo, p, s);
  return p.dropout ? launch_bwd_main<128, true, true>(mq, mk, mv, mdo, p, s)
                   : launch_bwd_main<128, false, true>(mq, mk, mv, mdo, p, s);
}

fa_status fa_bwd_split(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                       void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal,
                       const int32_t* key_lens, float dropout_p, uint64_t seed, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
  fa_status st = check_common(B, H, N, d, scale, dropout_p, Dims::kBf16);
  if (st != FA_OK) return st;
  FA_CHECK_PTR(q);
  FA_CHECK_PTR(k);
  FA_CHECK_PTR(v);
  FA_CHECK_PTR(lse);
  FA_CHECK_PTR(dO);
  FA_CHECK_PTR(dq);
  FA_CHECK_PTR(dk);
  FA_CHECK_PTR(dv);
  Workspace w;
  if ((st = check_workspace(workspace, workspace_bytes, B, H, N, d, &w)) != FA_OK) return st;
  if ((st = fa_bwd_prep(o, dO, B, H, N, d, workspace, workspace_bytes, stream)) != FA_OK) return st;
  CUtensorMap mq, mk, mv, mdo;
  if ((st = make_tile_map(&mq, q, B * H, N, d, "q")) != FA_OK) return st;
  if ((st = make_tile_map(&mk, k, B * H, N, d, "k")) != FA_OK) return st;
  if ((st = make_tile_map(&mv, v, B * H, N, d, "v")) != FA_OK) return st;
  if ((st = make_tile_map(&mdo, dO, B * H, N, d, "dO")) != FA_OK) return st;
  // dK and dV: the main kernel without its dQ part
  fa::BwdParams p = bwd_params(B, H, N, scale, causal, key_lens, dropout_p, seed, w);
  p.lse = lse;
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.out_align32 = ((reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv)) & 31u) == 0 ? 1 : 0;
  if (d == 64)
    st = p.dropout ? launch_bwd_main<64, true, false>(mq, mk, mv, mdo, p, stream)
                   : launch_bwd_main<64, false, false>(mq, mk, mv, mdo, p, stream);
  else
    st = p.dropout ? launch_bwd_main<128, true, false>(mq, mk, mv, mdo, p, stream)
                   : launch_bwd_main<128, false, false>(mq, mk, mv, mdo, p, stream);
  if (st != FA_OK) return st;
  // dQ: its own pass, query-tile-major
  fa::DqParams dp{};
  dp.dq = static_cast<__nv_bfloat16*>(dq);
  dp.lse = lse;
  dp.dvec = w.dvec;
  dp.key_lens = key_lens;
  dp.B = B;
  dp.H = H;
  dp.N = N;
  dp.n_qtiles = (N + 127) / 128;
  dp.causal = causal ? 1 : 0;
  dp.scale = scale;
  dp.scale_log2 = scale * 1.4426950408889634f;
  dp.dropout = dropout_p > 0.f ? 1 : 0;
  dp.drop_thr = drop_threshold(dropout_p);
  dp.drop_scale = dropout_p > 0.f ? 1.f / (1.f - dropout_p) : 1.f;
  dp.seed = seed;
  dp.wait_ns = g_wait_ns.load();
  int sms = 0;
  if ((st = sm_count(&sms)) != FA_OK) return st;
  const long long items = (long long)dp.n_qtiles * B * H;
  const dim3 grid(unsigned(items < sms ? items : sms));
  if (d == 64)
    return dp.dropout ? launch_dq_pass<64, true>(mq, mk, mv, mdo, dp, grid, stream)
                      : launch_dq_pass<64, false>(mq, mk, mv, mdo, dp, grid, stream);
  return dp.dropout ? launch_dq_pass<128, true>(mq, mk, mv, mdo, dp, grid, stream)
                    : launch_dq_pass<128, false>(mq, mk, mv, mdo, dp, grid, stream);
}

fa_status fa_bwd_dq_convert(void* dq, int B, int H, int N, int d, float scale, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  fa_status st = check_common(B, H, N, d, scale, 0.f, Dims::kBf16);
  if (st != FA_OK) return st;
  FA_CHECK_PTR(dq);
  Workspace w;
  if ((st = check_workspace(workspace, workspace_bytes, B, H, N, d, &w)) != FA_OK) return st;
  fa::BwdParams p = bwd_params(B, H, N, scale, 0, nullptr, 0.f, 0, w);
  p.dq = static_cast<__nv_bfloat16*>(dq);
  cudaStream_t s = stream;
  const uint64_t n8 = uint64_t(B) * H * N * d / 8;
  int sms = 0;
  if ((st = sm_count(&sms)) != FA_OK) return st;
  const unsigned cap = unsigned(sms) * 16u;   // grid-stride loop: 16 blocks of 256 threads per SM
  const unsigned grid = grid_for(n8, 256) > cap ? cap : grid_for(n8, 256);
  if (d == 64)
    fa::fa_bwd_dq_kernel<64><<<grid, 256, 0, s>>>(p);
  else
    fa::fa_bwd_dq_kernel<128><<<grid, 256, 0, s>>>(p);
  return launch_status("fa_bwd_dq_convert kernel launch");
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO, void* dq,
                 void* dk, void* dv, int B, int H, int N, int d, float scale, int causal, const int32_t* key_lens,
                 float dropout_p, uint64_t seed, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  FA_CHECK_PTR(dq);
  fa_status st = fa_bwd_prep(o, dO, B, H, N, d, workspace, workspace_bytes, stream);
  if (st != FA_OK) return st;
  st = fa_bwd_main(q, k, v, lse, dO, dk, dv, B, H, N, d, scale, causal, key_lens, dropout_p, seed, workspace,
                   workspace_bytes, stream);
  if (st != FA_OK) return st;
  return fa_bwd_dq_convert(dq, B, H, N, d, scale, workspace, workspace_bytes, stream);
}

size_t fa_fwd_decode_workspace_size(int B, int H, int Nq, int Nkv, int d) {
  if (B < 1 || H < 1 || Nq < 1 || Nkv < 1 || d < 1) return 0;
  return decode_ws_bytes(B * H, Nq, Nkv, d, decode_sms());
}

int fa_fwd_decode_split(int B, int H, int Nkv, int sms) {
  if (B < 1 || H < 1 || Nkv < 1) return 0;
  return decode_split(B * H, Nkv, sms).n_split;
}

fa_status fa_fwd_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
                        int Nkv, int d, float scale, int causal, const int32_t* key_lens, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  fa_status st = check_common(B, H, Nkv, d, scale, 0.f, Dims::kBf16);
  if (st != FA_OK) return st;
  if (Nq < 1 || Nq > 64) return fail(FA_ERR_UNSUPPORTED, "Nq = %d: fa_fwd_decode takes 1 <= Nq <= 64", Nq);
  FA_CHECK_PTR(q);
  FA_CHECK_PTR(k);
  FA_CHECK_PTR(v);
  FA_CHECK_PTR(o);
  FA_CHECK_PTR(lse);
  if (workspace == nullptr) return fail(FA_ERR_INVALID_ARG, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(FA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
  const int sms = decode_sms();
  const size_t need = decode_ws_bytes(B * H, Nq, Nkv, d, sms);
  if (workspace_bytes < need) return fail(FA_ERR_INVALID_ARG, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  const DecodeSplit sp = decode_split(B * H, Nkv, sms);
  CUtensorMap mq, mk, mv;
  if ((st = make_tile_map(&mq, q, B * H, Nq, d, "q", 64)) != FA_OK) return st;
  if ((st = make_tile_map(&mk, k, B * H, Nkv, d, "k")) != FA_OK) return st;
  if ((st = make_tile_map(&mv, v, B * H, Nkv, d, "v")) != FA_OK) return st;
  fa::DecodeParams p{};
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + decode_o_bytes(B * H, 2 * sp.n_split, Nq, d));
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.key_lens = key_lens;
  p.B = B;
  p.H = H;
  p.Nq = Nq;
  p.Nkv = Nkv;
  p.chunk = sp.chunk;
  p.n_split = sp.n_split;
  p.n_part = 2 * sp.n_split;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_ns = g_wait_ns.load();
  return d == 64 ? launch_decode<64>(mq, mk, mv, p, stream) : launch_decode<128>(mq, mk, mv, p, stream);
}

size_t fa_fwd_paged_workspace_size(int B, int Hq, int Hkv, int Nq, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Nq < 1 || d < 1 || B > fa::kPagedMaxB) return 0;
  if (int64_t(B) * Hq * Nq >= (int64_t(1) << 31)) return 0;
  // enough for either way of cutting the rows (which one it is depends on the page table's width too)
  const int sms = decode_sms();
  const size_t wide = paged_space(B, Hkv, paged_shape(B, Hq, Hkv, Nq, d, 0), d, sms).total;
  const size_t narrow = paged_space(B, Hkv, paged_shape(B, Hq, Hkv, Nq, d, int64_t(1) << 40), d, sms).total;
  return wide > narrow ? wide : narrow;
}

fa_status fa_fwd_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse, int64_t k_page_stride,
                       int64_t v_page_stride, const int32_t* page_table, const int32_t* key_lens, const int32_t* new_lens,
                       int B, int Hq, int Hkv, int Nq, int d, int n_pages, int page_size, int max_pages, float scale,
                       int causal, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return run_paged(false, q, k_cache, v_cache, nullptr, nullptr, o, lse, k_page_stride, v_page_stride, page_table, key_lens,
                   new_lens, B, Hq, Hkv, Nq, d, n_pages, page_size, max_pages, scale, causal, workspace, workspace_bytes,
                   stream);
}

fa_status fa_fwd_paged_e4m3(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                            const float* v_scale, void* o, float* lse, int64_t k_page_stride, int64_t v_page_stride,
                            const int32_t* page_table, const int32_t* key_lens, const int32_t* new_lens, int B, int Hq,
                            int Hkv, int Nq, int d, int n_pages, int page_size, int max_pages, float scale, int causal,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return run_paged(true, q, k_cache, v_cache, k_scale, v_scale, o, lse, k_page_stride, v_page_stride, page_table, key_lens,
                   new_lens, B, Hq, Hkv, Nq, d, n_pages, page_size, max_pages, scale, causal, workspace, workspace_bytes,
                   stream);
}

fa_status fa_kv_append(const void* q, const void* k, const void* v, const int64_t* strides, void* q_out, void* k_cache,
                       void* v_cache, int64_t k_page_stride, int64_t v_page_stride, const int32_t* page_table,
                       const int32_t* key_lens, const int32_t* new_lens, const float* rope_cos, const float* rope_sin,
                       int max_pos, int rot_dim, int interleaved, int B, int Hq, int Hkv, int Nq, int d, int n_pages,
                       int page_size, int max_pages, cudaStream_t stream) {
  return run_append(false, q, k, v, strides, q_out, k_cache, v_cache, nullptr, nullptr, k_page_stride, v_page_stride,
                    page_table, key_lens, new_lens, rope_cos, rope_sin, max_pos, rot_dim, interleaved, B, Hq, Hkv, Nq, d,
                    n_pages, page_size, max_pages, stream);
}

fa_status fa_kv_append_e4m3(const void* q, const void* k, const void* v, const int64_t* strides, void* q_out, void* k_cache,
                            void* v_cache, float* k_scale, float* v_scale, int64_t k_page_stride, int64_t v_page_stride,
                            const int32_t* page_table, const int32_t* key_lens, const int32_t* new_lens,
                            const float* rope_cos, const float* rope_sin, int max_pos, int rot_dim, int interleaved, int B,
                            int Hq, int Hkv, int Nq, int d, int n_pages, int page_size, int max_pages, cudaStream_t stream) {
  return run_append(true, q, k, v, strides, q_out, k_cache, v_cache, k_scale, v_scale, k_page_stride, v_page_stride,
                    page_table, key_lens, new_lens, rope_cos, rope_sin, max_pos, rot_dim, interleaved, B, Hq, Hkv, Nq, d,
                    n_pages, page_size, max_pages, stream);
}

fa_status fa_dropout_mask(uint8_t* keep, int B, int H, int N, float dropout_p, uint64_t seed, cudaStream_t stream) {
  if (keep == nullptr) return fail(FA_ERR_INVALID_ARG, "keep is NULL");
  if (B < 1 || H < 1 || N < 1) return fail(FA_ERR_INVALID_ARG, "B, H and N must be >= 1");
  if (!(dropout_p >= 0.f) || !(dropout_p < 1.f)) return fail(FA_ERR_INVALID_ARG, "dropout_p must be in [0, 1)");
  const uint64_t total = uint64_t(B) * H * N * uint64_t(N);
  cudaStream_t s = stream;
  int sms = 0;
  const fa_status st = sm_count(&sms);
  if (st != FA_OK) return st;
  const unsigned cap = unsigned(sms) * 32u;   // grid-stride loop: 32 blocks of 256 threads per SM
  const unsigned grid = grid_for(total, 256) > cap ? cap : grid_for(total, 256);
  fa::fa_dropout_mask_kernel<<<grid, 256, 0, s>>>(keep, total, N, seed, drop_threshold(dropout_p));
  return launch_status("fa_dropout_mask kernel launch");
}

fa_status fa_test_exp2_fma(const float* x, float* y, int n, cudaStream_t stream) {
  if (x == nullptr || y == nullptr) return fail(FA_ERR_INVALID_ARG, "x or y is NULL");
  if (n < 1) return fail(FA_ERR_INVALID_ARG, "n must be >= 1");
  fa::fa_exp2_fma_test_kernel<<<grid_for((uint64_t(n) + 1) / 2, 256), 256, 0, stream>>>(x, y, n);
  return launch_status("fa_test_exp2_fma kernel launch");
}

fa_status fa_check(cudaStream_t stream) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaStreamSynchronize: %s", cudaGetErrorString(e));
  int code = 0;
  e = cudaMemcpyFromSymbol(&code, fa::g_fa_device_status, sizeof(int));
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "reading the device status word: %s", cudaGetErrorString(e));
  if (code == 0) return FA_OK;
  const int zero = 0;
  e = cudaMemcpyToSymbol(fa::g_fa_device_status, &zero, sizeof(int));
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "clearing the device status word: %s", cudaGetErrorString(e));
  if (code == fa::kStatusTimeout) return fail(FA_ERR_TIMEOUT, "a kernel's bounded wait ran out");
  if (code == fa::kStatusRange)
    return fail(FA_ERR_RANGE, "a page number, length or position was outside the paged cache");
  return fail(FA_ERR_INTERNAL, "device status %d (dynamic shared memory not 1024-byte aligned)", code);
}

const char* fa_get_error(void) { return g_err; }

void fa_set_wait_limit_ns(uint64_t ns) { g_wait_ns.store(ns > 0 ? ns : default_wait_ns()); }

void fa_debug_set_flags(int flags) { g_debug_flags.store(flags); }

const char* fa_version(void) { return "exact-io-aware-attention sm_100a 0.1"; }

}  // extern "C"

// ----------------------------------------------------------------------------- backward without allocation
// Some callers cannot allocate device memory: a plugin running inside another runtime that owns
// every byte of device memory and gives its plugins no workspace, or a latency-critical loop where
// the implicit device synchronisation of cudaMalloc is not acceptable.  fa_bwd_noalloc serves
// them: the backward's scratch (the fp32 dQ accumulator and D) lives in the fixed array below,
// which is part of the library image.  Every GPU that loads the library holds these bytes until
// the process exits.
namespace {

constexpr size_t kNoallocScratchBytes = size_t(48) << 20;   // 48 MiB
static __device__ __align__(256) unsigned char g_fa_noalloc_scratch[kNoallocScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_noalloc_mu;
void* g_noalloc_addr[kMaxDevices] = {};

// The device address of the scratch array on the current device.  In host code the array's name
// is only a host-side stand-in, so the address is looked up once per device (with that device
// current) and cached.
fa_status noalloc_scratch(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(FA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(FA_ERR_UNSUPPORTED, "device ordinal %d is out of range", dev);
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_addr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_fa_noalloc_scratch);
    if (e != cudaSuccess || p == nullptr)
      return fail(FA_ERR_CUDA, "cudaGetSymbolAddress(static scratch): %s", cudaGetErrorString(e));
    g_noalloc_addr[dev] = p;
  }
  *out = g_noalloc_addr[dev];
  return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                         void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal,
                         const int32_t* key_lens, float dropout_p, uint64_t seed, cudaStream_t stream) {
  const size_t need = fa_bwd_workspace_size(B, H, N, d);
  if (need > kNoallocScratchBytes)
    return fail(FA_ERR_INVALID_ARG,
                "fa_bwd_noalloc: B=%d H=%d N=%d d=%d needs %zu bytes of scratch, more than the library's "
                "static %zu bytes; call fa_bwd with a workspace instead",
                B, H, N, d, need, kNoallocScratchBytes);
  void* ws = nullptr;
  const fa_status st = noalloc_scratch(&ws);
  if (st != FA_OK) return st;
  return fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, key_lens, dropout_p, seed, ws,
                kNoallocScratchBytes, stream);
}

size_t fa_bwd_noalloc_max_scratch(void) { return kNoallocScratchBytes; }

}  // extern "C"
