// C entry points of the operators around the MoE layer (include/moe_b200.h):
// products grouped by expert, the dense layer and its backward, and the
// orthogonalised update. Argument checks, tensor maps and launches; the
// products run in tile_gemm.cuh (few_rows.cuh for a few rows of one weight
// matrix), the element passes in operators.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/moe_b200.h"
#include "common.cuh"
#include "few_rows.cuh"
#include "operators.cuh"
#include "tile_gemm.cuh"

using namespace moe;

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load();
  if (f == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn.store(f = reinterpret_cast<EncodeFn>(p));
  }
  return f;
}

// A 16-bit operand: `inner` contiguous elements per row, `rows` rows of `pitch`
// elements, `batch` such matrices `bs` elements apart.
struct Operand {
  const void* base;
  uint64_t inner, rows, pitch, batch, bs;
};

bool map3(CUtensorMap* m, const Operand& o, uint32_t box_rows, bool f16) {
  EncodeFn enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {o.inner, o.rows, o.batch};
  const cuuint64_t strides[2] = {o.pitch * 2, (o.batch > 1 ? o.bs : o.pitch) * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.base),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool set_maps(TgParams& p, const Operand& P, bool p_mn, const Operand& Q, bool q_mn) {
  const bool h = p.f16 != 0;
  bool ok = map3(&p.tm_p, P, p_mn ? 64 : 128, h);
  if (q_mn) return ok && map3(&p.tm_q[0], Q, 64, h);
  for (int i = 0; i < 4; ++i) ok = ok && map3(&p.tm_q[i], Q, 128u >> i, h);
  return ok;
}

// The output of a product, written piece by piece: 32 x 32 entries, 64-byte rows swizzled as the epilogue lays them.
bool set_out(TgParams& p, void* out, uint64_t cols, uint64_t rows, uint64_t pitch, uint64_t batch, uint64_t bs) {
  EncodeFn enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {cols, rows, batch};
  const cuuint64_t strides[2] = {pitch * 2, (batch > 1 ? bs : pitch) * 2};
  const cuuint32_t box[3] = {32, 32, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  p.out = out;
  p.ldo = (long long)pitch;
  p.out_bs = (long long)bs;
  return enc(&p.tm_out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, out, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

int current_device(int* num_sms) {
  static std::atomic<int> sms[kMaxDevices];
  int d = -1;
  if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) return -1;
  int v = sms[d].load();
  if (v == 0) {
    int major = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d) != cudaSuccess ||
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, d) != cudaSuccess)
      return -1;
    sms[d].store(v = major == 10 ? v : -1);
  }
  *num_sms = v;
  return d;
}

// Stages that fit beside the epilogue's pieces for the largest N tile (`nt`) of a launch.
template <int Mode, int Epi>
int size_stages(TgParams& p, bool q_mn) {
  const int half = p.nt / 2;
  p.stage_bytes = kTgABytes + (q_mn ? (half + 63) / 64 * 8192 : half * 128);
  p.epi_bytes = tg_epi_bytes<Epi>(p.res != nullptr);
  const int table = Mode == kTgRaggedN || Mode == kTgRaggedK ? p.groups : 0;
  p.stages = std::min(kTgMaxStages, (kTgSmemMax - (int)tg_smem_bytes(0, 0, p.epi_bytes, table)) / p.stage_bytes);
  return (int)tg_smem_bytes(p.stages, p.stage_bytes, p.epi_bytes, table);
}

// One launch. `tiles`: output tiles where the host knows them, else 0 (the
// grid then covers every pair of SMs). Launched with programmatic stream
// serialisation: the kernel sets its barriers and TMEM up under the end of the
// stream's previous kernel and waits for it before it reads or writes any
// global memory. Returns a moe_status.
template <int Mode, bool PMn, bool QMn, int Epi, typename T>
int launch(TgParams& p, long long tiles, cudaStream_t st) {
  static std::atomic<int> clusters[kMaxDevices];
  int sms = 0;
  const int d = current_device(&sms);
  if (d < 0) return MOE_ERR_CUDA;
  if (sms < 0) return MOE_ERR_UNSUPPORTED_DEVICE;
  auto kernel = moe_tile_gemm_kernel<Mode, PMn, QMn, Epi, T>;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  cfg.blockDim = dim3(kTgThreads);
  cfg.stream = st;
  cfg.attrs = at;
  int c = clusters[d].load();
  if (c == 0) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTgSmemMax) != cudaSuccess)
      return MOE_ERR_CUDA;
    cfg.gridDim = dim3(2 * (sms / 2));
    cfg.dynamicSmemBytes = kTgSmemMax;
    if (cudaOccupancyMaxActiveClusters(&c, kernel, &cfg) != cudaSuccess || c < 1) return MOE_ERR_CUDA;
    clusters[d].store(c);
  }
  const int bytes = size_stages<Mode, Epi>(p, QMn);
  p.wait_cycles = tg_wait_cycles(p.K);
  cfg.gridDim = dim3(2 * (unsigned)(tiles > 0 && tiles < c ? tiles : c));
  cfg.dynamicSmemBytes = bytes;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// An element pass of 256 threads a block (operators.cuh), launched in the same way.
template <typename P>
int launch_pass(void (*kernel)(P), dim3 grid, const P& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

constexpr int kMaxExtent = 1 << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool operand_ok(const void* p) { return p != nullptr && aligned(p, 16); }
bool pitch_ok(long long ld, int width) { return ld >= width && ld % 8 == 0 && ld < (1ll << 36); }
// K and N of a product: rows of 16-byte multiples; all extents leave room for a tile in 32 bits
bool extents_ok(int K, int N, int rows) {
  return K >= 8 && N >= 8 && K % 8 == 0 && N % 8 == 0 && K <= kMaxExtent && N <= kMaxExtent && rows <= kMaxExtent;
}
bool half_type(int dtype) { return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_FP16; }

int clear_error_word(int32_t* err, cudaStream_t st) {
  if (err != nullptr && cudaMemsetAsync(err, 0, sizeof(int32_t), st) != cudaSuccess) return MOE_ERR_CUDA;
  return MOE_OK;
}

// N tile of a dense product of `rows` N-side rows and mt M tiles on `pairs` CTA
// pairs: the multiple of 32 with the least (rounds of tiles) x (256 + columns of
// a tile that are loaded). A k block's time is its loads, 16 KB of P and 64
// bytes a column of Q in each CTA, rather than its MMAs as soon as a tile is
// below 256 columns; an MN-major Q is loaded in boxes of 64 columns in each CTA.
int pick_tile(long long rows, int mt, int batch, int pairs, bool q_mn) {
  int best = 256;
  long long least = -1;
  for (int nt = 256; nt >= 32; nt -= 32) {
    const long long tiles = (rows + nt - 1) / nt;
    const long long each = ((rows + tiles - 1) / tiles + 31) / 32 * 32;
    const long long loaded = q_mn ? (each + 127) / 128 * 128 : each;
    const long long cost = (tiles * mt * batch + pairs - 1) / pairs * (256 + loaded);
    if (least < 0 || cost < least) {
      least = cost;
      best = (int)each;
    }
  }
  return best;
}

// Largest N tile of a ragged product (a group of fewer rows takes fewer columns
// anyway): 256, and less where the tiles would leave pairs idle, taking every
// group to end in half a tile, with the costs of pick_tile. A smaller limit for
// small groups makes no difference to their time (1 to 64 rows in each of 128
// experts of 2048 x 2048 or 768: within 2 % at 32, 64, 128 and 256, and 6 %
// slower at 32 for 16 and 32 rows) and costs a large group among them its reuse
// (1500 rows among experts of 4: 84 us at 32, 77 at 256).
int ragged_tile(int rows, int groups, int mt, int pairs) {
  int best = 256;
  long long least = -1;
  for (int nt = 256; nt >= 32; nt /= 2) {
    const long long tiles = ((long long)rows / nt + (groups + 1) / 2) * mt;
    const long long cost = (tiles + pairs - 1) / pairs * (256 + nt);
    if (least < 0 || cost < least) {
      least = cost;
      best = nt;
    }
  }
  return best;
}

// Forward products have the layer's epilogue; gradients (a transposed W, a weight gradient) store what they are.
int launch_rows(TgParams& p, bool transpose, int dtype, long long tiles, cudaStream_t st) {
  if (dtype == MOE_DTYPE_FP16)
    return transpose ? launch<kTgRaggedN, false, false, kTgPlain, __half>(p, tiles, st)
                     : launch<kTgRaggedN, true, false, kTgStore, __half>(p, tiles, st);
  return transpose ? launch<kTgRaggedN, false, false, kTgPlain, bf16>(p, tiles, st)
                   : launch<kTgRaggedN, true, false, kTgStore, bf16>(p, tiles, st);
}

int launch_wgrad(TgParams& p, int dtype, long long tiles, cudaStream_t st) {
  return dtype == MOE_DTYPE_FP16 ? launch<kTgRaggedK, true, true, kTgPlain, __half>(p, tiles, st)
                                 : launch<kTgRaggedK, true, true, kTgPlain, bf16>(p, tiles, st);
}

// The cut of a product of few tiles (few_rows.cuh) and its time in microseconds,
// and the time of the same product as whole reductions on CTA pairs
// (tile_gemm.cuh). The figures are fits to measured times of 8 to 160 MB of
// weights at 1 to 768 rows. Single CTAs: a k block (64 k of 128 features) 0.6 us
// when two run on every SM and W comes from HBM, less with fewer down to 0.3, and
// 4.5 us besides (set-up, first load, join), with 7 us more by 128 rows. Pairs: 0.27 us a k block of up to
// 240 columns of a 256-feature tile, and 3 us besides for whole reductions, 5.5
// and 3 more by 128 columns for split ones. Measured, split (the kind taken) /
// whole: 14336 -> 4096 features, 37 rows 25 (single) / 61 us; 4096 -> 14336 24 / 24;
// 2048 -> 40000 43 / 36.
struct FewCut {
  int nt, split;
  bool pair;
  double us;
};
FewCut few_cut(int T, int M, int K, int sms, bool q_mn) {
  const int nt = T <= 32 && !q_mn ? 32 : T <= 64 ? 64 : 128;   // an MN-major Q comes in boxes of 64
  FewCut best{nt, 1, false, 1e30};
  const int nk = (K + 63) / 64;
  const int across = (T + nt - 1) / nt;
  if (across > 65535) return best;   // the grid's second extent
  const long long cells = (long long)((M + 127) / 128) * across;
  for (int c = 1; c <= kFewMaxSplit && c <= std::max(1, nk / 2); ++c) {
    const double rounds = (double)((cells * c + 2 * sms - 1) / (2 * sms));
    const double block = std::max(0.3, 0.6 * std::min(1.0, (double)(cells * c) / (2 * sms)));
    const double us = rounds * ((nk + c - 1) / c * block + 4.5 + 7.0 * std::min(T, 128) / 128);
    if (us < best.us) best.split = c, best.us = us;
  }
  const int wide = (T + 255) / 256, unit = q_mn ? 128 : 32;
  const int each = ((T + wide - 1) / wide + unit - 1) / unit * unit;
  const long long pair_cells = (long long)((M + 255) / 256) * wide;
  for (int c = 2; 2 * c <= kFewMaxSplit && c <= nk / 2; ++c) {
    const int at_once = c == 2 ? sms / 4 - 1 : c == 3 ? sms / 7 : sms / 12;   // clusters: large ones leave SMs of a GPC over
    const double rounds = (double)((pair_cells + at_once - 1) / std::max(1, at_once));
    const double us = rounds * ((nk + c - 1) / c * std::max(0.27, each * 0.0011) + 5.5 + 3.0 * each / 128);
    if (us < best.us) best = FewCut{each, c, true, us};
  }
  return best;
}
double pairs_us(long long tiles, int nt, int K, int pairs) {
  return (double)((tiles + pairs - 1) / pairs) * ((K + 63) / 64 * std::max(0.27, nt * 0.0011) + 3.0);
}

template <bool PMn, bool QMn, bool Pair, typename T>
int launch_few_kind(const TgParams& p, const FewCut& cut, const Operand& P, const Operand& Q, cudaStream_t st) {
  static std::atomic<int> ready[kMaxDevices];
  int d = -1;
  if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) return MOE_ERR_CUDA;
  auto kernel = moe_few_rows_kernel<PMn, QMn, Pair, T>;
  constexpr int most = Pair ? kFewSmemTilesPair : kFewSmemTiles;
  if (!ready[d].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(most + 1024 + sizeof(FewSmem))) != cudaSuccess)
      return MOE_ERR_CUDA;
    ready[d].store(1);
  }
  FewParams f{};
  f.M = p.M;
  f.K = p.K;
  f.T = p.N;
  f.nt = cut.nt;
  f.split = cut.split;
  const int cols = Pair ? f.nt / 2 : f.nt;
  f.stages = std::min(kFewMaxStages, most / few_stage_bytes(cols));
  f.f16 = p.f16;
  f.err = p.err;
  f.wait_cycles = tg_wait_cycles(p.K);
  f.out = p.out;
  f.ldo = p.ldo;
  f.bias = p.bias;
  f.res = p.res;
  f.ldr = p.ldr;
  f.z = p.z;
  f.ldz = p.ldz;
  f.act = p.act;
  if (!map3(&f.tm_w, P, PMn ? 64 : 128, p.f16 != 0) || !map3(&f.tm_x, Q, QMn ? 64 : cols, p.f16 != 0)) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  const int ctas = f.split * (Pair ? 2 : 1);
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  cfg.blockDim = dim3(kFewThreads);
  const int features = Pair ? 256 : 128;
  cfg.gridDim = dim3((p.M + features - 1) / features * ctas, (p.N + f.nt - 1) / f.nt);
  cfg.dynamicSmemBytes = few_smem_bytes(cols, f.stages);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, f) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <bool PMn, bool QMn, typename T>
int launch_few(const TgParams& p, const FewCut& cut, const Operand& P, const Operand& Q, cudaStream_t st) {
  return cut.pair ? launch_few_kind<PMn, QMn, true, T>(p, cut, P, Q, st)
                  : launch_few_kind<PMn, QMn, false, T>(p, cut, P, Q, st);
}

// y = x W (transpose: x W^T) for one or several row groups; epilogue fields of p set by the caller.
int rows_product(TgParams& p, const void* x, long long ldx, const void* W, int rows, int groups, int K, int N,
                 bool transpose, int dtype, void* y, long long ldy, cudaStream_t st) {
  int sms = 0;
  if (current_device(&sms) < 0) return MOE_ERR_CUDA;
  p.M = N;
  p.N = rows;
  p.K = K;
  p.groups = groups;
  p.f16 = dtype == MOE_DTYPE_FP16;
  const int mt = (N + 255) / 256;
  long long tiles = 0;
  if (p.offsets == nullptr) {
    p.nt = pick_tile(rows, mt, 1, std::max(1, sms / 2), false);
    tiles = (long long)((rows + p.nt - 1) / p.nt) * mt;
  } else {
    p.nt = ragged_tile(rows, groups, mt, std::max(1, sms / 2));
  }
  if (((long long)rows / 32 + groups) * mt >= (1ll << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const Operand P = transpose ? Operand{W, (uint64_t)K, (uint64_t)N, (uint64_t)K, (uint64_t)groups, (uint64_t)K * N}
                              : Operand{W, (uint64_t)N, (uint64_t)K, (uint64_t)N, (uint64_t)groups, (uint64_t)K * N};
  const Operand Q{x, (uint64_t)K, (uint64_t)rows, (uint64_t)ldx, 1, 0};
  if (p.offsets == nullptr) {
    if (sms < 0) return MOE_ERR_UNSUPPORTED_DEVICE;
    const FewCut cut = few_cut(rows, N, K, sms, false);
    p.out = y;
    p.ldo = ldy;
    if (cut.us < pairs_us(tiles, p.nt, K, std::max(1, sms / 2))) {
      if (dtype == MOE_DTYPE_FP16)
        return transpose ? launch_few<false, false, __half>(p, cut, P, Q, st)
                         : launch_few<true, false, __half>(p, cut, P, Q, st);
      return transpose ? launch_few<false, false, bf16>(p, cut, P, Q, st) : launch_few<true, false, bf16>(p, cut, P, Q, st);
    }
  }
  if (!set_maps(p, P, !transpose, Q, false) || !set_out(p, y, N, rows, ldy, 1, 0)) return MOE_ERR_CUDA;
  return launch_rows(p, transpose, dtype, tiles, st);
}

// dW[g] = x_g^T dy_g
int weight_gradient(TgParams& p, const void* x, long long ldx, const void* dy, long long lddy, int rows, int groups,
                    int K, int N, int dtype, void* dW, cudaStream_t st) {
  int sms = 0;
  if (current_device(&sms) < 0) return MOE_ERR_CUDA;
  p.M = N;
  p.N = K;
  p.K = rows;
  p.groups = groups;
  p.f16 = dtype == MOE_DTYPE_FP16;
  const int mt = (N + 255) / 256;
  p.nt = pick_tile(K, mt, groups, std::max(1, sms / 2), true);
  const long long tiles = (long long)((K + p.nt - 1) / p.nt) * mt * groups;
  if (tiles >= (1ll << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const Operand P{dy, (uint64_t)N, (uint64_t)rows, (uint64_t)lddy, 1, 0};
  const Operand Q{x, (uint64_t)K, (uint64_t)rows, (uint64_t)ldx, 1, 0};
  if (p.offsets == nullptr) {   // few tiles: the reduction over the rows is split
    if (sms < 0) return MOE_ERR_UNSUPPORTED_DEVICE;
    const FewCut cut = few_cut(K, N, rows, sms, true);
    if (cut.us < pairs_us(tiles, p.nt, rows, std::max(1, sms / 2))) {
      p.out = dW;
      p.ldo = N;
      p.N = K;
      p.K = rows;
      return dtype == MOE_DTYPE_FP16 ? launch_few<true, true, __half>(p, cut, P, Q, st)
                                     : launch_few<true, true, bf16>(p, cut, P, Q, st);
    }
  }
  if (!set_maps(p, P, true, Q, true) || !set_out(p, dW, N, K, N, groups, (uint64_t)K * N)) return MOE_ERR_CUDA;
  return launch_wgrad(p, dtype, tiles, st);
}

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// ---- linear_backward workspace: dz [T, N] and the bias gradient's partial sums
int bias_chunks(int T) { return std::min(128, (T + kActRows - 1) / kActRows); }
size_t dz_bytes(int T, int N) { return up((size_t)T * N * 2, 256); }

// ---- orthogonalize workspace
struct OrthoLayout {
  size_t x[2], lo, a, b, partial, alpha, total;
  long long ldx, lda, bsx, bsa, bsl;
};
OrthoLayout ortho_layout(int batch, int m, int n) {
  OrthoLayout L{};
  const int p = std::min(m, n);   // X is kept with the long side contiguous
  L.ldx = (long long)up(std::max(m, n), 64);
  L.lda = (long long)up(p, 64);
  L.bsx = L.ldx * p;
  L.bsa = L.lda * p;
  L.bsl = L.ldx * (long long)up(p, 32);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up(bytes, 256);
    return at;
  };
  L.x[0] = take((size_t)batch * L.bsx * 2);
  L.x[1] = take((size_t)batch * L.bsx * 2);
  L.lo = take((size_t)batch * L.bsl);
  L.a = take((size_t)batch * L.bsa * 2);
  L.b = take((size_t)batch * L.bsa * 2);
  L.partial = take((size_t)batch * kOrthoChunks * 8);
  L.alpha = take((size_t)batch * 4);
  L.total = o;
  return L;
}

}  // namespace

extern "C" int moe_grouped_matmul(const void* x, long long ldx, const void* W, const int32_t* offsets, int rows,
                                  int groups, int K, int N, int transpose, int dtype, void* y, long long ldy,
                                  int32_t* error_word, void* stream) {
  if (rows < 0 || groups < 1 || !half_type(dtype) || !aligned(error_word, 4)) return MOE_ERR_INVALID_ARG;
  if (!extents_ok(K, N, rows) || groups > kTgMaxGroups) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!pitch_ok(ldx, K) || !pitch_ok(ldy, N)) return MOE_ERR_INVALID_ARG;
  if (offsets == nullptr || !aligned(offsets, 4) || !operand_ok(W)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!operand_ok(x) || !operand_ok(y))) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  (void)cudaGetLastError();
  if (int rc = clear_error_word(error_word, st)) return rc;
  if (rows == 0) return MOE_OK;
  TgParams p{};
  p.offsets = offsets;
  p.err = error_word;
  return rows_product(p, x, ldx, W, rows, groups, K, N, transpose != 0, dtype, y, ldy, st);
}

extern "C" int moe_grouped_matmul_wgrad(const void* x, long long ldx, const void* dy, long long lddy,
                                        const int32_t* offsets, int rows, int groups, int K, int N, int dtype, void* dW,
                                        int32_t* error_word, void* stream) {
  if (rows < 0 || groups < 1 || !half_type(dtype) || !aligned(error_word, 4)) return MOE_ERR_INVALID_ARG;
  if (!extents_ok(K, N, rows) || groups > kTgMaxGroups) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!pitch_ok(ldx, K) || !pitch_ok(lddy, N)) return MOE_ERR_INVALID_ARG;
  if (offsets == nullptr || !aligned(offsets, 4) || !operand_ok(dW)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!operand_ok(x) || !operand_ok(dy))) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  (void)cudaGetLastError();
  if (int rc = clear_error_word(error_word, st)) return rc;
  if (rows == 0)
    return cudaMemsetAsync(dW, 0, (size_t)groups * K * N * 2, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  TgParams p{};
  p.offsets = offsets;
  p.err = error_word;
  return weight_gradient(p, x, ldx, dy, lddy, rows, groups, K, N, dtype, dW, st);
}

extern "C" int moe_linear(const void* x, long long ldx, const void* W, const void* bias, const void* residual,
                          long long ldr, int T, int K, int N, int activation, int dtype, void* y, long long ldy,
                          void* preact, long long ldz, int32_t* error_word, void* stream) {
  if (T < 0 || !half_type(dtype) || activation < MOE_ACT_NONE || activation > MOE_ACT_SILU || !aligned(error_word, 4))
    return MOE_ERR_INVALID_ARG;
  if (!extents_ok(K, N, T)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!pitch_ok(ldx, K) || !pitch_ok(ldy, N)) return MOE_ERR_INVALID_ARG;
  if (!operand_ok(W) || !aligned(bias, 16)) return MOE_ERR_INVALID_ARG;
  if (residual != nullptr && (!aligned(residual, 16) || !pitch_ok(ldr, N))) return MOE_ERR_INVALID_ARG;
  if (preact != nullptr && (!aligned(preact, 16) || !pitch_ok(ldz, N))) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!operand_ok(x) || !operand_ok(y))) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  (void)cudaGetLastError();
  if (int rc = clear_error_word(error_word, st)) return rc;
  if (T == 0) return MOE_OK;
  TgParams p{};
  p.err = error_word;
  p.bias = bias;
  p.res = residual;
  p.ldr = ldr;
  p.z = preact;
  p.ldz = ldz;
  p.act = activation;
  return rows_product(p, x, ldx, W, T, 1, K, N, false, dtype, y, ldy, st);
}

extern "C" size_t moe_linear_backward_workspace_bytes(int T, int N, int activation, int bias_grad) {
  if (T < 1 || N < 1) return 0;
  return (activation != MOE_ACT_NONE ? dz_bytes(T, N) : 0) + (bias_grad ? (size_t)bias_chunks(T) * N * 4 : 0);
}

extern "C" int moe_linear_backward(const void* dy, long long lddy, const void* x, long long ldx, const void* W,
                                   const void* preact, long long ldz, int T, int K, int N, int activation, int dtype,
                                   void* dx, long long lddx, void* dW, void* dbias, void* workspace,
                                   size_t workspace_bytes, int32_t* error_word, void* stream) {
  if (T < 0 || !half_type(dtype) || activation < MOE_ACT_NONE || activation > MOE_ACT_SILU || !aligned(error_word, 4))
    return MOE_ERR_INVALID_ARG;
  if (!extents_ok(K, N, T)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const bool act = activation != MOE_ACT_NONE;
  if (!pitch_ok(lddy, N) || (act && !pitch_ok(ldz, N))) return MOE_ERR_INVALID_ARG;
  if (dx != nullptr && (!pitch_ok(lddx, K) || !aligned(dx, 16) || !operand_ok(W))) return MOE_ERR_INVALID_ARG;
  if (dW != nullptr && (!pitch_ok(ldx, K) || !aligned(dW, 16))) return MOE_ERR_INVALID_ARG;
  if (!aligned(dbias, 16)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!operand_ok(dy) || (act && !operand_ok(preact)) || (dW != nullptr && !operand_ok(x))))
    return MOE_ERR_INVALID_ARG;
  const size_t need = moe_linear_backward_workspace_bytes(T, N, activation, dbias != nullptr);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 256))) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  (void)cudaGetLastError();
  if (int rc = clear_error_word(error_word, st)) return rc;
  if (T == 0) {
    if (dW != nullptr && cudaMemsetAsync(dW, 0, (size_t)K * N * 2, st) != cudaSuccess) return MOE_ERR_CUDA;
    if (dbias != nullptr && cudaMemsetAsync(dbias, 0, (size_t)N * 2, st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  void* dz = act ? workspace : const_cast<void*>(dy);
  const long long lddz = act ? N : lddy;
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + (act ? dz_bytes(T, N) : 0));
  if (act || dbias != nullptr) {
    const int chunks = bias_chunks(T);
    ActParams a{dy, lddy, preact, ldz, act ? dz : nullptr, dbias ? partial : nullptr, dbias, T, N,
                (T + chunks - 1) / chunks, chunks, activation};
    const bool h = dtype == MOE_DTYPE_FP16;
    if (int rc = launch_pass(h ? moe_act_backward_kernel<__half> : moe_act_backward_kernel<bf16>,
                             dim3((N + kActCols - 1) / kActCols, chunks), a, st))
      return rc;
    if (dbias != nullptr)
      if (int rc = launch_pass(h ? moe_bias_sum_kernel<__half> : moe_bias_sum_kernel<bf16>, dim3((N + 31) / 32), a, st))
        return rc;
  }
  if (dx != nullptr) {
    TgParams p{};
    p.err = error_word;
    if (int rc = rows_product(p, dz, lddz, W, T, 1, N, K, true, dtype, dx, lddx, st)) return rc;
  }
  if (dW != nullptr) {
    TgParams p{};
    p.err = error_word;
    if (int rc = weight_gradient(p, x, ldx, dz, lddz, T, 1, K, N, dtype, dW, st)) return rc;
  }
  return MOE_OK;
}

extern "C" size_t moe_orthogonalize_workspace_bytes(int batch, int m, int n) {
  return batch < 1 || m < 1 || n < 1 ? 0 : ortho_layout(batch, m, n).total;
}

extern "C" int moe_orthogonalize(const void* G, long long ldg, long long bsg, int batch, int m, int n, int dtype,
                                 int steps, const float* coeffs, float eps, void* out, long long ldo, long long bso,
                                 void* workspace, size_t workspace_bytes, int32_t* error_word, void* stream) {
  const int elem = dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (batch < 0 || m < 1 || n < 1 || (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP32) || coeffs == nullptr ||
      !(eps >= 0.f) || !aligned(error_word, 4))
    return MOE_ERR_INVALID_ARG;
  if (steps < 1 || steps > 64 || std::max(m, n) > (1 << 16) || batch > 65535) return MOE_ERR_UNSUPPORTED_SHAPE;
  constexpr long long kMost = 1ll << 40;   // pitches, so that their products stay in 64 bits
  if (ldg < n || ldo < n || ldg > kMost || ldo > kMost || (batch > 1 && (bsg < ldg * (m - 1) + n || bso < ldo * (m - 1) + n)))
    return MOE_ERR_INVALID_ARG;
  if (batch > 0 && (G == nullptr || out == nullptr || !aligned(G, elem) || !aligned(out, 2))) return MOE_ERR_INVALID_ARG;
  const OrthoLayout L = ortho_layout(std::max(batch, 1), m, n);
  if (batch > 0 && (workspace == nullptr || !aligned(workspace, 256))) return MOE_ERR_INVALID_ARG;
  if (batch > 0 && workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  (void)cudaGetLastError();
  if (int rc = clear_error_word(error_word, st)) return rc;
  if (batch == 0) return MOE_OK;
  int sms = 0;
  if (current_device(&sms) < 0) return MOE_ERR_CUDA;
  const int pairs = std::max(1, sms / 2);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool tall = m > n;
  const int p0 = std::min(m, n), q0 = std::max(m, n);
  // X is stored times 2^13 and A and B times 2^10. Every entry of X is at most the root of A's largest, so both
  // leave fp16's range together, at 8 and 64; and X's entries are normal fp16 numbers down to 2^-27 (times
  // sqrt(q) alone, the size of an orthogonal matrix's entries, a row a millionth of the others' size came out
  // with an error of 2e-2 after the dozen steps that bring it up).
  const float xs = 8192.f, as = 1024.f;

  const bool fp32 = dtype == MOE_DTYPE_FP32;
  OrthoParams o{G, ldg, bsg, m, n, tall ? 1 : 0, xs, eps, reinterpret_cast<double*>(ws + L.partial),
                reinterpret_cast<float*>(ws + L.alpha), reinterpret_cast<__half*>(ws + L.x[0]),
                fp32 ? ws + L.lo : nullptr, L.ldx, L.bsx,
                L.bsl, 0};
  // blocks of 4096 entries or more, some sixteen to an SM over the batch
  o.chunks = (int)std::min<long long>({(long long)kOrthoChunks, ((long long)m * n + 4095) / 4096,
                                       std::max(1ll, (16ll * sms + batch - 1) / batch)});
  const dim3 grid(o.chunks, batch);
  if (int rc = launch_pass(fp32 ? moe_ortho_norm_kernel<float> : moe_ortho_norm_kernel<bf16>, grid, o, st)) return rc;
  if (int rc = launch_pass(fp32 ? moe_ortho_scale_pieces_kernel<float>
                           : tall ? moe_ortho_scale_pieces_kernel<bf16>
                                  : moe_ortho_scale_bf16_kernel,
                           grid, o, st))
    return rc;

  const Operand A{ws + L.a, (uint64_t)p0, (uint64_t)p0, (uint64_t)L.lda, (uint64_t)batch, (uint64_t)L.bsa};
  const Operand B{ws + L.b, (uint64_t)p0, (uint64_t)p0, (uint64_t)L.lda, (uint64_t)batch, (uint64_t)L.bsa};
  TgParams base{};
  base.err = error_word;
  base.f16 = 1;
  base.groups = batch;
  auto operand_x = [&](int k) {
    return Operand{ws + L.x[k], (uint64_t)q0, (uint64_t)p0, (uint64_t)L.ldx, (uint64_t)batch, (uint64_t)L.bsx};
  };
  // A = X X^T, from X in buffer k
  auto gram = [&](int k, TgParams& g) {
    const Operand X = operand_x(k);
    g = base;
    g.M = g.N = p0;
    g.K = q0;
    g.nt = 256;
    g.factors.cb = as / (xs * xs);
    g.backwards = 1;   // from the batches that the step before wrote last, which L2 still holds
    return set_maps(g, X, false, X, false) && set_out(g, ws + L.a, p0, p0, L.lda, batch, L.bsa);
  };
  // B = b A + c A A
  auto poly = [&](TgParams& g) {
    g = base;
    g.M = g.N = g.K = p0;
    g.nt = 256;
    g.in = reinterpret_cast<const __half*>(ws + L.a);
    g.ldi = L.lda;
    g.in_bs = L.bsa;
    return set_maps(g, A, false, A, false) && set_out(g, ws + L.b, p0, p0, L.lda, batch, L.bsa);
  };
  // X' = a X + B X, from buffer k to the other (last: to the caller, a tall matrix back in its own order):
  // rows of X on the N side, columns on the M side, X'[r, c] = sum_k X[k, c] B[r, k]
  auto update = [&](int k, bool last, TgParams& g) {
    const Operand X = operand_x(k);
    g = base;
    g.M = q0;
    g.N = g.K = p0;
    g.nt = pick_tile(p0, (q0 + 255) / 256, batch, pairs, false);
    g.in = reinterpret_cast<const __half*>(ws + L.x[k]);
    g.lo_out = ws + L.lo;
    g.lo_bs = L.bsl;
    g.ldi = L.ldx;
    g.in_bs = L.bsx;
    if (last) {   // any alignment: no TMA store
      g.out = out;
      g.ldo = ldo;
      g.out_bs = bso;
      g.transposed = tall ? 1 : 0;
    } else if (!set_out(g, ws + L.x[k ^ 1], q0, p0, L.ldx, batch, L.bsx)) {
      return false;
    }
    return set_maps(g, X, true, B, false);
  };
  const uint8_t* lo_first = fp32 ? ws + L.lo : nullptr;   // a scaled bf16 gradient needs none
  // the symmetric products: half of the 256 x 256 tiles, stored twice; or, where these would leave most
  // pairs idle, all tiles of a width that fills them (with the costs of pick_tile)
  const int mt = (p0 + 255) / 256;
  const long long tri = (long long)batch * mt * (mt + 1) / 2;
  const int all_nt = pick_tile(p0, mt, batch, pairs, false);
  const long long all = (long long)((p0 + all_nt - 1) / all_nt) * mt * batch;
  const bool half = (tri + pairs - 1) / pairs * (256 + 256) <= (all + pairs - 1) / pairs * (256 + all_nt);
  TgParams g1[2], g2, g3[2], g4;
  if (!gram(0, g1[0]) || !gram(1, g1[1]) || !poly(g2) || !update(0, false, g3[0]) || !update(1, false, g3[1]) ||
      !update((steps - 1) & 1, true, g4))
    return MOE_ERR_CUDA;
  const long long tiles = (long long)((p0 + g4.nt - 1) / g4.nt) * ((q0 + 255) / 256) * batch;
  if (tri >= (1ll << 30) || tiles >= (1ll << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
  // B is stored less a multiple d of the identity, X' = (a + d) X + (B - d I) X: once the singular values are
  // near 1, B's eigenvalues lie within a few tenths of b + c = -2.7, and the fp16 roundings of B and X enter X'
  // times what is left of B. d is B's eigenvalue at a singular value that is followed through the steps (a
  // guess: any d is exact up to rounding). Too large a guess costs the directions that are still small: their B
  // is near 0, and a rounding of X as a whole enters them times d. So it starts at a tenth of the root mean
  // square 1 / sqrt(p), or at 1 / p where that is more (p = 1: 1 itself). Errors against 64 bits of a 28 x 1835
  // matrix: without d 2.2e-3 (bf16's own rounding is 1.65e-3), from the root mean square 1.9e-3, from here
  // 1.8e-3; of one direction a thousand times the others, 20 x 30: 1.7e-3, 6.3e-3, 2.3e-3.
  double sigma = std::max(0.1, 1.0 / std::sqrt((double)p0)) / std::sqrt((double)p0);
  for (int i = 0; i < steps; ++i) {
    const double ca = coeffs[3 * i], cb = coeffs[3 * i + 1], cc = coeffs[3 * i + 2];
    const double t = std::min(1.0, sigma * sigma);
    const float d = (float)(cb * t + cc * t * t);
    sigma = std::fabs(sigma * (ca + cb * sigma * sigma + cc * sigma * sigma * sigma * sigma));
    const bool last = i == steps - 1;
    const float* alpha = i == 0 ? o.alpha : nullptr;
    TgParams& a = g1[i & 1];
    a.factors.alpha = alpha;
    g2.factors = TgFactors{coeffs[3 * i + 1], coeffs[3 * i + 2] / as, nullptr, nullptr, -d * as};
    int rc;
    if (half) {
      rc = launch<kTgSymmetric, false, false, kTgGram, __half>(a, tri, st);
      if (rc == MOE_OK) rc = launch<kTgSymmetric, false, false, kTgPoly, __half>(g2, tri, st);
    } else {
      a.nt = g2.nt = all_nt;
      rc = launch<kTgBatched, false, false, kTgGram, __half>(a, all, st);
      if (rc == MOE_OK) rc = launch<kTgBatched, false, false, kTgPoly, __half>(g2, all, st);
    }
    if (rc) return rc;
    TgParams& x = last ? g4 : g3[i & 1];
    const float back = last ? 1.f / xs : 1.f;
    x.factors = TgFactors{(coeffs[3 * i] + d) * back, back / as, alpha, i == 0 ? lo_first : ws + L.lo, 0.f};
    rc = last ? launch<kTgBatched, true, false, kTgUpdateOut, __half>(x, tiles, st)
              : launch<kTgBatched, true, false, kTgUpdate, __half>(x, tiles, st);
    if (rc) return rc;
  }
  return MOE_OK;
}
