// Element passes of the operators around the MoE layer: the activation's
// backward with the bias gradient's sums, and the normalisation that opens the
// Newton-Schulz iteration. All are one read and one write of their tensors,
// bound by HBM; sums are fp32 (fp64 for the norm) in a fixed order, so a result
// does not depend on timing.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "common.cuh"
#include "tile_gemm.cuh"

namespace moe {

constexpr int kActCols = 256;   // columns of a block: 32 lanes x 8
constexpr int kActRows = 32;    // least rows of a block's chunk
constexpr int kOrthoChunks = 256;

struct ActParams {
  const void* dy;
  long long lddy;
  const void* z;
  long long ldz;
  void* dz;          // [T, N], or null (no activation: dz is dy)
  float* partial;    // [chunks, N], or null
  void* dbias;       // [N]
  int T, N, rows, chunks, act;
};

// d act(z) / dz
template <int Act>
__device__ __forceinline__ float act_slope(float z) {
  if (Act == kActRelu) return z > 0.f ? 1.f : 0.f;
  if (Act == kActGelu) {
    float density;
    const float phi = tg_normal(z, density);
    return fmaf(z, density, phi);
  }
  if (Act == kActGeluTanh) {
    // q(v) + z q (1 - q) v'(z). z q (1 - q) is formed first and v' bounded (from |z| = 473 on, long after
    // q is 0 or 1): a zero then never meets an infinity, however large z is
    const float w = fminf(0.044715f * z * z, 1e4f);
    float slope;
    const float q = tg_sigmoid(1.59576912160573071f * fmaf(w, z, z), slope);
    return fmaf(slope * z, 1.59576912160573071f * fmaf(3.f, w, 1.f), q);
  }
  if (Act == kActSilu) {
    float slope;
    const float q = tg_sigmoid(z, slope);
    return fmaf(z, slope, q);
  }
  return 1.f;
}

// dz = dy act'(z), rounded once to the operand type of the two products that
// read it (half the width of an fp32 dz, and the tensor cores take no other), and
// this chunk's column sums of the unrounded dz. 4093 x 7168 with the erf slope:
// 38 us for 176 MB (4.6 TB/s), 29 with relu.
template <int Act, typename T>
__device__ __forceinline__ void act_rows(const ActParams& p, int col, int first, int last, float (&acc)[8]) {
  const T* dy = reinterpret_cast<const T*>(p.dy);
  const T* z = reinterpret_cast<const T*>(p.z);
  T* dz = reinterpret_cast<T*>(p.dz);
#pragma unroll 2
  for (int r = first; r < last; r += 8) {
    const uint4 g = *reinterpret_cast<const uint4*>(dy + (long long)r * p.lddy + col);
    uint4 v = g;
    if (Act != kActNone) v = *reinterpret_cast<const uint4*>(z + (long long)r * p.ldz + col);
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, zw[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 d = TgPair<T>::unpack(gw[i]);
      if (Act != kActNone) {
        const float2 zf = TgPair<T>::unpack(zw[i]);
        d.x *= act_slope<Act>(zf.x);
        d.y *= act_slope<Act>(zf.y);
      }
      acc[2 * i] += d.x;
      acc[2 * i + 1] += d.y;
      o[i] = TgPair<T>::pack(d.x, d.y);
    }
    if (Act != kActNone) *reinterpret_cast<uint4*>(dz + (long long)r * p.N + col) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) moe_act_backward_kernel(const ActParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tg_after_stream();
  __shared__ float sums[8][kActCols];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = blockIdx.x * kActCols + tx * 8;
  const int r0 = blockIdx.y * p.rows + ty, r1 = min(p.T, (int)(blockIdx.y + 1) * p.rows);
  float acc[8] = {};
  if (col < p.N) {   // N is a multiple of 8
    switch (p.act) {
      case kActRelu: act_rows<kActRelu, T>(p, col, r0, r1, acc); break;
      case kActGelu: act_rows<kActGelu, T>(p, col, r0, r1, acc); break;
      case kActGeluTanh: act_rows<kActGeluTanh, T>(p, col, r0, r1, acc); break;
      case kActSilu: act_rows<kActSilu, T>(p, col, r0, r1, acc); break;
      default: act_rows<kActNone, T>(p, col, r0, r1, acc);
    }
  }
  if (p.partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[ty][tx * 8 + i] = acc[i];
  __syncthreads();
  const int c = blockIdx.x * kActCols + threadIdx.x;
  if (c < p.N) {
    float v = 0.f;
#pragma unroll
    for (int y = 0; y < 8; ++y) v += sums[y][threadIdx.x];
    p.partial[(long long)blockIdx.y * p.N + c] = v;
  }
}

// 32 columns a block, the chunks' sums over 8 warps.
template <typename T>
__global__ void __launch_bounds__(256) moe_bias_sum_kernel(const ActParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tg_after_stream();
  __shared__ float sums[8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float v = 0.f;
  if (c < p.N) {
#pragma unroll 4
    for (int i = ty; i < p.chunks; i += 8) v += p.partial[(long long)i * p.N + c];
  }
  sums[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < p.N) {
#pragma unroll
    for (int y = 1; y < 8; ++y) v += sums[y][tx];
    reinterpret_cast<T*>(p.dbias)[c] = T(v);
  }
}

// ---------------------------------------------------------------- orthogonalize
struct OrthoParams {
  const void* g;
  long long ldg, bsg;
  int m, n;
  int tall;          // m > n: X is G^T, its rows the short side
  float xs, eps;
  double* partial;   // [batch, kOrthoChunks]
  float* alpha;      // [batch]
  __half* hi;
  uint8_t* lo;       // fp32 gradients, in pieces (tg_low_at's order), or null
  long long ldx, bsx, lo_bs;
  int chunks;
};

template <typename T>
__device__ __forceinline__ float ortho_value(const T* p) { return (float)*p; }

// Threads of a block along a row (the rest along rows): enough for the row, 32 at least.
__device__ __forceinline__ int ortho_lanes(int items) { return items > 128 ? 256 : items > 64 ? 128 : items > 32 ? 64 : 32; }

template <typename F>
__device__ __forceinline__ double block_sum(double v, F* scratch) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += scratch[i];
  return s;
}

// Eight elements where every row starts on 16 bytes, else one at a time.
template <typename T>
__device__ __forceinline__ bool ortho_wide(const OrthoParams& p) {
  return p.n % 8 == 0 && p.ldg % 8 == 0 && p.bsg % 8 == 0 && (reinterpret_cast<uintptr_t>(p.g) & 15) == 0;
}
template <typename T>
__device__ __forceinline__ void ortho_load8(const T* p, float (&v)[8]) {
  if (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = TgPair<bf16>::unpack(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// Squares summed in fp64: neither a large fp32 gradient overflows nor a small one
// vanishes. 64 matrices of 2048 x 768 in bf16 (201 MB): 50 us.
template <typename T>
__global__ void __launch_bounds__(256) moe_ortho_norm_kernel(const OrthoParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tg_after_stream();
  __shared__ double scratch[8];
  const T* g = reinterpret_cast<const T*>(p.g) + blockIdx.y * p.bsg;
  const bool wide = ortho_wide<T>(p);
  const int items = wide ? p.n / 8 : p.n;
  const int lanes = ortho_lanes(items);
  const int tx = threadIdx.x & (lanes - 1), ty = threadIdx.x / lanes, rows = 256 / lanes;
  double acc = 0;
  for (int r = blockIdx.x * rows + ty; r < p.m; r += gridDim.x * rows) {
    const T* row = g + (long long)r * p.ldg;
    if (wide) {
#pragma unroll 4
      for (int c = tx; c < items; c += lanes) {
        float v[8];
        ortho_load8(row + c * 8, v);
        float s8 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s8 = fmaf(v[i], v[i], s8);
        if (s8 > 1e-30f && s8 < 1e37f) {   // eight squares in fp32 where they stay normal numbers
          acc += s8;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc += (double)v[i] * v[i];
        }
      }
    } else {
#pragma unroll 4
      for (int c = tx; c < items; c += lanes) {
        const double v = ortho_value(row + c);
        acc += v * v;
      }
    }
  }
  const double s = block_sum(acc, scratch);
  if (threadIdx.x == 0) p.partial[blockIdx.y * kOrthoChunks + blockIdx.x] = s;
}

// X0 = G / (|G| + eps) as two factors: G times a power of two, which brings the norm to 2^13 .. 2^14 (a bf16
// entry is exact in fp16 down to 2^-30 of the norm, an fp32 one has 8 bits more down to 2^-27), and alpha =
// 2^E / (|G| + eps), which the first step's epilogues apply in fp32.
__device__ __forceinline__ double ortho_scale(const OrthoParams& p, double* scratch) {
  const double total =
      block_sum(threadIdx.x < p.chunks ? p.partial[blockIdx.y * kOrthoChunks + threadIdx.x] : 0.0, scratch);
  const double norm = sqrt(total);
  const int e = norm > 0 && norm < 1e300 ? ilogb(norm) : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0)
    p.alpha[blockIdx.y] = norm > 0 ? (float)(ldexp(1.0, e) / (norm + p.eps)) : norm == 0 ? 0.f : (float)norm;
  return ldexp((double)p.xs, -e);
}

__global__ void __launch_bounds__(256) moe_ortho_scale_bf16_kernel(const OrthoParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tg_after_stream();
  __shared__ double scratch[8];
  const double scale = ortho_scale(p, scratch);
  const bf16* g = reinterpret_cast<const bf16*>(p.g) + blockIdx.y * p.bsg;
  __half* hi = p.hi + blockIdx.y * p.bsx;
  const bool wide = ortho_wide<bf16>(p);
  const int items = wide ? p.n / 8 : p.n;
  const int lanes = ortho_lanes(items);
  const int tx = threadIdx.x & (lanes - 1), ty = threadIdx.x / lanes, rows = 256 / lanes;
  for (int r = blockIdx.x * rows + ty; r < p.m; r += gridDim.x * rows) {
    const bf16* row = g + (long long)r * p.ldg;
    if (wide) {
#pragma unroll 4
      for (int c = tx; c < items; c += lanes) {
        float v[8];
        ortho_load8(row + c * 8, v);
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = TgPair<__half>::pack((float)(v[2 * i] * scale), (float)(v[2 * i + 1] * scale));
        *reinterpret_cast<uint4*>(hi + (long long)r * p.ldx + c * 8) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    } else {
#pragma unroll 4
      for (int c = tx; c < items; c += lanes)
        hi[(long long)r * p.ldx + c] = __float2half_rn((float)(ortho_value(row + c) * scale));
    }
  }
}

// Two neighbouring entries of a row, the second zero past its end.
__device__ __forceinline__ float2 ortho_pair(const float* p, bool second) { return make_float2(p[0], second ? p[1] : 0.f); }
__device__ __forceinline__ float2 ortho_pair(const bf16* p, bool second) {
  if (second && (reinterpret_cast<uintptr_t>(p) & 3) == 0)
    return TgPair<bf16>::unpack(*reinterpret_cast<const uint32_t*>(p));
  return make_float2((float)p[0], second ? (float)p[1] : 0.f);
}

// fp32 gradients, and tall ones, which are transposed on the way: a warp turns
// 32 x 32 pieces of X into the update epilogue's order. 64 tall matrices of 2048 x
// 768 in bf16: 88 us for 403 MB (one entry at a time instead of 16-byte vectors
// and ldmatrix 209 us; without the transposition 80 us).
template <typename T>
__global__ void __launch_bounds__(256) moe_ortho_scale_pieces_kernel(const OrthoParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tg_after_stream();
  __shared__ double scratch[8];
  __shared__ __align__(128) uint8_t stage[8][kTgPiece];
  const double scale = ortho_scale(p, scratch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t piece = ptx::smem_u32(stage[warp]);
  const T* g = reinterpret_cast<const T*>(p.g) + blockIdx.y * p.bsg;
  __half* hi = p.hi + blockIdx.y * p.bsx;
  const int rows = p.tall ? p.n : p.m, cols = p.tall ? p.m : p.n;   // of X
  const bool vectors = sizeof(T) == 2 && p.tall && ortho_wide<T>(p);
  const int across = (cols + 31) / 32, pieces = across * ((rows + 31) / 32);
  for (int at = blockIdx.x * 8 + warp; at < pieces; at += gridDim.x * 8) {
    const int r0 = at / across * 32, c0 = (at - at / across * across) * 32;
    float2 f[16];
    if (vectors) {   // rows of G as 16-byte vectors, turned by ldmatrix
      const int c = lane & 3;
      uint4 raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = c0 + 8 * i + (lane >> 2), row = r0 + 8 * c;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (col < cols && row < rows) raw[i] = *reinterpret_cast<const uint4*>(g + (long long)col * p.ldg + row);
      }
      __syncwarp();   // every lane has read the piece before
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(stage[warp] + tg_piece_at(8 * i + (lane >> 2), c)) = raw[i];
      __syncwarp();
      uint32_t v[16];
      tg_piece_get<kRowsM>(piece, v, lane);
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = TgPair<bf16>::unpack(v[j]);
    }
    // 8 x 8 block j (row block j / 4, column block j % 4): two rows, one column of X
    const int row0 = r0 + 2 * (lane & 3), col0 = c0 + (lane >> 2);
    if (!vectors && p.tall) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int row = row0 + 8 * (j >> 2), col = col0 + 8 * (j & 3);
        f[j] = make_float2(0.f, 0.f);
        if (col < cols && row < rows) f[j] = ortho_pair(g + (long long)col * p.ldg + row, row + 1 < rows);
      }
    } else if (!vectors) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int row = row0 + 8 * (j >> 2), col = col0 + 8 * (j & 3);
        f[j] = make_float2(0.f, 0.f);
        if (col < cols && row < rows) f[j].x = ortho_value(g + (long long)row * p.ldg + col);
        if (col < cols && row + 1 < rows) f[j].y = ortho_value(g + (long long)(row + 1) * p.ldg + col);
      }
    }
    uint32_t v[16], w[8];
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      int q[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = (float)(f[j + h].x * scale), y = (float)(f[j + h].y * scale);
        v[j + h] = TgPair<__half>::pack(x, y);
        const float2 n = TgPair<__half>::unpack(v[j + h]);
        q[2 * h] = tg_low(x, n.x);
        q[2 * h + 1] = tg_low(y, n.y);
      }
      w[j >> 1] = tg_low4(q[0], q[1], q[2], q[3]);
    }
    if (p.lo != nullptr) {
      uint4* out = reinterpret_cast<uint4*>(p.lo + blockIdx.y * p.lo_bs +
                                            ((long long)(r0 >> 5) * (p.ldx >> 5) + (c0 >> 5)) * 1024 + lane * 32);
      out[0] = make_uint4(w[0], w[1], w[2], w[3]);
      out[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    __syncwarp();
    tg_piece_put<kRowsN>(piece, v, lane);
    __syncwarp();
    tg_piece_out(piece, hi + (long long)r0 * p.ldx + c0, p.ldx, rows - r0, 32, lane);
  }
}

}  // namespace moe
