// Products of few tiles: y = act(x W + bias) + residual for few rows of x
// (serving: one token to some hundred), where the time is that of reading W once,
// and products whose reduction is long for their size (a weight gradient of a
// small layer over thousands of rows). A CTA holds 128 output features (the MMA's
// M rows) and up to 128 tokens (its N columns); the reduction is split over the S
// CTAs of a cluster so that about two CTAs run on every SM whatever the sizes
// are, each with some 100 KB of operands in flight. The S partial tiles meet in
// distributed shared memory: every CTA leaves its fp32 tile in its own shared
// memory, and after a cluster barrier adds up its 1/S of the entries over the
// peers, in rank order, so a result does not depend on timing and no workspace
// or counter is needed. Bound by HBM and by the 4 to 5 us of set-up, first load
// and join: one row of 14336 -> 4096 features 22 us (117 MB, 5.3 TB/s), 37 rows
// 24 to 26 us, 4096 -> 4096 10.5 us; without the split 60 and 21 us. A second
// form (Pair below) does the same with CTA pairs for some hundred rows.
#pragma once
#include "common.cuh"
#include "ptx.cuh"
#include "tile_gemm.cuh"

namespace moe {

constexpr int kFewThreads = 192;   // warp 0 TMA, warp 1 MMA and TMEM, warps 2..5 the partial tile
constexpr int kFewMaxStages = 6;
constexpr int kFewMaxSplit = 8;    // portable cluster size
constexpr int kFewSmemTiles = 108 * 1024;   // two CTAs on an SM
constexpr int kFewSmemTilesPair = 192 * 1024;   // pairs: one

struct FewParams {
  CUtensorMap tm_w;   // MN-major: {n, k} box {64, 64}; K-major: {k, n} box {64, 128}
  CUtensorMap tm_x;   // K-major: {k, t} box {64, nt (nt / 2 on pairs)}; MN-major: {t, k} box {64, 64}
  int M, K, T;        // output features, reduction, tokens
  int nt;             // MMA columns, a multiple of 32: up to 128, on pairs 256
  int split, stages;  // parts of the reduction
  int f16;
  int32_t* err;
  long long wait_cycles;
  void* out;
  long long ldo;
  const void* bias;
  const void* res;
  long long ldr;
  void* z;
  long long ldz;
  int act;
};

struct FewSmem {
  uint64_t full[kFewMaxStages];
  uint64_t empty[kFewMaxStages];
  uint64_t acc_full;
  uint32_t tmem_base;
  int abort;
};

// cols: a CTA's columns of Q
__host__ __device__ constexpr int few_stage_bytes(int cols) { return kTgABytes + cols * 128; }
__host__ __device__ constexpr size_t few_smem_bytes(int cols, int stages) {
  return 1024 + (size_t)stages * few_stage_bytes(cols) + sizeof(FewSmem);
}
// TMEM columns of an accumulator of nt
__host__ __device__ constexpr int few_tmem_cols(int nt) { return nt <= 32 ? 32 : nt <= 64 ? 64 : nt <= 128 ? 128 : 256; }

__device__ __forceinline__ bool few_wait(uint64_t* bar, uint32_t parity, const FewParams& p, FewSmem& s) {
  bool ok = tg_try_wait(bar, parity);
  if (!ok) {
    const long long t0 = clock64();
    while (!(ok = tg_try_wait(bar, parity))) {
      if (*reinterpret_cast<volatile int*>(&s.abort)) break;
      if (clock64() - t0 > p.wait_cycles) {
        if (p.err != nullptr) atomicCAS(p.err, 0, (int)kDevTimeout);
        *reinterpret_cast<volatile int*>(&s.abort) = 1;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void few_load3(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(0)
      : "memory");
}

__device__ __forceinline__ float4 few_ld_cluster(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at)
               : "memory");
  return v;
}

// Not inlined: a call runs this code once or twice, so the time of a copy is that of fetching it.
__device__ __noinline__ float4 few_act4(float4 a, int act) {
  if (act == kActRelu) return make_float4(tg_act<kActRelu>(a.x), tg_act<kActRelu>(a.y), tg_act<kActRelu>(a.z), tg_act<kActRelu>(a.w));
  if (act == kActGelu) return make_float4(tg_act<kActGelu>(a.x), tg_act<kActGelu>(a.y), tg_act<kActGelu>(a.z), tg_act<kActGelu>(a.w));
  if (act == kActGeluTanh)
    return make_float4(tg_act<kActGeluTanh>(a.x), tg_act<kActGeluTanh>(a.y), tg_act<kActGeluTanh>(a.z), tg_act<kActGeluTanh>(a.w));
  return make_float4(tg_act<kActSilu>(a.x), tg_act<kActSilu>(a.y), tg_act<kActSilu>(a.z), tg_act<kActSilu>(a.w));
}

// Bias, pre-activation, activation, residual and the store of features m .. m + 3 of token t.
template <typename T>
__device__ __forceinline__ void few_finish(const FewParams& p, float4 a, long long t, int m) {
  if (m >= p.M) return;   // M is a multiple of 8
  if (p.bias != nullptr) {
    const uint2 b = *reinterpret_cast<const uint2*>(reinterpret_cast<const T*>(p.bias) + m);
    const float2 lo = TgPair<T>::unpack(b.x), hi = TgPair<T>::unpack(b.y);
    a.x += lo.x;
    a.y += lo.y;
    a.z += hi.x;
    a.w += hi.y;
  }
  if (p.z != nullptr)
    *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.z) + t * p.ldz + m) =
        make_uint2(TgPair<T>::pack(a.x, a.y), TgPair<T>::pack(a.z, a.w));
  if (p.act != kActNone) a = few_act4(a, p.act);
  if (p.res != nullptr) {
    const uint2 b = *reinterpret_cast<const uint2*>(reinterpret_cast<const T*>(p.res) + t * p.ldr + m);
    const float2 lo = TgPair<T>::unpack(b.x), hi = TgPair<T>::unpack(b.y);
    a.x += lo.x;
    a.y += lo.y;
    a.z += hi.x;
    a.w += hi.y;
  }
  *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.out) + t * p.ldo + m) =
      make_uint2(TgPair<T>::pack(a.x, a.y), TgPair<T>::pack(a.z, a.w));
}

// The join's vector v of one part: four features of one token.
__device__ __forceinline__ void few_add(float4& a, uint32_t from, int v) {
  const float4 f = few_ld_cluster(from + v * 16);
  a.x += f.x;
  a.y += f.y;
  a.z += f.z;
  a.w += f.w;
}

// Pair: the parts are CTA pairs (tcgen05 cta_group::2, 256 features by up to 256
// tokens), one CTA on an SM, for products that the pairs of tile_gemm.cuh would
// leave most SMs without: half the operand bytes a FLOP of the single CTAs', and
// the reduction split (384 rows of 14336 -> 4096 features 43 us; single CTAs 73,
// whole reductions on pairs 69).
template <bool PMn, bool QMn, bool Pair, typename T>
__global__ void __launch_bounds__(kFewThreads, Pair ? 1 : 2) moe_few_rows_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kCtas = Pair ? 2 : 1;           // CTAs of a part
  const int cols = Pair ? p.nt >> 1 : p.nt;     // this CTA's columns of Q
  const int stage_bytes = few_stage_bytes(cols);
  FewSmem& s = *reinterpret_cast<FewSmem*>(tiles + (size_t)p.stages * stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ctas = p.split * kCtas;
  const int cta = ctas > 1 ? (int)ptx::cluster_ctarank() : 0;
  const int part = cta / kCtas, half = cta % kCtas, leader = cta - half;
  const int m0 = ((int)(blockIdx.x / ctas) * kCtas + half) * 128;
  const int t0 = (int)blockIdx.y * p.nt, rows = min(p.nt, p.T - t0);
  const int nk = (p.K + 63) >> 6;
  const int kb0 = (int)((long long)nk * part / p.split), kb1 = (int)((long long)nk * (part + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 1);
    }
    ptx::mbar_init(&s.acc_full, 1);
    s.abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tm_w);
    ptx::prefetch_tmap(&p.tm_x);
  }
  if (warp == 1) {
    if (Pair) {
      ptx::tmem_alloc_pair(&s.tmem_base, few_tmem_cols(p.nt));
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(&s.tmem_base, few_tmem_cols(p.nt));
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (Pair) ptx::cluster_sync();   // both CTAs' barriers exist before any remote arrive
  ptx::tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t tmem = s.tmem_base;
  const uint32_t base = ptx::smem_u32(tiles);

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!(ok = few_wait(&s.empty[stage], phase ^ 1, p, s))) break;
      if (tg_elect()) {
        const uint32_t dst = base + stage * stage_bytes, q = dst + kTgABytes;
        const int t = t0 + half * cols;
        if (Pair) {   // both CTAs' bytes on the leader's barrier
          const uint32_t bar = ptx::mapa(ptx::smem_u32(&s.full[stage]), leader);
          if (half == 0) ptx::mbar_arrive_expect_tx(&s.full[stage], 2 * stage_bytes);
          if (PMn) {
            tg_load3(dst, &p.tm_w, bar, m0, kb * 64, 0);
            tg_load3(dst + 8192, &p.tm_w, bar, m0 + 64, kb * 64, 0);
          } else {
            tg_load3(dst, &p.tm_w, bar, kb * 64, m0, 0);
          }
          if (QMn) {
            for (int j = 0; j < cols; j += 64) tg_load3(q + j * 128, &p.tm_x, bar, t + j, kb * 64, 0);
          } else {
            tg_load3(q, &p.tm_x, bar, kb * 64, t, 0);
          }
        } else {
          uint64_t* bar = &s.full[stage];
          ptx::mbar_arrive_expect_tx(bar, stage_bytes);
          if (PMn) {
            few_load3(dst, &p.tm_w, bar, m0, kb * 64);
            few_load3(dst + 8192, &p.tm_w, bar, m0 + 64, kb * 64);
          } else {
            few_load3(dst, &p.tm_w, bar, kb * 64, m0);
          }
          if (QMn) {
            for (int j = 0; j < cols; j += 64) few_load3(q + j * 128, &p.tm_x, bar, t + j, kb * 64);
          } else {
            few_load3(q, &p.tm_x, bar, kb * 64, t);
          }
        }
      }
      __syncwarp();
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // the commits that free the stages have arrived before the peer's barriers and tiles are given up
    for (int i = 0; Pair && ok && i < p.stages; ++i) {
      if (!(ok = few_wait(&s.empty[stage], phase ^ 1, p, s))) break;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok)   // given up: let the copies in flight land before the shared memory goes away
      for (int i = 0; i < 5000; ++i) __nanosleep(1000);
  } else if (warp == 1) {
    if (half == 0) {   // the leader of a pair issues for both
      const uint32_t fmt = p.f16 ? 0u : 1u;
      const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((PMn ? 1u : 0u) << 15) | ((QMn ? 1u : 0u) << 16) |
                             ((uint32_t)(p.nt >> 3) << 17) | (((Pair ? 256u : 128u) >> 4) << 24);
      const uint16_t both = (uint16_t)(3u << leader);
      const uint64_t pdesc = PMn ? ptx::smem_desc_sw128(base, 8192, 1024) : ptx::smem_desc_sw128(base, 16, 1024);
      const uint64_t qdesc = QMn ? ptx::smem_desc_sw128(base + kTgABytes, 8192, 1024)
                                 : ptx::smem_desc_sw128(base + kTgABytes, 16, 1024);
      constexpr uint64_t pstep = (PMn ? 2048 : 32) >> 4, qstep = (QMn ? 2048 : 32) >> 4;
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!few_wait(&s.full[stage], phase, p, s)) break;
        ptx::tc_fence_after();
        const uint64_t off = (uint64_t)(uint32_t)(stage * stage_bytes) >> 4;
        if (tg_elect()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (Pair) ptx::mma_bf16_pair(tmem, pdesc + off + kk * pstep, qdesc + off + kk * qstep, idesc, kb != kb0 || kk != 0 ? 1u : 0u);
            else ptx::mma_bf16(tmem, pdesc + off + kk * pstep, qdesc + off + kk * qstep, idesc, kb != kb0 || kk != 0 ? 1u : 0u);
          if (Pair) {
            ptx::mma_commit_pair_multicast(&s.empty[stage], both);
            if (kb == kb1 - 1) ptx::mma_commit_pair_multicast(&s.acc_full, both);
          } else {
            ptx::mma_commit(&s.empty[stage]);
            if (kb == kb1 - 1) ptx::mma_commit(&s.acc_full);
          }
        }
        __syncwarp();
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (few_wait(&s.acc_full, 0, p, s)) {
    // every MMA has read its tiles: their place takes the fp32 partial tile, [token][128 features]
    ptx::tc_fence_after();
    const int quad = warp & 3;
    float* mine = reinterpret_cast<float*>(tiles) + quad * 32 + lane;
    for (int c = 0; c < rows; c += 32) {
      uint32_t r[32];
      ptx::tmem_ld32(tmem + c + ((uint32_t)(quad * 32) << 16), r);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) mine[(c + i) * 128] = __uint_as_float(r[i]);
    }
    ptx::tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (ctas > 1) ptx::cluster_sync();

  // this CTA's share of the rows x 128 entries, four features at a time and four such vectors in flight
  const int vecs = rows * 32;
  const int v0 = (int)((long long)vecs * part / p.split), v1 = (int)((long long)vecs * (part + 1) / p.split);
  constexpr int kStep = kFewThreads;
#pragma unroll 1
  for (int v = v0 + (int)threadIdx.x; v < v1; v += 4 * kStep) {
    // vectors past the end are read at the last one and dropped
    const int at[4] = {v, min(v + kStep, v1 - 1), min(v + 2 * kStep, v1 - 1), min(v + 3 * kStep, v1 - 1)};
    float4 a[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.split > 1) {
#pragma unroll 2
      for (int i = 0; i < p.split; ++i) {
        const uint32_t from = ptx::mapa(base, i * kCtas + half);
#pragma unroll
        for (int u = 0; u < 4; ++u) few_add(a[u], from, at[u]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) a[u] = reinterpret_cast<const float4*>(tiles)[at[u]];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v + u * kStep < v1) few_finish<T>(p, a[u], t0 + (at[u] >> 5), m0 + (at[u] & 31) * 4);
  }
  __syncthreads();
  if (ctas > 1) ptx::cluster_sync();   // no peer still reads this CTA's partial tile
  ptx::tc_fence_after();
  if (warp == 1) {
    if (Pair) ptx::tmem_dealloc_pair(tmem, few_tmem_cols(p.nt));
    else ptx::tmem_dealloc(tmem, few_tmem_cols(p.nt));
  }
}

}  // namespace moe
