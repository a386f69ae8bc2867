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
// 26 us, 4096 -> 4096 10.5 us; without the split 60 and 21 us.
#pragma once
#include "common.cuh"
#include "ptx.cuh"
#include "tile_gemm.cuh"

namespace moe {

constexpr int kFewThreads = 192;   // warp 0 TMA, warp 1 MMA and TMEM, warps 2..5 the partial tile
constexpr int kFewMaxStages = 6;
constexpr int kFewMaxSplit = 8;    // portable cluster size
constexpr int kFewSmemTiles = 108 * 1024;   // two CTAs on an SM

struct FewParams {
  CUtensorMap tm_w;   // MN-major: {n, k} box {64, 64}; K-major: {k, n} box {64, 128}
  CUtensorMap tm_x;   // K-major: {k, t} box {64, nt}; MN-major: {t, k} box {64, 64}
  int M, K, T;        // output features, reduction, tokens
  int nt;             // MMA columns: 32, 64 or 128
  int split, stages;
  int f16;
  int32_t* err;
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

__host__ __device__ constexpr int few_stage_bytes(int nt) { return kTgABytes + nt * 128; }
__host__ __device__ constexpr size_t few_smem_bytes(int nt, int stages) {
  return 1024 + (size_t)stages * few_stage_bytes(nt) + sizeof(FewSmem);
}

__device__ __forceinline__ bool few_wait(uint64_t* bar, uint32_t parity, const FewParams& p, FewSmem& s) {
  bool ok = tg_try_wait(bar, parity);
  if (!ok) {
    const long long t0 = clock64();
    while (!(ok = tg_try_wait(bar, parity))) {
      if (*reinterpret_cast<volatile int*>(&s.abort)) break;
      if (clock64() - t0 > kTgTimeoutCycles) {
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

template <bool PMn, bool QMn, typename T>
__global__ void __launch_bounds__(kFewThreads, 2) moe_few_rows_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = few_stage_bytes(p.nt);
  FewSmem& s = *reinterpret_cast<FewSmem*>(tiles + (size_t)p.stages * stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)ptx::cluster_ctarank() : 0;
  const int m0 = (int)(blockIdx.x / p.split) * 128;
  const int t0 = (int)blockIdx.y * p.nt, rows = min(p.nt, p.T - t0);
  const int nk = (p.K + 63) >> 6;
  const int kb0 = (int)((long long)nk * rank / p.split), kb1 = (int)((long long)nk * (rank + 1) / p.split);

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
    ptx::tmem_alloc(&s.tmem_base, p.nt);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
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
        const uint32_t dst = base + stage * stage_bytes;
        ptx::mbar_arrive_expect_tx(&s.full[stage], stage_bytes);
        if (PMn) {
          few_load3(dst, &p.tm_w, &s.full[stage], m0, kb * 64);
          few_load3(dst + 8192, &p.tm_w, &s.full[stage], m0 + 64, kb * 64);
        } else {
          few_load3(dst, &p.tm_w, &s.full[stage], kb * 64, m0);
        }
        if (QMn) {
          for (int j = 0; j < p.nt; j += 64) few_load3(dst + kTgABytes + j * 128, &p.tm_x, &s.full[stage], t0 + j, kb * 64);
        } else {
          few_load3(dst + kTgABytes, &p.tm_x, &s.full[stage], kb * 64, t0);
        }
      }
      __syncwarp();
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok)   // given up: let the copies in flight land before the shared memory goes away
      for (int i = 0; i < 5000; ++i) __nanosleep(1000);
  } else if (warp == 1) {
    const uint32_t fmt = p.f16 ? 0u : 1u;
    const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((PMn ? 1u : 0u) << 15) | ((QMn ? 1u : 0u) << 16) |
                           ((uint32_t)(p.nt >> 3) << 17) |
                           ((128u >> 4) << 24);
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
          ptx::mma_bf16(tmem, pdesc + off + kk * pstep, qdesc + off + kk * qstep, idesc, kb != kb0 || kk != 0 ? 1u : 0u);
        ptx::mma_commit(&s.empty[stage]);
        if (kb == kb1 - 1) ptx::mma_commit(&s.acc_full);
      }
      __syncwarp();
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
  } else if (few_wait(&s.acc_full, 0, p, s)) {
    // every MMA has read its tiles: their place takes the fp32 partial tile, [token][128 features]
    ptx::tc_fence_after();
    const int quad = warp & 3;
    float* part = reinterpret_cast<float*>(tiles) + quad * 32 + lane;
    for (int c = 0; c < rows; c += 32) {
      uint32_t r[32];
      ptx::tmem_ld32(tmem + c + ((uint32_t)(quad * 32) << 16), r);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) part[(c + i) * 128] = __uint_as_float(r[i]);
    }
    ptx::tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (p.split > 1) ptx::cluster_sync();

  // this CTA's share of the rows x 128 entries, four features at a time; two vectors' parts in flight
  const int vecs = rows * 32;
  const int v0 = (int)((long long)vecs * rank / p.split), v1 = (int)((long long)vecs * (rank + 1) / p.split);
#pragma unroll 1
  for (int v = v0 + (int)threadIdx.x; v < v1; v += 2 * kFewThreads) {
    const int w = v + kFewThreads < v1 ? v + kFewThreads : v;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (p.split > 1) {
#pragma unroll 4
      for (int i = 0; i < p.split; ++i) {
        const uint32_t from = ptx::mapa(base, i);
        const float4 f = few_ld_cluster(from + v * 16), g = few_ld_cluster(from + w * 16);
        a.x += f.x;
        a.y += f.y;
        a.z += f.z;
        a.w += f.w;
        b.x += g.x;
        b.y += g.y;
        b.z += g.z;
        b.w += g.w;
      }
    } else {
      a = reinterpret_cast<const float4*>(tiles)[v];
      b = reinterpret_cast<const float4*>(tiles)[w];
    }
#pragma unroll 1
    for (int u = v;; u = w, a = b) {
      few_finish<T>(p, a, t0 + (u >> 5), m0 + (u & 31) * 4);
      if (u == w) break;
    }
  }
  __syncthreads();
  if (p.split > 1) ptx::cluster_sync();   // no peer still reads this CTA's partial tile
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, p.nt);
}

}  // namespace moe
