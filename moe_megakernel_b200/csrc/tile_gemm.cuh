// Tiled matrix products on CTA pairs (tcgen05 cta_group::2) for the operators
// around the MoE layer: products grouped by expert over ragged row groups, the
// dense layer, the weight gradients of both, and the symmetric products of the
// Newton-Schulz iteration.
//
// Every product is written as  out[n, m] = sum_k P[m, k] * Q[n, k]  with m
// contiguous in the output. P, the M side, fills the 256 rows of a pair's MMA
// (128 in each CTA); Q, the N side, its 32 .. 256 columns. For a layer's
// forward P is W^T (so the tile's 256 rows are output features) and Q the
// token rows: a group of c tokens then costs ceil(c / 32) * 32 columns of MMA
// instead of whole 256-row tiles, and a weight tile is read once for up to 256
// tokens. Either operand may have its k index contiguous ("K-major") or its m
// / n index contiguous ("MN-major"); the tensor core reads both, so no operand
// is ever transposed in memory.
//
// Roles per CTA: warp 0 TMA loads, warp 1 MMA issue (leader CTA), warp 2 the
// zero rows of a ragged reduction's last block, warp 3 TMEM and the list of
// tiles, warps 4..11 the epilogue. Each CTA loads its 128 rows of P and half of the tile's Q into its
// own shared memory; both CTAs' bytes are counted on the leader's barrier.
// Two TMEM accumulators let a tile's epilogue run under the next tile's MMAs.
// Tiles are dealt round robin; nothing is exchanged between pairs. Warp 3 works
// out each tile (up to six integer divisions, about 1200 cycles) up to four tiles
// ahead of the others, so that no role spends its own time on it.
//
// What bounds it: a k block (64 k) of a 256 x 256 tile is 512 cycles of MMA by
// the nominal rate (474 measured with its operands at hand) and 32 KB of loads in
// each CTA, 64 bytes a cycle and SM, which is what L2 delivers: with operands
// shared by few pairs at a time a k block takes 600 to 750 cycles. 8192 x 4096 ->
// 14336 features, bf16: 609 us (1.58 PFLOP/s) in a burst and 718 us (1.34) under
// the 1 kW cap, where the clock settles near 1.2 GHz; the library's plain product
// of the same matrices 628 and 716 us on the same GPU. Tensor pipe busy 85 to 87 %
// of the cycles (dense 4096 x 4096 -> 14336 and 128 uneven groups, ncu). Tiles of
// 256 columns are the largest with two accumulators in TMEM; smaller ones load
// more a FLOP (see pick_tile in operators.cu).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstddef>
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kTgThreads = 384;
constexpr int kTgEpiWarps = 8;
constexpr int kTgMaxStages = 12;
constexpr int kTgMaxGroups = 1024;
constexpr int kTgSorted = 256;           // groups that a weight gradient sorts by size
constexpr int kTgRing = 4;               // tiles worked out ahead
constexpr int kTgABytes = 128 * 128;     // 128 rows of P, 64 k each
// A wait's bound: about two seconds, and 4096 cycles for each block of 64 of the launch's longest reduction
// (measured 600 to 1200): the longest wait of a sound call is the epilogue's, for all of a tile's blocks, and a
// group may have 2^24 of them.
constexpr long long kTgTimeoutCycles = 4000000000ll, kTgBlockCycles = 4096;
constexpr long long tg_wait_cycles(long long k) { return kTgTimeoutCycles + (k + 63) / 64 * kTgBlockCycles; }

enum TgMode : int {
  kTgRaggedN = 0,    // groups of N-side rows, one P per group (offsets == null: one group of all rows)
  kTgRaggedK = 1,    // groups of the reduction, one output per group (offsets == null: one group)
  kTgBatched = 2,    // the same product for every batch index
  kTgSymmetric = 3,  // batched, P = Q: only the tiles on and below the diagonal, stored twice
};

enum TgEpilogue : int {
  kTgStore = 0,     // act(acc + bias) + residual, the pre-activation kept on request
  kTgGram = 1,      // Newton-Schulz: A = X X^T, scaled
  kTgPoly = 2,      // B = b A + c A A
  kTgUpdate = 3,    // X' = a X + B X (X as fp16 and 8 bits more)
  kTgUpdateOut = 4, // the same, stored as bf16 at the caller's place, transposed on request
  kTgPlain = 5,     // the accumulator alone (gradients)
};

enum TgAct : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// The Newton-Schulz epilogues' coefficients.
struct TgFactors {
  float ca, cb;           // on the stored value and on the accumulator
  const float* alpha;     // [batches] or null: times the update, squared times the Gram matrix
  const uint8_t* lo_in;   // the low bits of X, or null
  float diagonal;         // kTgPoly: added to the diagonal
};

struct TgParams {
  CUtensorMap tm_p;      // K-major: {k, m, batch} box {64, 128}; MN-major: {m, k, batch} box {64, 64}
  CUtensorMap tm_q[4];   // K-major: {k, n, batch} boxes of 128, 64, 32, 16 rows; MN-major: [0] box {64, 64}
  CUtensorMap tm_out;    // {m, n, batch} box {32, 32}: one piece of the epilogue (not kTgUpdateOut)
  int M, N, K;           // extents (N: rows of Q in a ragged-N product; K: rows in a ragged-K one)
  int groups;            // groups or batches
  int nt;                // largest N tile, a multiple of 32 up to 256
  int stages, stage_bytes, epi_bytes;
  int f16;               // operands are fp16 (else bf16)
  const int32_t* offsets;   // [groups + 1] device, or null
  int32_t* err;             // device error word, or null
  long long wait_cycles;    // bound of a wait (tg_wait_cycles of the longest reduction)
  // output
  void* out;
  long long ldo, out_bs;    // row and batch pitch in elements
  // kTgStore
  const void* bias;         // [M]
  const void* res;
  long long ldr;
  void* z;
  long long ldz;
  int act;
  // Newton-Schulz
  const __half* in;         // kTgPoly: A; kTgUpdate: X, the fp16 part
  uint8_t* lo_out;          // kTgUpdate: X, the 8 bits below it, in pieces
  long long ldi, in_bs, lo_bs;
  TgFactors factors;
  int backwards;            // batches from the last to the first
  int transposed;           // kTgUpdateOut: rows m of n
};

struct TgTask {
  int g;        // group or batch; -1: no more tiles
  int m0;       // first M row of the tile
  int n0;       // first N row of the tile (within Q; absolute in a ragged-N product)
  int cols;     // valid N rows
  int nt;       // MMA columns (multiple of 32)
  int k0, klen; // reduction range
  int mirror;   // the tile is also stored transposed (symmetric products, off the diagonal)
};

struct TgSmem {
  uint64_t full[kTgMaxStages];
  uint64_t empty[kTgMaxStages];
  uint64_t tail[kTgMaxStages];
  uint64_t peer_tail[kTgMaxStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t task_full[kTgRing];
  uint64_t task_empty[kTgRing];
  TgTask task[kTgRing];
  uint32_t tmem_base;
  int abort;
  int total;
  // behind it, in ragged products: start[groups] and count[groups], the groups' rows as used (an
  // invalid group is empty), and tile0[groups + 1], the first N tile of each group (ragged N), or
  // order[groups], the groups from the largest to the smallest (ragged K)
  __device__ int* start() { return reinterpret_cast<int*>(this + 1); }
  __device__ int* count(int groups) { return start() + groups; }
  __device__ int* tile0(int groups) { return start() + 2 * groups; }
  __device__ int* order(int groups) { return start() + 2 * groups; }
};

constexpr int kTgSmemMax = 232448;   // shared memory of a CTA
constexpr size_t tg_smem_bytes(int stages, int stage_bytes, int epi_bytes, int table_groups) {
  return 1024 + (size_t)stages * stage_bytes + epi_bytes + sizeof(TgSmem) + (3 * (size_t)table_groups + 1) * 4;
}

__device__ __forceinline__ void tg_set_error(const TgParams& p, TgSmem& s, int code, bool stop) {
  if (p.err != nullptr) atomicCAS(p.err, 0, code);
  if (stop) *reinterpret_cast<volatile int*>(&s.abort) = 1;
}

// Bounded wait on a local barrier phase, by one thread or by a whole warp (all
// lanes poll; tg_wait_warp's answer is the same in every lane). The hint lets the
// hardware suspend the warp for up to a millisecond per attempt: polling warps
// cost power, which at full load is clock. The bound is on SM cycles, which are
// cheap to read.
__device__ __forceinline__ bool tg_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(ptx::smem_u32(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
// Cluster: the arrival is the peer CTA's and orders what it wrote to its shared memory.
template <bool Cluster = false>
__device__ __forceinline__ bool tg_wait(uint64_t* bar, uint32_t parity, const TgParams& p, TgSmem& s) {
  auto arrived = [&] { return Cluster ? ptx::mbar_try_wait_cluster(bar, parity) : tg_try_wait(bar, parity); };
  if (arrived()) return true;
  const long long t0 = clock64();
  while (!arrived()) {
    if (*reinterpret_cast<volatile int*>(&s.abort)) return false;
    if (clock64() - t0 > p.wait_cycles) {
      tg_set_error(p, s, kDevTimeout, true);
      return false;
    }
  }
  return true;
}
template <bool Cluster = false>
__device__ __forceinline__ bool tg_wait_warp(uint64_t* bar, uint32_t parity, const TgParams& p, TgSmem& s) {
  const bool ok = tg_wait<Cluster>(bar, parity, p, s);
  return __all_sync(0xffffffffu, ok);
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool tg_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Position of tile `idx` in a grid of mt x ntl tiles: bands of 8 M tiles, all
// N tiles of a band before the next band, so that the pairs working at one
// time share both operands in L2 (74 pairs cover about 8 x 9 tiles).
__device__ __forceinline__ void tg_raster(int idx, int mt, int ntl, int& m, int& n) {
  constexpr int kBand = 8;
  const int band = idx / (kBand * ntl);
  const int wide = min(kBand, mt - band * kBand);
  const int rem = idx - band * kBand * ntl;
  n = rem / wide;
  m = band * kBand + rem - n * wide;
}

// N tile j of `rows` rows: equal tiles of a multiple of 32 rows, at most cap
// (their number is the smallest possible, so none is empty).
__device__ __forceinline__ void tg_split(int rows, int cap, int j, int& at, int& cols) {
  const int tiles = (rows + cap - 1) / cap;
  const int each = ((rows + tiles - 1) / tiles + 31) & ~31;
  at = j * each;
  cols = min(each, rows - at);
}

template <int Mode>
__device__ __forceinline__ TgTask tg_decode(int t, const TgParams& p, TgSmem& s) {
  TgTask k{};
  const int mt = (p.M + 255) >> 8;
  if (Mode == kTgRaggedN) {
    const int* tile0 = s.tile0(p.groups);
    int lo = 0, hi = p.groups - 1;   // the last group whose first tile is at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile0[mid] * mt <= t) lo = mid;
      else hi = mid - 1;
    }
    k.g = lo;
    const int ntl = tile0[lo + 1] - tile0[lo];
    int m, n;
    tg_raster(t - tile0[lo] * mt, mt, ntl, m, n);
    tg_split(s.count(p.groups)[lo], p.nt, n, k.n0, k.cols);
    k.n0 += s.start()[lo];
    k.m0 = m << 8;
    k.k0 = 0;
    k.klen = p.K;
  } else if (Mode == kTgSymmetric) {
    const int per = mt * (mt + 1) / 2;
    k.g = t / per;
    int r = t - k.g * per, m = 0;
    while (r > m) r -= ++m;          // row m of the triangle has m + 1 tiles
    k.m0 = m << 8;
    k.n0 = r << 8;
    k.cols = min(256, p.N - k.n0);
    k.klen = p.K;
    k.mirror = k.m0 != k.n0;
  } else {
    const int ntl = (p.N + p.nt - 1) / p.nt;
    k.g = t / (mt * ntl);
    int m, n;
    tg_raster(t - k.g * mt * ntl, mt, ntl, m, n);
    tg_split(p.N, p.nt, n, k.n0, k.cols);
    k.m0 = m << 8;
    if (Mode == kTgRaggedK) {
      k.g = s.order(p.groups)[k.g];
      k.k0 = s.start()[k.g];
      k.klen = s.count(p.groups)[k.g];
    } else {
      k.klen = p.K;
    }
  }
  if ((Mode == kTgBatched || Mode == kTgSymmetric) && p.backwards) k.g = p.groups - 1 - k.g;
  k.nt = (k.cols + 31) & ~31;
  return k;
}

// Reduction steps (of 16) of k block kb.
__device__ __forceinline__ int tg_ksteps(const TgTask& k, int kb) { return min(4, (k.klen - kb * 64 + 15) >> 4); }

// The stream's earlier work is done and visible (programmatic stream serialisation).
__device__ __forceinline__ void tg_after_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------- list of tiles (warp 3)
// A warp's place in the list.
struct TgCursor {
  int q = 0;
  uint32_t phase = 0;
  // The next tile; false at the end (or once a wait has been given up).
  __device__ __forceinline__ bool next(TgTask& k, const TgParams& p, TgSmem& s) {
    if (!tg_wait_warp(&s.task_full[q], phase, p, s)) return false;
    k = s.task[q];
    __syncwarp();
    if (ptx::lane_id() == 0) ptx::mbar_arrive(&s.task_empty[q]);
    step();
    return k.g >= 0;
  }
  __device__ __forceinline__ void step() {
    if (++q == kTgRing) {
      q = 0;
      phase ^= 1;
    }
  }
};

// Where a role stands in the rings of stages, accumulators and tiles; one per
// warp.
struct TgState {
  int stage = 0;
  uint32_t phase = 0;
  int acc = 0;
  uint32_t acc_phase = 0;
  TgCursor list;
  __device__ __forceinline__ void next_stage(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ void next_acc() {
    if (++acc == 2) {
      acc = 0;
      acc_phase ^= 1;
    }
  }
};

template <int Mode>
__device__ void tg_schedule(const TgParams& p, TgSmem& s, TgState& at, int first, int end, int step) {
  int t = first;
  for (int round = 0;; ++round) {
    TgTask k{};
    k.g = -1;
    if (t < end) k = tg_decode<Mode>(t, p, s);
    if (!tg_wait_warp(&s.task_empty[at.list.q], at.list.phase ^ 1, p, s)) return;
    if (ptx::lane_id() == 0) {
      s.task[at.list.q] = k;
      ptx::mbar_arrive(&s.task_full[at.list.q]);
    }
    __syncwarp();
    at.list.step();
    if (k.g < 0) return;
    if (round == 0) tg_after_stream();   // before a wait that runs against the clock
    // round robin; tiles sorted by their time (ragged K) in turn from either end
    t = Mode == kTgRaggedK && (round & 1) == 0 ? (round + 1) * step + step - 1 - first : (round + 1) * step + first;
  }
}

// ---------------------------------------------------------------- loads
__device__ __forceinline__ void tg_load3(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// This CTA's half of one stage; returns nothing, all bytes are counted on `bar`.
template <bool PMn, bool QMn>
__device__ __forceinline__ void tg_load_stage(uint32_t dst, const TgParams& p, const TgTask& k, int kpos, int rank,
                                              uint32_t bar, int pbatch, int qbatch) {
  const int m = k.m0 + rank * 128;
  if (PMn) {
    tg_load3(dst, &p.tm_p, bar, m, kpos, pbatch);
    tg_load3(dst + 8192, &p.tm_p, bar, m + 64, kpos, pbatch);
  } else {
    tg_load3(dst, &p.tm_p, bar, kpos, m, pbatch);
  }
  const uint32_t q = dst + kTgABytes;
  const int half = k.nt >> 1;
  const int n = k.n0 + rank * half;
  if (QMn) {
    for (int j = 0; j < half; j += 64) tg_load3(q + j * 128, &p.tm_q[0], bar, n + j, kpos, qbatch);
  } else {
    int at = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // half = a sum of boxes of 128, 64, 32 and 16 rows
      const int rows = 128 >> i;
      if (half & rows) {
        tg_load3(q + at * 128, &p.tm_q[i], bar, kpos, n + at, qbatch);
        at += rows;
      }
    }
  }
}

template <bool QMn>
__device__ __forceinline__ uint32_t tg_stage_tx(const TgTask& k) {
  const int half = k.nt >> 1;
  return kTgABytes + (QMn ? ((half + 63) >> 6) * 8192 : half * 128);
}

template <int Mode>
__device__ __forceinline__ bool tg_has_tail(const TgTask& k, int kb) {
  // a ragged reduction's last block runs into the next group's rows inside a step of 16
  return Mode == kTgRaggedK && k.klen - kb * 64 < 64 && (k.klen & 15) != 0;
}

template <int Mode, bool PMn, bool QMn>
__device__ void tg_producer(const TgParams& p, TgSmem& s, TgState& at, uint32_t tiles, uint32_t rank) {
  bool ok = true;
  TgTask k;
  while (ok && at.list.next(k, p, s)) {
    const int nk = (k.klen + 63) >> 6;
    const uint32_t tx = tg_stage_tx<QMn>(k);
    const int pbatch = Mode == kTgRaggedK ? 0 : k.g;
    const int qbatch = Mode == kTgRaggedK || Mode == kTgRaggedN ? 0 : k.g;
    for (int kb = 0; kb < nk; ++kb) {
      if (!tg_wait_warp(&s.empty[at.stage], at.phase ^ 1, p, s)) {
        ok = false;
        break;
      }
      const uint32_t dst = tiles + at.stage * p.stage_bytes;
      const bool tail = tg_has_tail<Mode>(k, kb);
      // both CTAs' bytes on the leader's barrier; a tail block's on each CTA's own
      const uint32_t bar = tail ? ptx::mapa(ptx::smem_u32(&s.tail[at.stage]), rank)
                                : ptx::mapa(ptx::smem_u32(&s.full[at.stage]), 0);
      if (tg_elect()) {
        if (tail) ptx::mbar_arrive_expect_tx(&s.tail[at.stage], tx);
        else if (rank == 0) ptx::mbar_arrive_expect_tx(&s.full[at.stage], 2 * tx);
        tg_load_stage<PMn, QMn>(dst, p, k, k.k0 + kb * 64, rank, bar, pbatch, qbatch);
      }
      __syncwarp();
      at.next_stage(p.stages);
    }
  }
  // the commits that free the stages have arrived before this CTA's barriers go away
  TgState drain = at;
  for (int i = 0; ok && i < p.stages; ++i) {
    ok = tg_wait_warp(&s.empty[drain.stage], drain.phase ^ 1, p, s);
    drain.next_stage(p.stages);
  }
  if (!ok) {   // given up: let the copies in flight land before the shared memory goes away
    for (int i = 0; i < 5000; ++i) __nanosleep(1000);
  }
}

// ---------------------------------------------------------------- zero rows of a ragged reduction's last block
// The block holds the group's last klen % 64 rows and then rows of the next
// group. Steps of 16 past the group are not issued; the rows left inside the
// last step are overwritten with zeros in both operands (zeros in one alone
// would still meet an infinity or NaN of another group in the other).
template <int Mode>
__device__ void tg_tail_warp(const TgParams& p, TgSmem& s, TgState& at, uint8_t* tiles, uint32_t rank) {
  const int lane = ptx::lane_id();
  int stage = 0;
  uint32_t used = 0;   // parity of each stage's tail barrier
  TgTask k;
  while (at.list.next(k, p, s)) {
    const int nk = (k.klen + 63) >> 6;
    if (nk == 0) continue;
    const int last = (stage + nk - 1) % p.stages;
    if (tg_has_tail<Mode>(k, nk - 1)) {
      if (!tg_wait_warp(&s.tail[last], (used >> last) & 1, p, s)) return;
      const int r0 = k.klen & 63, r1 = (r0 + 15) & ~15;
      const int boxes = 2 + (((k.nt >> 1) + 63) >> 6);
      uint8_t* rows = tiles + (size_t)last * p.stage_bytes;
      for (int b = 0; b < boxes; ++b)
        for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
          *reinterpret_cast<uint4*>(rows + b * 8192 + i * 16) = make_uint4(0, 0, 0, 0);
      ptx::fence_proxy_async_shared();
      __syncwarp();
      if (rank != 0) {
        if (lane == 0) ptx::mbar_arrive_remote(ptx::mapa(ptx::smem_u32(&s.peer_tail[last]), 0));
      } else {   // in place of the producer's arrival, once both CTAs' blocks are clean
        if (!tg_wait_warp<true>(&s.peer_tail[last], (used >> last) & 1, p, s)) return;
        if (lane == 0) ptx::mbar_arrive(&s.full[last]);
      }
      __syncwarp();
      used ^= 1u << last;
    }
    stage = (stage + nk) % p.stages;
  }
}

// ---------------------------------------------------------------- MMA (leader)
// The warp runs the loop together and one lane issues: the descriptors are then
// warp-uniform values. With the loop inside a one-lane branch a k block took some
// 550 cycles to issue whatever its columns (an MMA 75, the barriers 250), which
// held narrow tiles back most: 256 rows over 163 experts of 7168 x 2048 took
// 955 us instead of 729, 37 rows of 14336 -> 4096 109 us instead of 61.
template <int Mode, bool PMn, bool QMn>
__device__ void tg_mma(const TgParams& p, TgSmem& s, TgState& at, uint32_t tiles, uint32_t tmem) {
  const uint32_t fmt = p.f16 ? 0u : 1u;
  const uint32_t idesc0 = (1u << 4) | (fmt << 7) | (fmt << 10) | ((PMn ? 1u : 0u) << 15) | ((QMn ? 1u : 0u) << 16) |
                          ((256u >> 4) << 24);
  const uint64_t pdesc = PMn ? ptx::smem_desc_sw128(tiles, 8192, 1024) : ptx::smem_desc_sw128(tiles, 16, 1024);
  const uint64_t qdesc = QMn ? ptx::smem_desc_sw128(tiles + kTgABytes, 8192, 1024)
                             : ptx::smem_desc_sw128(tiles + kTgABytes, 16, 1024);
  constexpr uint64_t pstep = (PMn ? 2048 : 32) >> 4, qstep = (QMn ? 2048 : 32) >> 4;   // 16 k further
  TgTask k;
  while (at.list.next(k, p, s)) {
    const int nk = (k.klen + 63) >> 6;
    if (nk == 0) continue;
    if (!tg_wait_warp(&s.acc_empty[at.acc], at.acc_phase ^ 1, p, s)) return;
    ptx::tc_fence_after();
    const uint32_t d = tmem + at.acc * 256;
    const uint32_t idesc = idesc0 | ((uint32_t)(k.nt >> 3) << 17);
    for (int kb = 0; kb < nk; ++kb) {
      if (!tg_wait_warp(&s.full[at.stage], at.phase, p, s)) return;
      ptx::tc_fence_after();
      const uint64_t off = (uint64_t)(uint32_t)(at.stage * p.stage_bytes) >> 4;
      const int steps = Mode == kTgRaggedK ? tg_ksteps(k, kb) : 4;
      if (tg_elect()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (Mode != kTgRaggedK || kk < steps)
            ptx::mma_bf16_pair(d, pdesc + off + kk * pstep, qdesc + off + kk * qstep, idesc, (kb | kk) != 0 ? 1u : 0u);
        ptx::mma_commit_pair_multicast(&s.empty[at.stage], 0x3);
        if (kb == nk - 1) ptx::mma_commit_pair_multicast(&s.acc_full[at.acc], 0x3);
      }
      __syncwarp();
      at.next_stage(p.stages);
    }
    at.next_acc();
  }
}

// ---------------------------------------------------------------- epilogue
template <typename T>
struct TgPair;
template <>
struct TgPair<bf16> {
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <>
struct TgPair<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// Activations in some 15 instructions a value. The erf form takes Phi(z), the normal distribution, from its
// smaller tail, Phi(-|z|) = e^(-z^2/2) t P(t) with t = 1 / (1 + 0.265 |z|): the scaled tail
// e^(z^2/2) Phi(-|z|) falls from 1/2 to 1 / (|z| sqrt(2 pi)) and has no other feature, so a polynomial in t
// fits it evenly, and the exponential is the one that the slope's density needs. P is of degree 6, fitted
// here by linear programming to the least largest relative error over 0 <= |z| <= 14: 6.3e-7, in fp32 1e-6
// and, as the exponential's argument is rounded, 5e-6 at |z| = 12. A bound on the relative error, so that
// small values on the negative side (z = -8: 5e-15) have all of their bits. The tanh form is z sigmoid(2 u).
// Both are far within a 16-bit rounding (2^-11). With erff the dense layer's backward pass spent 54 us in
// 4093 x 7168 slopes, above the 27 us of their memory traffic.
// sigmoid(z) and its slope q (1 - q), both from e^-|z|: neither side cancels, and no divisor leaves 1 .. 2 (a
// divisor above 2^126, at z = -87.4, makes __fdividef's quotient 0).
__device__ __forceinline__ float tg_sigmoid(float z, float& slope) {
  const float e = __expf(-fabsf(z));
  const float r = __fdividef(1.f, 1.f + e), s = e * r;
  slope = r * s;
  return z > 0.f ? r : s;
}
__device__ __forceinline__ float tg_sigmoid(float z) {
  float slope;
  return tg_sigmoid(z, slope);
}
// Phi(z); density: e^(-z^2/2) / sqrt(2 pi)
__device__ __forceinline__ float tg_normal(float z, float& density) {
  const float e = __expf(-0.5f * z * z);
  const float t = __fdividef(1.f, fmaf(0.265f, fabsf(z), 1.f));
  float q = fmaf(t, -0.067787088f, 0.195273280f);
  q = fmaf(t, q, -0.066363171f);
  q = fmaf(t, q, 0.142493516f);
  q = fmaf(t, q, 0.082946517f);
  q = fmaf(t, q, 0.107836798f);
  q = fmaf(t, q, 0.105599836f);
  const float tail = t * q * e;   // the smaller side
  density = e * 0.39894228040143268f;
  return z > 0.f ? 1.f - tail : tail;
}
template <int Act>
__device__ __forceinline__ float tg_act(float z) {
  if (Act == kActRelu) return z > 0.f || z != z ? z : 0.f;
  if (Act == kActGelu) {
    float density;
    return z * tg_normal(z, density);
  }
  if (Act == kActGeluTanh) return z * tg_sigmoid(1.59576912160573071f * fmaf(0.044715f * z * z, z, z));
  if (Act == kActSilu) return z * tg_sigmoid(z);
  return z;
}
template <int Act>
__device__ __forceinline__ void tg_act_each(uint32_t (&r)[2][16]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i >> 4][i & 15] = __float_as_uint(tg_act<Act>(__uint_as_float(r[i >> 4][i & 15])));
}
// One branch per 32 values: chosen inside the loop, the five functions' code
// (each inlined per value) was jumped over for every value.
__device__ __forceinline__ void tg_act_all(uint32_t (&r)[2][16], int act) {
  if (act == kActNone) return;
  if (act == kActRelu) tg_act_each<kActRelu>(r);
  else if (act == kActGelu) tg_act_each<kActGelu>(r);
  else if (act == kActGeluTanh) tg_act_each<kActGeluTanh>(r);
  else tg_act_each<kActSilu>(r);
}

// A warp works on 32 x 32 pieces of the accumulator: 32 M rows (its TMEM lanes)
// by 32 N columns. tcgen05.ld.16x256b hands each thread, for every 8 x 8 block,
// two neighbouring n of one m - the fragment that stmatrix and ldmatrix move to
// and from shared memory, transposed on request. So the piece is turned to
// output order (n rows of contiguous m) by four stmatrix and stored by one TMA
// copy (16-byte vectors where a group ends inside it), and what the epilogue
// reads (the residual, X, A) comes in the same way, copied ahead with cp.async.
// Storing straight from a 32x32b load took about 490 instructions a piece, mostly lane
// swaps and addresses, and held the weight gradient at 1.6 TB/s.
//
// A piece in shared memory: 32 rows of 64 bytes, the row's 16-byte chunk c at
// place c ^ (row / 2 % 4), which spreads both the matrix and the row accesses
// over all banks.
constexpr int kTgPiece = 2048;
__device__ __forceinline__ uint32_t tg_piece_at(int row, int c) { return row * 64 + ((c ^ ((row >> 1) & 3)) << 4); }

__device__ __forceinline__ void tg_tmem_frag(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Four 8 x 8 matrices whose rows start at the addresses of lanes 0-7, 8-15, 16-23, 24-31.
template <bool Trans>
__device__ __forceinline__ void tg_stmatrix(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  if (Trans)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
  else
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
template <bool Trans>
__device__ __forceinline__ void tg_ldmatrix(uint32_t at, uint32_t (&v)[4]) {
  if (Trans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ uint4 tg_lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// One piece as a thread holds it: v[4 i + b] packs n = 8 i + 2 (lane % 4) and
// n + 1 of m = 8 b + lane / 4.
// To shared memory as n rows of m (kRows = N) or as m rows of n (kRows = M).
enum TgRows { kRowsN, kRowsM };
template <TgRows R>
__device__ __forceinline__ void tg_piece_put(uint32_t piece, const uint32_t (&v)[16], int lane) {
  const int j = lane >> 3, r = lane & 7;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (R == kRowsN) tg_stmatrix<true>(piece + tg_piece_at(8 * i + r, j), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    else tg_stmatrix<false>(piece + tg_piece_at(8 * i + r, j), v[i], v[4 + i], v[8 + i], v[12 + i]);
  }
}
template <TgRows R>
__device__ __forceinline__ void tg_piece_get(uint32_t piece, uint32_t (&v)[16], int lane) {
  const int j = lane >> 3, r = lane & 7;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4];
    if (R == kRowsN) {
      tg_ldmatrix<true>(piece + tg_piece_at(8 * i + r, j), w);
#pragma unroll
      for (int b = 0; b < 4; ++b) v[4 * i + b] = w[b];
    } else {
      tg_ldmatrix<false>(piece + tg_piece_at(8 * i + r, j), w);
#pragma unroll
      for (int b = 0; b < 4; ++b) v[4 * b + i] = w[b];
    }
  }
}

// Copies a piece to / from `rows` global rows (2-byte elements, pitch ld, every
// row 16-byte aligned) of which the first `cols` columns (a multiple of 8) exist.
__device__ __forceinline__ void tg_piece_out(uint32_t piece, void* g, long long ld, int rows, int cols, int lane) {
  const int c = lane & 3;
  uint16_t* at = reinterpret_cast<uint16_t*>(g) + (lane >> 2) * ld + c * 8;
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = tg_lds16(piece + tg_piece_at(i * 8 + (lane >> 2), c));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i * 8 + (lane >> 2) < rows && c * 8 < cols) *reinterpret_cast<uint4*>(at + i * 8 * ld) = w[i];
}
__device__ __forceinline__ void tg_piece_in(uint32_t piece, const void* g, long long ld, int rows, int cols, int lane) {
  const int c = lane & 3;
  const uint16_t* at = reinterpret_cast<const uint16_t*>(g) + (lane >> 2) * ld + c * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i * 8 + (lane >> 2);
    if (row < rows && c * 8 < cols) ptx::cp_async_16(piece + tg_piece_at(row, c), at + i * 8 * ld);
  }
}
// A piece as one TMA store (its place order is the 64-byte swizzle), clipped at
// the tensor's ends. The piece's shared memory is in use until tg_bulk_read.
__device__ __forceinline__ void tg_bulk_store(uint32_t piece, const CUtensorMap* m, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(piece), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void tg_piece_bulk(uint32_t piece, const CUtensorMap* m, int c0, int c1, int c2, int lane) {
  ptx::fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    tg_bulk_store(piece, m, c0, c1, c2);
    ptx::bulk_commit();
  }
}
__device__ __forceinline__ void tg_bulk_read(int lane) {
  if (lane == 0) ptx::bulk_wait_read_all();
  __syncwarp();
}
// The same for rows of any alignment and length.
__device__ __forceinline__ void tg_piece_out_any(uint32_t piece, uint16_t* g, long long ld, int rows, int cols, int lane) {
  if (lane >= cols) return;
  for (int row = 0; row < rows; ++row) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(piece + tg_piece_at(row, lane >> 3) + (lane & 7) * 2) : "memory");
    g[row * ld + lane] = v;
  }
}

template <typename T>
__device__ __forceinline__ void tg_pack(const uint32_t (&r)[2][16], uint32_t (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      v[4 * i + b] = TgPair<T>::pack(__uint_as_float(r[b >> 1][4 * i + 2 * (b & 1)]),
                                     __uint_as_float(r[b >> 1][4 * i + 2 * (b & 1) + 1]));
}

// Pieces a warp keeps in shared memory: all of its share of a tile when the
// epilogue reads, so that a tile's whole input is on its way before its MMAs end
// (with two, the wait for each third and fourth piece took longer than the piece).
template <int Epi>
__host__ __device__ constexpr int tg_slots(bool residual) {
  return Epi == kTgPlain ? 2 : Epi == kTgGram || (Epi == kTgStore && !residual) ? 1 : 4;
}
template <int Epi>
__host__ __device__ constexpr int tg_epi_bytes(bool residual) { return kTgEpiWarps * kTgPiece * tg_slots<Epi>(residual); }

// X is carried as an fp16 value, which the products read, and 8 bits more: the
// difference of the fp32 pattern from the fp16 value's, in units of 2^-18 of the
// value. Together 19 bits, so that a X keeps small singular directions beside
// large ones at 3 bytes an entry. The 8 bits never leave this epilogue and lie
// in the order its threads hold them: a piece is 32 lanes x 32 bytes.
__device__ __forceinline__ int tg_low(float x, float h) { return (__float_as_int(x) - __float_as_int(h)) >> 5; }
// Four of them as bytes (saturated: a tie rounded down leaves +128, and below fp16's normal numbers, 2^-27 of X,
// more).
__device__ __forceinline__ uint32_t tg_low4(int a, int b, int c, int d) {
  uint32_t hi, all;
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(hi) : "r"(d), "r"(c));
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(all) : "r"(b), "r"(a), "r"(hi));
  return all;
}
// hi: two fp16 whose low bits are bytes 2 half and 2 half + 1 of w; the dot product with 32 at one byte
// extends its sign, scales and adds it in one instruction
__device__ __forceinline__ float2 tg_wide(uint32_t hi, uint32_t w, int half) {
  const float2 f = TgPair<__half>::unpack(hi);
  return make_float2(__int_as_float(__dp4a((int)w, half ? 0x200000 : 0x20, __float_as_int(f.x))),
                     __int_as_float(__dp4a((int)w, half ? 0x20000000 : 0x2000, __float_as_int(f.y))));
}
// a x + b y for two values at once
__device__ __forceinline__ float2 tg_axpby(float a, float2 x, float b, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, x, y;\n\t"
      "mov.b64 a, {%2, %2};\n\tmov.b64 b, {%3, %3};\n\tmov.b64 x, {%4, %5};\n\tmov.b64 y, {%6, %7};\n\t"
      "mul.rn.f32x2 y, b, y;\n\tfma.rn.f32x2 y, a, x, y;\n\tmov.b64 {%0, %1}, y;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a), "f"(b), "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

template <int Epi, typename T>
__device__ __forceinline__ void tg_prefetch(uint32_t slot, const TgParams& p, const TgTask& k, int c, int m, int lane) {
  const int row0 = k.n0 + c * 32, nrow = k.cols - c * 32, mcol = p.M - m;
  if (mcol > 0) {
    if (Epi == kTgStore) {
      tg_piece_in(slot, reinterpret_cast<const T*>(p.res) + (long long)row0 * p.ldr + m, p.ldr, nrow, mcol, lane);
    } else if (Epi == kTgPoly) {   // rows of A (m), whose pitch reaches past the last column
      tg_piece_in(slot, p.in + k.g * p.in_bs + (long long)m * p.ldi + row0, p.ldi, mcol, 32, lane);
    } else if (Epi == kTgUpdate || Epi == kTgUpdateOut) {
      tg_piece_in(slot, p.in + k.g * p.in_bs + (long long)row0 * p.ldi + m, p.ldi, nrow, 32, lane);
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// The low bits of one piece (k.n0 and m are multiples of 32).
__device__ __forceinline__ long long tg_low_at(const TgParams& p, const TgTask& k, int c, int m, int lane) {
  return k.g * p.lo_bs + ((long long)((k.n0 >> 5) + c) * (p.ldi >> 5) + (m >> 5)) * 1024 + lane * 32;
}

// One piece, first half: from its accumulator r and its inputs in `slot` (landed)
// to the packed result v (and lo, the lower half of X). m is the piece's first
// column of the output, bias[b] belongs to m + 8 b + lane / 4.
template <int Epi, typename T>
__device__ __forceinline__ void tg_piece_value(uint32_t slot, uint32_t (&r)[2][16], uint32_t (&v)[16],
                                               uint32_t (&lo)[8], const TgParams& p, const TgTask& k, int c, int m,
                                               int lane, const float (&bias)[4], float ca, float cb,
                                               float diagonal) {
  if (Epi == kTgStore) {
    uint32_t res[16];
    if (p.res != nullptr) tg_piece_get<kRowsN>(slot, res, lane);
    if (p.bias != nullptr) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t* e = &r[b >> 1][4 * i + 2 * (b & 1)];
          e[0] = __float_as_uint(__uint_as_float(e[0]) + bias[b]);
          e[1] = __float_as_uint(__uint_as_float(e[1]) + bias[b]);
        }
    }
    if (p.z != nullptr) {
      const int row0 = k.n0 + c * 32;
      tg_pack<T>(r, v);
      tg_bulk_read(lane);
      tg_piece_put<kRowsN>(slot, v, lane);
      __syncwarp();
      tg_piece_out(slot, reinterpret_cast<T*>(p.z) + (long long)row0 * p.ldz + m, p.ldz, k.cols - c * 32, p.M - m,
                   lane);
    }
    tg_act_all(r, p.act);
    if (p.res != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float2 f = TgPair<T>::unpack(res[4 * i + b]);
          uint32_t* e = &r[b >> 1][4 * i + 2 * (b & 1)];
          e[0] = __float_as_uint(__uint_as_float(e[0]) + f.x);
          e[1] = __float_as_uint(__uint_as_float(e[1]) + f.y);
        }
    }
    tg_pack<T>(r, v);
  } else if (Epi == kTgGram || Epi == kTgPoly) {
    if (Epi == kTgPoly) tg_piece_get<kRowsM>(slot, v, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t* e = &r[b >> 1][4 * i + 2 * (b & 1)];
        float x = cb * __uint_as_float(e[0]), y = cb * __uint_as_float(e[1]);
        if (Epi == kTgPoly) {
          const float2 f = TgPair<__half>::unpack(v[4 * i + b]);
          x += ca * f.x;
          y += ca * f.y;
          if (i == b && m == k.n0 + c * 32) {
            if ((lane >> 2) == 2 * (lane & 3)) x += diagonal;
            if ((lane >> 2) == 2 * (lane & 3) + 1) y += diagonal;
          }
        }
        v[4 * i + b] = TgPair<__half>::pack(x, y);
      }
  } else {
    tg_piece_get<kRowsN>(slot, v, lane);
#pragma unroll
    for (int j = 0; j < 16; j += 2) {   // two 8 x 8 blocks: four values, one word of low bits
      int q[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = (j + h) >> 2, b = (j + h) & 3;
        const uint32_t* e = &r[b >> 1][4 * i + 2 * (b & 1)];
        const float2 x = tg_axpby(ca, tg_wide(v[j + h], lo[j >> 1], h), cb,
                                  make_float2(__uint_as_float(e[0]), __uint_as_float(e[1])));
        if (Epi == kTgUpdate) {
          v[j + h] = TgPair<__half>::pack(x.x, x.y);
          const float2 n = TgPair<__half>::unpack(v[j + h]);
          q[2 * h] = tg_low(x.x, n.x);
          q[2 * h + 1] = tg_low(x.y, n.y);
        } else {
          v[j + h] = TgPair<bf16>::pack(x.x, x.y);
        }
      }
      if (Epi == kTgUpdate) lo[j >> 1] = tg_low4(q[0], q[1], q[2], q[3]);
    }
  }
}

// Second half: through `slot` to the output.
template <int Mode, int Epi, typename T>
__device__ __forceinline__ void tg_piece_store(uint32_t slot, const uint32_t (&v)[16], const uint32_t (&lo)[8],
                                               const TgParams& p, const TgTask& k, int c, int m, int lane, long long low_at) {
  const int row0 = k.n0 + c * 32, nrow = k.cols - c * 32, mcol = p.M - m;
  if (Epi == kTgUpdate && mcol > 0 && nrow > 0) {
    uint4* at = reinterpret_cast<uint4*>(p.lo_out + low_at);
    at[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    at[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
  }
  tg_bulk_read(lane);   // the slot's last piece has been read (and every lane is done with its input)
  if (Epi == kTgGram || Epi == kTgPoly) {
    // A = X X^T and B = b A + c A A are symmetric: the piece goes out as it lies (rows m) and, off the
    // diagonal tiles, transposed to the mirrored place
    if (mcol <= 0) return;
    tg_piece_put<kRowsM>(slot, v, lane);
    tg_piece_bulk(slot, &p.tm_out, row0, m, k.g, lane);
    if (k.mirror) {
      tg_bulk_read(lane);
      tg_piece_put<kRowsN>(slot, v, lane);
      tg_piece_bulk(slot, &p.tm_out, m, row0, k.g, lane);
    }
    return;
  }
  if (mcol <= 0 || nrow <= 0) return;
  if (Epi == kTgUpdateOut) {
    if (p.transposed) tg_piece_put<kRowsM>(slot, v, lane);
    else tg_piece_put<kRowsN>(slot, v, lane);
    __syncwarp();
    const int rows = p.transposed ? mcol : nrow, cols = p.transposed ? nrow : mcol;
    bf16* o = reinterpret_cast<bf16*>(p.out) + k.g * p.out_bs +
              (p.transposed ? (long long)m * p.ldo + row0 : (long long)row0 * p.ldo + m);
    // the row's length is a multiple of 8 where the rest of it from here is
    if (p.ldo % 8 == 0 && cols % 8 == 0 && (reinterpret_cast<uintptr_t>(o) & 15) == 0)
      tg_piece_out(slot, o, p.ldo, rows, cols, lane);
    else
      tg_piece_out_any(slot, reinterpret_cast<uint16_t*>(o), p.ldo, min(rows, 32), cols, lane);
    __syncwarp();
    return;
  }
  tg_piece_put<kRowsN>(slot, v, lane);
  if (Mode == kTgRaggedN && nrow < 32 && row0 + nrow != p.N) {   // the group ends inside the piece
    __syncwarp();
    tg_piece_out(slot, reinterpret_cast<T*>(p.out) + (long long)row0 * p.ldo + m, p.ldo, nrow, mcol, lane);
    __syncwarp();
  } else {
    tg_piece_bulk(slot, &p.tm_out, m, row0, Mode == kTgRaggedN ? 0 : k.g, lane);
  }
}

// The accumulator alone, two pieces at a time: half as many waits and fences,
// which weigh as much as the stores where a tile's reduction is short (a weight
// gradient of 256 rows has four k blocks and writes 128 KB): 32768 rows in 128
// uneven groups of 2048 x 768 182 us instead of 188, of which writing 403 MB is
// 104 by itself.
template <int Mode, typename T>
__device__ void tg_epilogue_plain(const TgParams& p, TgSmem& s, TgState& at, uint32_t store, uint32_t tmem, uint32_t rank,
                                  int warp) {
  constexpr int kParts = kTgEpiWarps / 4;
  const int lane = ptx::lane_id();
  const int quad = warp & 3, part = (warp - 4) >> 2;
  const uint32_t leader_empty0 = ptx::mapa(ptx::smem_u32(&s.acc_empty[0]), 0);
  const uint32_t slot = store + (warp - 4) * 2 * kTgPiece;
  TgTask k, next;
  bool more = at.list.next(k, p, s);
  while (more) {
    const bool any = k.klen > 0;
    const int m = k.m0 + (int)rank * 128 + quad * 32;
    const uint32_t from = tmem + at.acc * 256 + ((uint32_t)(quad * 32) << 16);
    uint32_t r[2][2][16];   // [piece]
    auto fetch = [&](int c) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if ((2 * c + h) * 32 < k.nt) {
          tg_tmem_frag(from + (2 * c + h) * 32, r[h][0]);
          tg_tmem_frag(from + (2 * c + h) * 32 + (16u << 16), r[h][1]);
        }
    };
    if (any) {
      if (!tg_wait_warp(&s.acc_full[at.acc], at.acc_phase, p, s)) break;
      ptx::tc_fence_after();
      fetch(part);
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) r[i >> 5][(i >> 4) & 1][i & 15] = 0;
    }
    more = at.list.next(next, p, s);
#pragma unroll 1
    for (int c = part; c * 64 < k.nt; c += kParts) {
      const bool again = (c + kParts) * 64 < k.nt;
      if (any) ptx::tmem_ld_wait();
      uint32_t v[2][16];
      tg_pack<T>(r[0], v[0]);
      tg_pack<T>(r[1], v[1]);
      if (any) {
        if (again) {
          fetch(c + kParts);
        } else {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_peer(leader_empty0 + at.acc * 8);
        }
      }
      if (m >= p.M) continue;
      tg_bulk_read(lane);
      tg_piece_put<kRowsN>(slot, v[0], lane);
      tg_piece_put<kRowsN>(slot + kTgPiece, v[1], lane);
      ptx::fence_proxy_async_shared();
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row0 = k.n0 + (2 * c + h) * 32, nrow = k.cols - (2 * c + h) * 32;
        if (nrow <= 0) break;
        if (Mode == kTgRaggedN && nrow < 32 && row0 + nrow != p.N)   // the group ends inside the piece
          tg_piece_out(slot + h * kTgPiece, reinterpret_cast<T*>(p.out) + (long long)row0 * p.ldo + m, p.ldo, nrow,
                       p.M - m, lane);
        else if (lane == 0)
          tg_bulk_store(slot + h * kTgPiece, &p.tm_out, m, row0, Mode == kTgRaggedN ? 0 : k.g);
      }
      if (lane == 0) ptx::bulk_commit();
      __syncwarp();
    }
    if (any) {
      if (part * 64 >= k.nt && lane == 0) ptx::mbar_arrive_peer(leader_empty0 + at.acc * 8);
      at.next_acc();
    }
    k = next;
  }
  if (lane == 0) ptx::bulk_wait_all();
  __syncwarp();
}

// The accumulator of the next piece (and its low bits of X) is on its way while
// a piece is stored, and the accumulator buffer is given back before the last
// piece is.
template <int Mode, int Epi, typename T>
__device__ void tg_epilogue(const TgParams& p, TgSmem& s, TgState& at, uint32_t store, uint32_t tmem, uint32_t rank,
                            int warp) {
  const TgFactors& f = p.factors;
  constexpr bool kWide = Epi == kTgUpdate || Epi == kTgUpdateOut;
  constexpr int kParts = kTgEpiWarps / 4;   // warps that share a quarter of the lanes, every kParts-th piece each
  const int lane = ptx::lane_id();
  const int quad = warp & 3, part = (warp - 4) >> 2;
  const uint32_t leader_empty0 = ptx::mapa(ptx::smem_u32(&s.acc_empty[0]), 0);
  const bool reads = Epi == kTgPoly || kWide || (Epi == kTgStore && p.res != nullptr);
  const uint32_t base = store + (warp - 4) * kTgPiece * tg_slots<Epi>(p.res != nullptr);
  TgTask k, next;
  bool more = at.list.next(k, p, s);
  while (more) {
    const bool any = k.klen > 0;
    const int m = k.m0 + (int)rank * 128 + quad * 32;
    uint32_t slot = base;
    if (reads) {
      tg_bulk_read(lane);
#pragma unroll
      for (int c = 0; c < 8 / kParts; ++c)   // one group each, empty past the tile
        if ((part + kParts * c) * 32 < k.nt) tg_prefetch<Epi, T>(base + c * kTgPiece, p, k, part + kParts * c, m, lane);
        else asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    float alpha = 1.f;
    if (Epi == kTgStore) {
      if (p.bias != nullptr)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (m + 8 * b < p.M) bias[b] = (float)reinterpret_cast<const T*>(p.bias)[m + 8 * b + (lane >> 2)];
    } else if (f.alpha != nullptr) {
      alpha = f.alpha[k.g];
    }
    const float ca = kWide ? f.ca * alpha : f.ca, cb = kWide ? f.cb * alpha : f.cb * alpha * alpha;
    const bool low = kWide && f.lo_in != nullptr && m < p.M;
    uint4 l0 = make_uint4(0, 0, 0, 0), l1 = l0;
    long long low_at = kWide ? tg_low_at(p, k, part, m, lane) : 0;
    const long long low_step = kWide ? (p.ldi >> 5) * (1024 * kParts) : 0;
    if (low && part * 32 < k.nt) {
      const uint4* from = reinterpret_cast<const uint4*>(f.lo_in + low_at);
      l0 = __ldcg(from);
      l1 = __ldcg(from + 1);
    }
    uint32_t r[2][16];
    const uint32_t from = tmem + at.acc * 256 + ((uint32_t)(quad * 32) << 16);
    if (any) {
      if (!tg_wait_warp(&s.acc_full[at.acc], at.acc_phase, p, s)) break;
      ptx::tc_fence_after();
      if (part * 32 < k.nt) {
        tg_tmem_frag(from + part * 32, r[0]);
        tg_tmem_frag(from + part * 32 + (16u << 16), r[1]);
      }
    }
    more = at.list.next(next, p, s);
#pragma unroll 1
    for (int c = part; c * 32 < k.nt; c += kParts) {
      const bool again = (c + kParts) * 32 < k.nt;
      if (reads) {
        switch (8 / kParts - 1 - c / kParts) {   // groups that may still be under way
          case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
          case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
          case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
          default: asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
      }
      uint32_t v[16], lo[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
      if (low && again) {
        const uint4* low_from = reinterpret_cast<const uint4*>(f.lo_in + low_at + low_step);
        l0 = __ldcg(low_from);
        l1 = __ldcg(low_from + 1);
      }
      if (any) {
        ptx::tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) r[0][i] = r[1][i] = 0;
      }
      tg_piece_value<Epi, T>(slot, r, v, lo, p, k, c, m, lane, bias, ca, cb, f.diagonal);
      if (any && again) {
        tg_tmem_frag(from + (c + kParts) * 32, r[0]);
        tg_tmem_frag(from + (c + kParts) * 32 + (16u << 16), r[1]);
      }
      if (any && !again) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_peer(leader_empty0 + at.acc * 8);
      }
      tg_piece_store<Mode, Epi, T>(slot, v, lo, p, k, c, m, lane, low_at);
      low_at += low_step;
      if (reads) slot += kTgPiece;
    }
    if (any) {
      if (part * 32 >= k.nt && lane == 0) ptx::mbar_arrive_peer(leader_empty0 + at.acc * 8);
      at.next_acc();
    }
    k = next;
  }
  ptx::cp_async_wait_all();
  if (lane == 0) ptx::bulk_wait_all();
  __syncwarp();
}

// ---------------------------------------------------------------- kernel
// Barriers and TMEM; the caller synchronises the cluster afterwards.
template <bool RaggedK>
__device__ __forceinline__ void tg_setup(TgSmem& s, int stages, uint32_t rank) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 1);
      ptx::mbar_init(&s.tail[i], 1);
      ptx::mbar_init(&s.peer_tail[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s.acc_full[i], 1);
      ptx::mbar_init(&s.acc_empty[i], 2 * kTgEpiWarps);
    }
    for (int i = 0; i < kTgRing; ++i) {
      ptx::mbar_init(&s.task_full[i], 1);
      // readers: the producer, the leader's MMA warp, the tail warp of a ragged reduction, the epilogue
      ptx::mbar_init(&s.task_empty[i], 1 + (rank == 0 ? 1 : 0) + (RaggedK ? 1 : 0) + kTgEpiWarps);
    }
    s.abort = 0;
    ptx::fence_mbar_init();
  }
  if ((threadIdx.x >> 5) == 3) {
    ptx::tmem_alloc_pair(&s.tmem_base, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
}

// One product, all roles: tiles first, first + step, ... below end.
template <int Mode, bool PMn, bool QMn, int Epi, typename T>
__device__ __forceinline__ void tg_product(const TgParams& p, TgSmem& s, uint8_t* tiles, uint32_t tmem, uint32_t rank,
                                           int warp, int first, int end, int step) {
  TgState at;
  const uint32_t base = ptx::smem_u32(tiles);
  // Warp 3 works its first tile out under the end of the previous kernel. The others touch global memory or
  // wait for those that do, and a bounded wait must not run while that kernel does: it may take any time.
  if (warp != 3) tg_after_stream();
  if (warp == 0) {
    tg_producer<Mode, PMn, QMn>(p, s, at, base, rank);
  } else if (warp == 1) {
    if (rank == 0) tg_mma<Mode, PMn, QMn>(p, s, at, base, tmem);
  } else if (warp == 2) {
    if (Mode == kTgRaggedK) tg_tail_warp<Mode>(p, s, at, tiles, rank);
  } else if (warp == 3) {
    tg_schedule<Mode>(p, s, at, first, end, step);
  } else {
    if (Epi == kTgPlain) tg_epilogue_plain<Mode, T>(p, s, at, base + p.stages * p.stage_bytes, tmem, rank, warp);
    else tg_epilogue<Mode, Epi, T>(p, s, at, base + p.stages * p.stage_bytes, tmem, rank, warp);
  }
  __syncwarp();
}

template <int Mode, bool PMn, bool QMn, int Epi, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTgThreads, 1)
    moe_tile_gemm_kernel(const __grid_constant__ TgParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TgSmem& s = *reinterpret_cast<TgSmem*>(tiles + (size_t)p.stages * p.stage_bytes + p.epi_bytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();

  tg_setup<Mode == kTgRaggedK>(s, p.stages, rank);
  if (threadIdx.x == 32) {
    ptx::prefetch_tmap(&p.tm_p);
    for (int i = 0; i < (QMn ? 1 : 4); ++i) ptx::prefetch_tmap(&p.tm_q[i]);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int mt = (p.M + 255) >> 8;
  if (Mode == kTgRaggedN || Mode == kTgRaggedK) {
    tg_after_stream();
    const int rows = Mode == kTgRaggedN ? p.N : p.K;
    for (int e = threadIdx.x; e < p.groups; e += kTgThreads) {
      int lo = p.offsets ? p.offsets[e] : 0, hi = p.offsets ? p.offsets[e + 1] : rows;
      if (lo < 0 || hi < lo || hi > rows) {
        tg_set_error(p, s, kDevBounds, false);
        lo = hi = 0;
      }
      s.start()[e] = lo;
      s.count(p.groups)[e] = hi - lo;
    }
  }
  __syncthreads();
  if (Mode == kTgRaggedK) {
    // The time of a tile goes with its group's rows, and all tiles of a group take the same: dealt from
    // the largest group to the smallest, forwards and backwards in turn, the pairs' shares differ less
    // (128 groups of 100 to 6000 rows: 6 % of the mean instead of 15 %). Ranks by counting, so only for
    // some hundred groups.
    const int* count = s.count(p.groups);
    int* order = s.order(p.groups);
    for (int e = threadIdx.x; e < p.groups; e += kTgThreads) {
      int rank_of = e;
      if (p.groups <= kTgSorted) {
        rank_of = 0;
        for (int f = 0; f < p.groups; ++f) rank_of += count[f] > count[e] || (count[f] == count[e] && f < e) ? 1 : 0;
      }
      order[rank_of] = e;
    }
  }
  if (Mode == kTgRaggedN) {
    if (warp == 0) {
      const int* count = s.count(p.groups);
      int* tile0 = s.tile0(p.groups);
      int run = 0;
      for (int b = 0; b < p.groups; b += 32) {
        const int e = b + lane;
        const int mine = e < p.groups ? (count[e] + p.nt - 1) / p.nt : 0;
        int sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += up;
        }
        if (e < p.groups) tile0[e] = run + sum - mine;
        run += __shfl_sync(0xffffffffu, sum, 31);
      }
      if (lane == 0) {
        tile0[p.groups] = run;
        s.total = run * mt;
      }
    }
  } else if (threadIdx.x == 0) {
    s.total = Mode == kTgSymmetric ? p.groups * (mt * (mt + 1) / 2) : p.groups * mt * ((p.N + p.nt - 1) / p.nt);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // both CTAs' barriers exist before any remote arrive
  ptx::tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  tg_product<Mode, PMn, QMn, Epi, T>(p, s, tiles, tmem, rank, warp, blockIdx.x >> 1, s.total, gridDim.x >> 1);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // no peer still arrives on this CTA's barriers or reads its tiles
  ptx::tc_fence_after();
  if (warp == 3) ptx::tmem_dealloc_pair(tmem, kTmemCols);
}

}  // namespace moe
