// bf16 products by expert for rows in a dispatch plan's order, and their
// gradients, on tcgen05 (sm_103a).  For the rows r of expert e
// (offsets[e] <= r < offsets[e+1]) and its N x K matrix W_e:
//
//   forward   D[r]  = act(alpha * A[r] * W_e^T)        rows x N, sum over K
//   rows      dA[r] = alpha * dD[r] * W_e              rows x K, sum over N
//   weights   dW_e  = alpha * dD_e^T * A_e + beta * C_e   N x K, sum over e's rows
//
// The row counts are read on the device: no call waits for them, and all of
// them may be captured.  What differs from a dense GEMM:
//
// - Tiles.  Each CTA (pair) reads the offsets, takes their running maximum
//   (so that the experts' rows are disjoint and inside the matrices whatever
//   the plan holds) and numbers the tiles of all experts by a prefix sum.
//   Tiles start at an expert's first row: a TMA box may start at any row.
//   Forward and rows: a tile's rows past the expert's last belong to the next
//   one; they only reach their own rows of the accumulator, which are not
//   stored.  Boxes of 32 rows that are all the expert's leave by TMA, others
//   row by row.  Rows that no expert has are written as zeros, by tiles
//   without k-blocks.
// - Operand order.  An operand whose summation index is its row index (W in
//   `rows`, both in `weights`) is loaded as it lies, as boxes of 64 columns x
//   64 rows, and is an "MN-major" operand of the MMA: nothing is transposed
//   in memory.
// - Ragged sums.  In `weights` an expert's last k-block holds rows of the next
//   expert.  The MMA takes 16 rows at a time; those past the last are left
//   out, and the ones inside the last 16 are zeroed in shared memory in both
//   operands (a NaN there must not meet a zero).  A warp of its own does that
//   between the TMA's completion and the MMA's start.
//
// Structure (one CTA per SM): warp 0 loads, warp 1 multiplies, warps 2..5
// store, warp 6 (weights only) passes stages on.  CG = 2 pairs two CTAs on a
// 256 x 256 tile, CG = 1 takes 128 x bn.  Accumulators are double buffered in
// Tensor Memory, so that a tile's epilogue runs beside the next one's loop.
//
// Every mbarrier wait is bounded by %globaltimer; one that gives up sets a
// CTA abort flag and the device status word, and all roles leave.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace gtn {

namespace {

constexpr int kBlockK = 64;                // summation indices per ring stage
constexpr int kChunkBytes = 64 * 128;      // 64 rows of 64 bf16: one box of an MN-major operand
constexpr int kEpiWarps = 4;
constexpr int kBoxBytes = 32 * 64;         // staged box of an output: 32 rows of 64 bytes
constexpr int kErrTimeout = -5;            // GEMM_ERR_TIMEOUT
constexpr int kMaxStages = 16;

template <int OP>
struct Shape {
  static constexpr bool kWeights = OP == kExpertsWeights;
  static constexpr bool kMnA = kWeights, kMnB = OP != kExpertsForward;
  static constexpr int kThreads = 32 * (2 + kEpiWarps + (kWeights ? 1 : 0));
};

// barriers: full, empty, ready per stage; accumulators; C boxes; the drain
constexpr int kBars = 3 * kMaxStages + 4 + kEpiWarps * kExpertsMaxBoxes + 1;

__host__ __device__ constexpr int table_bytes(int E) { return 4 * (2 * E + 4); }

struct Abort {
  volatile uint32_t* flag;
  uint64_t timeout_ns;
  int* status;
  int role;
};

template <bool CLUSTER>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  if constexpr (CLUSTER) return mbar_try_wait_cluster(bar, parity);
  else return mbar_try_wait(bar, parity);
}

template <bool CLUSTER>
__device__ __noinline__ bool wait_bar_slow(uint32_t bar, uint32_t parity, volatile uint32_t* flag, uint64_t timeout_ns,
                                           int* status, int role) {
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (try_wait<CLUSTER>(bar, parity)) return true;
    if (flag && *flag) return false;
    if (globaltimer() - t0 > timeout_ns) {
      if (flag) *flag = 1;
      if (atomicCAS(status, 0, kErrTimeout) == 0) atomicExch(status + 1, (role << 24) | (int)blockIdx.x);
      return false;
    }
  }
}

// Bounded wait on an mbarrier phase.  False if this CTA is aborting.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Abort& ab) {
  if (try_wait<CLUSTER>(bar, parity)) return true;
  return wait_bar_slow<CLUSTER>(bar, parity, ab.flag, ab.timeout_ns, ab.status, ab.role);
}

__device__ __noinline__ void settle(uint64_t ns) {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < ns) __nanosleep(1000);
}

// Descriptor of an MN-major operand in shared memory: chunks of 64 columns
// (128 bytes, 128-byte swizzle) by 64 summation indices, one row of a chunk
// per summation index.  PTX ISA, tcgen05 shared memory descriptor: the stride
// from one group of 8 summation indices to the next (1024 bytes) in bits
// 32-45, that from one chunk of columns to the next in bits 16-29.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kChunkBytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The experts' first rows (E + 1) and first tiles (E + 2: behind the experts
// the rows of nobody) of one launch, in shared memory.
struct Table {
  int* row;
  int* tile;
};

// Fills the table from the clamped offsets that lie in its rows: one warp, 32
// experts at a time.  tile_rows = 0: the rows only.
__device__ __forceinline__ void fill_table(const ExpertsParams& p, const Table& tb, int tile_rows) {
  const int lane = threadIdx.x & 31;
  int top = 0;            // running maximum of the offsets so far
  for (int e0 = 0; e0 <= p.E; e0 += 32) {
    const int e = e0 + lane;
    int v = e <= p.E ? tb.row[e] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v = max(v, o);
    }
    v = max(v, top);
    if (e <= p.E) tb.row[e] = v;
    top = __shfl_sync(0xffffffffu, v, 31);
  }
  __syncwarp();
  if (tile_rows == 0) return;
  int sum = 0;
  for (int e0 = 0; e0 <= p.E; e0 += 32) {
    const int e = e0 + lane;
    int n = 0;            // row blocks of expert e, or of the rows of nobody
    if (e <= p.E) n = ((e < p.E ? tb.row[e + 1] : p.R) - tb.row[e] + tile_rows - 1) / tile_rows;
    int v = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += o;
    }
    if (e <= p.E) tb.tile[e] = sum + v - n;
    sum += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) tb.tile[p.E + 1] = sum;
}

// One tile: its expert (E: the rows of nobody), its rows of the output
// [row0, row_end), its first column, and its sum's rows and blocks.
struct Tile {
  int e, row0, row_end, col0;
  int k0, k_end, num_kb;      // weights: the expert's rows; else 0 and the sum's length
};

template <int OP>
__device__ __forceinline__ Tile tile_of(int t, const ExpertsParams& p, const Table& tb, int tile_rows) {
  Tile r;
  int local, tiles_m;
  if constexpr (OP == kExpertsWeights) {
    const int per = p.tiles_m * p.tiles_n;
    r.e = t / per;
    local = t - r.e * per;
    tiles_m = p.tiles_m;
    r.k0 = tb.row[r.e];
    r.k_end = tb.row[r.e + 1];
    r.num_kb = (r.k_end - r.k0 + kBlockK - 1) / kBlockK;
  } else {
    // the last entry whose first row block is not past this one; entries
    // without rows share their first block with the next
    const int b = t / p.tiles_n;
    int lo = 0, hi = p.E;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tb.tile[mid] <= b) lo = mid;
      else hi = mid - 1;
    }
    r.e = lo;
    local = t - tb.tile[lo] * p.tiles_n;
    tiles_m = tb.tile[lo + 1] - tb.tile[lo];
    r.k0 = 0;
    r.k_end = p.S;
    r.num_kb = lo < p.E ? (p.S + kBlockK - 1) / kBlockK : 0;
  }
  // strips of p.strip row blocks, row blocks fastest within a strip
  const int strip = local / (p.strip * p.tiles_n);
  const int first = strip * p.strip, high = min(p.strip, tiles_m - first);
  const int in = local - first * p.tiles_n;
  const int tm = first + in % high;
  r.col0 = (in / high) * p.bn;
  if constexpr (OP == kExpertsWeights) {
    r.row0 = tm * tile_rows;
    r.row_end = p.rows_out;
  } else {
    r.row0 = tb.row[r.e] + tm * tile_rows;
    r.row_end = r.e < p.E ? tb.row[r.e + 1] : p.R;
  }
  return r;
}

// ---------------------------------------------------------------- epilogue pieces
// 16 or 32 values of this lane's row, to or from a staged box (64-byte rows,
// 64-byte swizzle: 16-byte chunk j of row l sits at j ^ ((l / 2) % 4)).
template <bool F32>
__device__ __forceinline__ void stage_row(uint32_t box, int lane, const float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t at = box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4);
    if constexpr (F32)
      st_shared_v4(at, __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                   __float_as_uint(v[4 * j + 3]));
    else
      st_shared_v4(at, pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                   pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
  }
}

template <bool F32>
__device__ __forceinline__ void add_staged_row(uint32_t box, int lane, float beta, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t x[4];
    ld_shared_v4(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), x[0], x[1], x[2], x[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        v[4 * j + i] = fmaf(beta, __uint_as_float(x[i]), v[4 * j + i]);
      } else {
        v[8 * j + 2 * i] = fmaf(beta, __uint_as_float(x[i] << 16), v[8 * j + 2 * i]);
        v[8 * j + 2 * i + 1] = fmaf(beta, __uint_as_float(x[i] & 0xFFFF0000u), v[8 * j + 2 * i + 1]);
      }
    }
  }
}

// Copies the first `rows` rows of a staged box to (or from) global memory
// element by element, a row (two rows for fp32) per step: neighbouring lanes
// move neighbouring elements.  Any alignment; columns past the last are left out.
template <bool F32, bool LOAD>
__device__ __forceinline__ void copy_rows(uint8_t* box, int lane, void* base, long long ld, int rows, int cols) {
  constexpr int kCols = F32 ? 16 : 32, kPerChunk = F32 ? 4 : 8, kBytes = F32 ? 4 : 2;
  const int c = lane % kCols;
  if (c >= cols) return;
  for (int i = lane / kCols; i < rows; i += 32 / kCols) {
    uint8_t* s = box + i * 64 + (((c / kPerChunk) ^ ((i >> 1) & 3)) << 4) + (c % kPerChunk) * kBytes;
    if constexpr (F32) {
      float* d = static_cast<float*>(base) + i * ld + c;
      if constexpr (LOAD) *reinterpret_cast<float*>(s) = *d;
      else *d = *reinterpret_cast<const float*>(s);
    } else {
      uint16_t* d = static_cast<uint16_t*>(base) + i * ld + c;
      if constexpr (LOAD) *reinterpret_cast<uint16_t*>(s) = *d;
      else *d = *reinterpret_cast<const uint16_t*>(s);
    }
  }
}

// One epilogue warp's place: its staging boxes, their barriers, and how many
// boxes it has used since the start (a box i uses buffer i % boxes).
struct Out {
  uint8_t* boxes;
  uint32_t sboxes, bars;
  int n;                   // buffers
  unsigned used, loaded;   // boxes stored, boxes of C asked for
};

// Element address of (row, col) of expert e's output or C.
__device__ __forceinline__ uint8_t* at(const void* base, long long ld, long long stride, int e, int row, int col,
                                       int bytes) {
  return const_cast<uint8_t*>(static_cast<const uint8_t*>(base)) + ((long long)e * stride + (long long)row * ld + col) * bytes;
}

template <int OP>
__device__ __forceinline__ void store_box(const CUtensorMap* m, int x, int y, int e, uint32_t src) {
  if constexpr (OP == kExpertsWeights) tma_store_3d(m, x, y, e, src);
  else tma_store_2d(m, x, y, src);
}

// The box of 32 rows x 64 bytes at (row, col) of the tile: beta * C, staging,
// store.  `rows` of its rows are to be stored.
template <int OP, bool F32>
__device__ __forceinline__ bool emit_box(const ExpertsParams& p, const CUtensorMap* tD, Out& o, int lane, int e,
                                         int row, int rows, int col, float* v, bool direct, const Abort& ab) {
  constexpr int kBytes = F32 ? 4 : 2;
  if (col >= p.cols_out) return true;
  const int b = (int)(o.used & (unsigned)(o.n - 1));
  const uint32_t sbox = o.sboxes + b * kBoxBytes;
  uint8_t* box = o.boxes + b * kBoxBytes;
  const int e_out = OP == kExpertsWeights ? e : 0;
  if (OP == kExpertsWeights && p.has_c) {
    if (direct) {
      __syncwarp();
      copy_rows<F32, true>(box, lane, at(p.C, p.ldc, p.stride_c, e_out, row, col, kBytes), p.ldc, rows, p.cols_out - col);
      __syncwarp();
    } else if (!__all_sync(0xffffffffu, wait_bar<false>(o.bars + 8u * b, (o.used / (unsigned)o.n) & 1u, ab))) {
      return false;
    }
    add_staged_row<F32>(sbox, lane, p.beta, v);
  } else {
    if (lane == 0) bulk_wait_read<1>();      // two buffers: this one's last store has read it
    __syncwarp();
  }
  stage_row<F32>(sbox, lane, v);
  if (direct) {
    __syncwarp();
    copy_rows<F32, false>(box, lane, at(p.D, p.ldd, p.stride_d, e_out, row, col, kBytes), p.ldd, rows, p.cols_out - col);
    __syncwarp();
    if (lane == 0) bulk_commit();            // an empty group: the buffers' count of groups stays in step
  } else {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      store_box<OP>(tD, col, row, e_out, sbox);
      bulk_commit();
    }
  }
  ++o.used;
  return true;
}

template <int CG, int OP>
__global__ void __launch_bounds__(Shape<OP>::kThreads, 1)
    gemm_experts_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmD,
                        const __grid_constant__ ExpertsParams p) {
  using S_ = Shape<OP>;
  constexpr bool kPair = CG == 2;
  constexpr int kTileRows = 128 * CG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // A's stages lie before B's: an MMA reads 128 rows of A also where fewer were
  // loaded, and what it finds there (in this CTA's memory, and only for rows
  // that are not stored) must not lie past the end.
  const uint32_t sA = smem_u32(smem);
  const uint32_t sB = sA + p.stages * p.a_bytes;
  uint8_t* boxes = smem + p.stages * (p.a_bytes + p.b_bytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(boxes + kEpiWarps * p.boxes * kBoxBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto ready_bar = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (3 * kMaxStages + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (3 * kMaxStages + 2 + b); };
  const uint32_t c_bars = bar0 + 8u * (3 * kMaxStages + 4);
  const uint32_t drain_bar = c_bars + 8u * kEpiWarps * kExpertsMaxBoxes;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  Table tb;
  tb.row = reinterpret_cast<int*>(tmem_slot + 2);
  tb.tile = tb.row + p.E + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const int first_tile = blockIdx.x / CG, step = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(ready_bar(s), CG);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), kEpiWarps * CG);
    }
    for (int b = 0; b < kEpiWarps * kExpertsMaxBoxes; ++b) mbar_init(c_bars + 8u * b, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    if (p.has_ab) {
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmB);
    }
    if (!p.direct) tma_prefetch_desc(&tmD);
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(tmem_slot), 2 * p.bn);
  // Inputs may come from the previous kernel on the stream: no global memory
  // access before this point.
  griddep_wait();
  griddep_launch_dependents();
  for (int e = threadIdx.x; e <= p.E; e += S_::kThreads) tb.row[e] = min(max(p.offsets[e], 0), p.R);
  __syncthreads();
  if (warp == 2) fill_table(p, tb, S_::kWeights ? 0 : kTileRows);
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int num_tiles = S_::kWeights ? p.E * p.tiles_m * p.tiles_n : tb.tile[p.E + 1] * p.tiles_n;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      Abort ab{abort_flag, p.timeout_ns, p.status, kRoleProducer};
      bool ok = true;
      int stage = 0;
      uint32_t phase = 0;
      const int b_cols = p.bn / CG;          // this CTA's share of the tile's columns
      const uint32_t tx = (uint32_t)(p.a_bytes + p.b_bytes);
      for (int t = first_tile; t < num_tiles && ok; t += step) {
        const Tile r = tile_of<OP>(t, p, tb, kTileRows);
        const int a_at = r.row0 + (int)rank * 128;
        const int b_at = r.col0 + (int)rank * b_cols;
        for (int kb = 0; kb < r.num_kb; ++kb) {
          if (!wait_bar<kPair>(empty_bar(stage), phase ^ 1, ab)) {
            ok = false;
            break;
          }
          const int k = r.k0 + kb * kBlockK;
          const uint32_t a = sA + stage * p.a_bytes, b = sB + stage * p.b_bytes;
          const uint32_t fb = full_bar(stage);
          if constexpr (S_::kWeights) {
            // each CTA's bytes on its own barrier: its warp 6 passes them on
            mbar_arrive_expect_tx(fb, tx);
            for (int c = 0; c < 2; ++c) tma_load_2d(a + c * kChunkBytes, &tmA, a_at + 64 * c, k, fb);
            for (int c = 0; c < b_cols / 64; ++c) tma_load_2d(b + c * kChunkBytes, &tmB, b_at + 64 * c, k, fb);
          } else {
            const uint32_t to = kPair ? mapa_shared(fb, 0) : fb;    // a pair's bytes all count on its leader's barrier
            if (leader) mbar_arrive_expect_tx(fb, tx * CG);
            if constexpr (kPair) tma_load_2d_pair(a, &tmA, k, a_at, to);
            else tma_load_2d(a, &tmA, k, a_at, to);
            if constexpr (S_::kMnB) {
              for (int c = 0; c < b_cols / 64; ++c) {
                if constexpr (kPair) tma_load_3d_pair(b + c * kChunkBytes, &tmB, b_at + 64 * c, k, r.e, to);
                else tma_load_3d(b + c * kChunkBytes, &tmB, b_at + 64 * c, k, r.e, to);
              }
            } else {
              if constexpr (kPair) tma_load_3d_pair(b, &tmB, k, b_at, r.e, to);
              else tma_load_3d(b, &tmB, k, b_at, r.e, to);
            }
          }
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) settle(2000000);   // copies already issued land before teardown
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0 && leader) {
      Abort ab{abort_flag, p.timeout_ns, p.status, kRoleMma};
      const uint32_t idesc = instr_desc_bf16_f32(kTileRows, p.bn) | (S_::kMnA ? 1u << 15 : 0u) | (S_::kMnB ? 1u << 16 : 0u);
      bool ok = true;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      for (int t = first_tile; t < num_tiles && ok; t += step) {
        const Tile r = tile_of<OP>(t, p, tb, kTileRows);
        if (!wait_bar<kPair>(acce_bar(acc), acc_phase ^ 1, ab)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * p.bn);
        for (int kb = 0; kb < r.num_kb; ++kb) {
          if (!wait_bar<kPair>(S_::kWeights ? ready_bar(stage) : full_bar(stage), phase, ab)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = sA + stage * p.a_bytes, b = sB + stage * p.b_bytes;
          const uint64_t a0 = S_::kMnA ? desc_mn(a) : smem_desc_sw128(a);
          const uint64_t b0 = S_::kMnB ? desc_mn(b) : smem_desc_sw128(b);
          // 16 summation indices are 32 bytes of a K-major operand's rows, 2048 of an MN-major operand
          constexpr uint64_t kStepA = S_::kMnA ? 128 : 2, kStepB = S_::kMnB ? 128 : 2;
          const int steps = S_::kWeights ? (min(kBlockK, r.k_end - r.k0 - kb * kBlockK) + 15) / 16 : 4;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < steps)
              mma_issue<CG, kKindF16>(d_tmem, a0 + kStepA * i, b0 + kStepB * i, idesc, (kb != 0 || i != 0) ? 1u : 0u);
          if constexpr (kPair) mma_commit_pair(empty_bar(stage), 0x3);
          else mma_commit(empty_bar(stage));
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if constexpr (kPair) mma_commit_pair(accf_bar(acc), 0x3);
        else mma_commit(accf_bar(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      // All MMAs issued by this thread complete before TMEM is released.
      if constexpr (kPair) mma_commit_pair(drain_bar, 0x1);
      else mma_commit(drain_bar);
      Abort ab_drain{nullptr, p.timeout_ns, p.status, kRoleMma};
      wait_bar<kPair>(drain_bar, 0, ab_drain);
    }
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const int ew = warp - 2;
    const int q = warp & 3;               // TMEM lane quarter this warp may access
    Abort ab{abort_flag, p.timeout_ns, p.status, kRoleEpilogue};
    Out o;
    o.boxes = boxes + ew * p.boxes * kBoxBytes;
    o.sboxes = smem_u32(o.boxes);
    o.bars = c_bars + 8u * (ew * kExpertsMaxBoxes);
    o.n = p.boxes;
    o.used = o.loaded = 0;
    const int box_cols = p.out_f32 ? 16 : 32;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    const uint32_t acce_target = kPair ? mapa_shared(acce_bar(0), 0) : acce_bar(0);
    for (int t = first_tile; t < num_tiles && ok; t += step) {
      const Tile r = tile_of<OP>(t, p, tb, kTileRows);
      const int row = r.row0 + (int)rank * 128 + q * 32;
      const int rows = min(32, r.row_end - row);       // of this warp's 32
      const bool direct = p.direct || (OP != kExpertsWeights && rows < 32);
      const int cols = min(p.bn, p.cols_out - r.col0);
      const unsigned end = o.used + (rows > 0 ? (unsigned)((cols + box_cols - 1) / box_cols) : 0u);
      const unsigned begin = o.used;
      // boxes of C, asked for as their buffers become free
      auto ask = [&](unsigned upto) {
        for (; o.loaded < upto; ++o.loaded) {
          const int b = (int)(o.loaded & (unsigned)(o.n - 1));
          mbar_arrive_expect_tx(o.bars + 8u * b, kBoxBytes);
          tma_load_3d(o.sboxes + b * kBoxBytes, &tmC, r.col0 + (int)(o.loaded - begin) * box_cols, row, r.e, o.bars + 8u * b);
        }
      };
      const bool ask_c = OP == kExpertsWeights && p.has_c && !p.direct && rows > 0;
      if (ask_c && lane == 0) {
        bulk_wait_read<0>();
        o.loaded = o.used;
        ask(min(end, o.used + (unsigned)o.n));
      }
      // (the whole warp leaves, or none of it: what follows is warp-wide)
      ok = __all_sync(0xffffffffu, wait_bar<kPair>(accf_bar(acc), acc_phase, ab));
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < p.bn; c += 32) {
        float v[32];
        if (rows > 0 && r.num_kb > 0 && c < cols) {
          uint32_t x[32];
          tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * p.bn + c), x);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = p.alpha * __uint_as_float(x[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        }
        if (c + 32 >= p.bn) {
          // accumulator fully read: hand it back to the MMA warp
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPair) mbar_arrive_cluster(acce_target + 8u * acc);
            else mbar_arrive(acce_bar(acc));
          }
        }
        if (rows <= 0 || c >= cols) continue;
        if constexpr (OP == kExpertsForward) activate_chunk(v, p.act);
        const int col = r.col0 + c;
        if (p.out_f32) {
          ok = emit_box<OP, true>(p, &tmD, o, lane, r.e, row, rows, col, v, direct, ab) &&
               emit_box<OP, true>(p, &tmD, o, lane, r.e, row, rows, col + 16, v + 16, direct, ab);
        } else {
          ok = emit_box<OP, false>(p, &tmD, o, lane, r.e, row, rows, col, v, direct, ab);
        }
        if (ask_c && lane == 0 && ok) {
          bulk_wait_read<1>();      // all stores but the last have read their buffers
          ask(min(end, o.used - 1 + (unsigned)o.n));
        }
        if (!ok) break;
      }
      ok = __all_sync(0xffffffffu, ok && !*abort_flag);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (lane == 0) {
      bulk_wait<0>();
      if (!ok && p.has_c) settle(1000000);   // boxes of C that were asked for land before teardown
    }
  } else if constexpr (S_::kWeights) {
    // ------------------------------------------------------------ stages passed on
    Abort ab{abort_flag, p.timeout_ns, p.status, kRoleProducer};
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const int chunks_b = p.bn / CG / 64;
    for (int t = first_tile; t < num_tiles && ok; t += step) {
      const Tile r = tile_of<OP>(t, p, tb, kTileRows);
      for (int kb = 0; kb < r.num_kb; ++kb) {
        ok = __all_sync(0xffffffffu, wait_bar<kPair>(full_bar(stage), phase, ab));
        if (!ok) break;
        const int valid = min(kBlockK, r.k_end - r.k0 - kb * kBlockK);
        const int bad = (16 - (valid & 15)) & 15;      // rows of the last MMA that are another expert's
        if (bad) {
          const uint32_t a = sA + stage * p.a_bytes, b = sB + stage * p.b_bytes;
          for (int i = lane; i < (2 + chunks_b) * bad * 8; i += 32) {
            const int chunk = i / (bad * 8), in = i - chunk * (bad * 8);
            const uint32_t base = chunk < 2 ? a + chunk * kChunkBytes : b + (chunk - 2) * kChunkBytes;
            st_shared_v4(base + (valid + in / 8) * 128 + (in % 8) * 16, 0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair) mbar_arrive_cluster(mapa_shared(ready_bar(stage), 0));
          else mbar_arrive(ready_bar(stage));
        }
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  }

  __syncthreads();
  if constexpr (kPair) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem_base, 2 * p.bn);
  }
}

const void* kernel_for(int cg, int op) {
  static const void* const table[2][3] = {
      {(const void*)gemm_experts_kernel<1, kExpertsForward>, (const void*)gemm_experts_kernel<1, kExpertsRows>,
       (const void*)gemm_experts_kernel<1, kExpertsWeights>},
      {(const void*)gemm_experts_kernel<2, kExpertsForward>, (const void*)gemm_experts_kernel<2, kExpertsRows>,
       (const void*)gemm_experts_kernel<2, kExpertsWeights>}};
  return table[cg - 1][op];
}

constexpr int kSmemMax = 232448;

int smem_bytes(const ExpertsParams& p) {
  return 1024 + p.stages * (p.a_bytes + p.b_bytes) + kEpiWarps * p.boxes * kBoxBytes + kBars * 8 + 8 + table_bytes(p.E);
}

}  // namespace

// Tile shape and ring of a call (see the header of kernels.h): cg, bn, a_rows
// and from them stages and the stages' bytes.
void experts_geometry(ExpertsParams* p, int sms) {
  const bool weights = p->op == kExpertsWeights;
  if (weights) {
    p->cg = 2;
    p->bn = 256;
    p->a_rows = 64;
  } else {
    const int active = p->E < p->R ? p->E : p->R;
    if (active > 0 && p->R / active >= 96) {
      p->cg = 2;
      p->bn = 256;
    } else {
      p->cg = 1;
      p->bn = 256;
      while (p->bn > 64 && (long long)active * ((p->cols_out + p->bn - 1) / p->bn) * 2 <= sms) p->bn /= 2;
    }
    p->a_rows = p->R >= 128 || p->cg == 2 ? 128 : (p->R + 7) / 8 * 8;
    if (p->a_rows == 0) p->a_rows = 8;
  }
  p->a_bytes = weights ? 2 * kChunkBytes : p->a_rows * 128;
  p->b_bytes = p->bn / p->cg * 128;
  p->boxes = weights && p->has_c ? kExpertsMaxBoxes : 2;
  const int left = kSmemMax - (smem_bytes(*p) - p->stages * (p->a_bytes + p->b_bytes));
  p->stages = left / (p->a_bytes + p->b_bytes);
  if (p->stages > kMaxStages) p->stages = kMaxStages;
}

cudaError_t launch_experts(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmC, const CUtensorMap& tmD,
                           ExpertsParams p, int sms, cudaStream_t stream, LaunchInfo* info) {
  static bool configured[64] = {};
  static int pairs[64][3] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const void* kern = kernel_for(p.cg, p.op);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cg;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(p.op == kExpertsWeights ? Shape<kExpertsWeights>::kThreads : Shape<kExpertsForward>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes(p);
  cfg.stream = stream;
  cfg.attrs = attr;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    for (int op = 0; op < 3; ++op) {
      for (int cg = 1; cg <= 2; ++cg)
        if ((e = cudaFuncSetAttribute(kernel_for(cg, op), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax)))
          return e;
      cudaLaunchConfig_t c2 = cfg;
      cudaLaunchAttribute pair = attr[0];
      pair.val.clusterDim.x = 2;
      c2.gridDim = dim3(2);
      c2.blockDim = dim3(op == kExpertsWeights ? Shape<kExpertsWeights>::kThreads : Shape<kExpertsForward>::kThreads);
      c2.dynamicSmemBytes = kSmemMax;
      c2.attrs = &pair;
      c2.numAttrs = 1;
      int n = 0;
      if ((e = cudaOccupancyMaxActiveClusters(&n, kernel_for(2, op), &c2))) return e;
      pairs[dev][op] = n;
    }
    configured[dev] = true;
  }
  const int most = p.cg == 2 ? pairs[dev][p.op] : sms;
  if (most < 1) return cudaErrorInvalidConfiguration;
  // Tiles: known for the weights' gradient; else the most that the rows can
  // make, each expert and the rows of nobody ending with one part tile.
  const int tile_rows = 128 * p.cg;
  const long long tiles = p.op == kExpertsWeights
                              ? (long long)p.E * p.tiles_m * p.tiles_n
                              : ((long long)p.R / tile_rows + (p.E + 1 < p.R ? p.E + 1 : p.R)) * p.tiles_n;
  const int units = (int)(tiles < most ? tiles : most);
  cfg.gridDim = dim3(units * p.cg);
  cfg.numAttrs = 2;
  *info = LaunchInfo{};
  info->grid = units * p.cg;
  info->cluster = p.cg;
  info->block = cfg.blockDim.x;
  info->tile_m = tile_rows;
  info->tile_n = p.bn;
  info->stages = p.stages;
  info->smem_bytes = cfg.dynamicSmemBytes;
  info->k_parts = 1;
  info->scheduler = 1;
  static const char* const names[3] = {"gemm_experts_kernel<forward>", "gemm_experts_kernel<rows>",
                                       "gemm_experts_kernel<weights>"};
  info->kernel = names[p.op];
  void* args[5] = {const_cast<CUtensorMap*>(&tmA), const_cast<CUtensorMap*>(&tmB), const_cast<CUtensorMap*>(&tmC),
                   const_cast<CUtensorMap*>(&tmD), &p};
  return cudaLaunchKernelExC(&cfg, kern, args);
}

}  // namespace gtn
