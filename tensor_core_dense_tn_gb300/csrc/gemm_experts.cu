// bf16 products by expert for rows in a dispatch plan's order, and their
// gradients, on tcgen05 (sm_103a).  For the rows r of expert e
// (offsets[e] <= r < offsets[e+1]) and its N x K matrix W_e:
//
//   forward   D[r]  = act(alpha * A[r] * W_e^T)           R x N, sums over K
//   rows      dA[r] = alpha * dD[r] * W_e                 R x K, sums over N
//   weights   dW_e  = alpha * dD_e^T * A_e + beta * C_e   N x K, sums over e's rows
//
// The row counts are read on the device: no call waits for them, and all of
// them may be captured.  What differs from a dense GEMM:
//
// - The output's columns are the MMA's M (lanes of Tensor Memory), its rows
//   the MMA's N.  N may be any multiple of 16 (32 for a pair), so that an
//   expert's last tile computes at most 15 (31) rows too many, and a decode
//   step's few rows cost as few columns; with the rows as M, 512 rows an
//   expert in tiles of 256 computed a quarter more than they had to.  A lane
//   then holds one column of the output and neighbouring lanes neighbouring
//   columns: the epilogue stores (and reads C) straight from registers, row by
//   row, whatever the alignment, and leaves out the rows past the expert's last.
// - Tiles.  Each CTA (pair) reads the offsets, takes their running maximum
//   (so that the experts' rows are disjoint and inside the matrices whatever
//   the plan holds) and numbers the tiles of all experts by a prefix sum.  An
//   expert's rows are cut into equal tiles of at most 256.  Tiles start at
//   any row, and so may a TMA box; rows of the next expert that a box brings
//   along only reach columns of the accumulator that are not stored.  Rows that no
//   expert has are written as zeros, by tiles without a sum.
// - Operand order.  An operand whose summation index is its row index (W in
//   `rows`, both in `weights`) is loaded as it lies, as boxes of 64 columns x
//   64 rows, and is an "MN-major" operand of the MMA: nothing is transposed
//   in memory.
// - Ragged sums.  In `weights` an expert's last k-block holds rows of the next
//   expert.  The MMA takes 16 rows at a time; those past the last are left
//   out, and where the last 16 are not all the expert's, the others are zeroed
//   in shared memory in both operands (a NaN there must not meet a zero) by a
//   warp of its own.  Only such blocks take that way: when all blocks did, it
//   doubled the kernel's time.
//
// Structure (one CTA per SM): warp 0 loads, warp 1 multiplies, the next 8 (weights
// and LONG: 16) store, the last (weights only) zeroes.  CG = 2 pairs two CTAs on a tile of
// 256 columns x up to 256 rows, CG = 1 takes 128 columns.  Accumulators are double
// buffered in Tensor Memory, so that a tile's epilogue runs beside the next
// one's loop; half of the storing warps belong to each.  GROUPS: stages of two
// or four k-blocks in one box, for products of few rows.  LONG: fp32 results of
// long sums, added up in segments.
//
// What bounds it and what it measured (graph-replayed, bf16 results unless said;
// floor: bytes at 6793 GB/s or operations at 1895 TFLOP/s):
//   weights' bytes   16 tokens, 2 of 8 experts of 4096 x 4096     43.5 us, floor 39.2
//                    16 rows for each of 64 of 4096 x 2048       160, floor 160
//   operations       8192 tokens, 8 of 128 of 4096 x 2048, silu  684-713, floor 580
//                    rows, 16384 rows, 8 of 8192 x 4096          599-629, floor 569
//                    weights, the same                           587-608, floor 569
//   both             9003 rows, 61 of 5000 x 2000, fp32          239, floor 211
//   output's bytes   weights, 64 of 2048 x 2048 fp32 with C      400, floor 336
//                    weights, 61 of 1000 x 2000, 3 rows each      53, floor 36
// (The ranges are of one program at different times: at 1400 W the clock moves.)
// In the second group the tensor pipe is active 89-91% of the time with about 1000
// rows an expert, and 72-74% in `weights`, whose tiles are 16 k-blocks then.
//
// Every mbarrier wait is bounded by %globaltimer: it gives up where its CTA has
// stood still (no block multiplied, no accumulator handed over) for as long as the
// limit, however long the call takes.  It then sets the abort flags of its CTA and
// of the pair's other one and the device status word, and all roles of both leave.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace gtn {

namespace {

constexpr int kBlockK = 64;                // summation indices per ring stage
constexpr int kChunkBytes = 64 * 128;      // 64 rows of 64 bf16: a chunk of an MN-major operand
constexpr int kPartBytes = 16 * 128;       // 16 rows of it: a chunk of a sum's last, shorter block
constexpr int kColBytes = 128 * 128;       // a stage of the columns' operand: 128 of them per CTA
constexpr int kErrTimeout = -5;            // GEMM_ERR_TIMEOUT
constexpr uint64_t kSettleNs = 2000000;    // what copies in flight are given to land after a wait has run out

// Terms that the tensor core adds up by itself for an fp32 result of a long sum
// (LONG).  Its accumulator cuts bits off at every MMA instead of rounding, so
// the error grows with the number of terms: 1.0e-6 of the result's norm at 1024,
// 2.1e-6 at 2000, about 8e-6 at 8192.  In LONG the two accumulators take segments
// in turn and the storing warps add them, rounded, in registers.  Segments of 8,
// 12 and 16 blocks leave 4.7e-7, 7.2e-7 and 1.0e-6 at every length; 9003 rows of
// 61 experts of 5000 x 2000 take 239, 239 and 238 us with them (233 without any),
// 8192 tokens through 8 of 128 of 4096 x 2048 817, 795 and 790 us.  bf16 results
// (an error of 1e-3) are added up by the tensor core alone.
//   In `weights` every tile goes by its own expert's rows, so that an expert's
// error, and its bits, do not depend on how many the others have.  A sum of one
// segment takes the path without sums in registers, on which C is loaded ahead:
// 64 matrices of 2048 x 2048 with C, 256 rows each, 400 us (539 with the other
// path for all tiles, 391 in a kernel without it); 1000 rows each of 32, some of
// one segment and some of two, 300.
constexpr int kSegmentBlocks = 12;         // k-blocks of a segment
static_assert(kSegmentBlocks % 4 == 0, "a whole number of stages of four k-blocks");

template <int OP, bool LONG>
struct Shape {
  static constexpr bool kWeights = OP == kExpertsWeights;
  static constexpr bool kMnCols = OP != kExpertsForward, kMnRows = kWeights;   // operands that are MN-major
  // Storing warps, half of them for each accumulator, and the rows that one
  // takes at a time.  With more of them more of C is on its way (64 matrices of
  // 2048 x 2048 fp32 with C: 16 warps 404 us, 8 424); a product's long sums hide
  // the stores of 8 (one prompt through 128 experts: 818 us, with 16 840).
  // LONG: all of them take every segment, 64 rows each, whose fp32 sums fill
  // most of a thread's 96 registers.
  static constexpr int kEpiWarps = kWeights || LONG ? 16 : 8;
  static constexpr int kRowsAtOnce = kWeights || LONG ? 16 : 32;
  static constexpr int kThreads = 32 * (2 + kEpiWarps + (kWeights ? 1 : 0));
};

// Ring stages at most (of `weights`: 32 or 48 KB each, 7 fit), and barriers: full,
// empty, and for ragged blocks tail and ready, per stage; accumulators; the drain.
__host__ __device__ constexpr int max_stages(bool weights) { return weights ? 8 : 16; }
__host__ __device__ constexpr int bars_of(bool weights) { return (weights ? 4 : 2) * max_stages(weights) + 5; }

__host__ __device__ constexpr int table_bytes(int E) { return 4 * (2 * E + 4); }

// What the roles of a CTA share at addresses known to the compiler, which take
// no registers.
struct __align__(16) Control {
  uint32_t tmem;              // base of the accumulators
  uint32_t abort;             // a wait of this CTA, or of the pair's other one, has run out
  uint32_t stages;            // barriers that show progress: `stages` of them from `empty` on, two from `accf` on
  uint32_t empty, accf;
  uint32_t since[16];         // LONG: a storing warp's clock (wait_bar_lean)
};
constexpr uint32_t kLate = 2;   // abort: set by wait_bar_lean

struct Abort {
  Control* c;
  uint64_t timeout_ns;
  int* status;
  int role;
  bool pair;
};

__device__ __forceinline__ bool aborting(const Control& c) { return *const_cast<const volatile uint32_t*>(&c.abort) != 0; }

// This CTA and the other one of its pair leave.  (Every wait ends before its CTA
// meets the other for the last time, so the other's shared memory is there.)
__device__ __forceinline__ void give_up(Control* c, bool pair, int* status, int role) {
  *const_cast<volatile uint32_t*>(&c->abort) = 1;
  if (pair) st_shared_cluster_u32(mapa_shared(smem_u32(&c->abort), cluster_ctarank() ^ 1u), 1);
  if (atomicCAS(status, 0, kErrTimeout) == 0) atomicExch(status + 1, (role << 24) | (int)blockIdx.x);
}

template <bool CLUSTER>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  if constexpr (CLUSTER) return mbar_try_wait_cluster(bar, parity);
  else return mbar_try_wait(bar, parity);
}

// A number that changes with every block whose MMAs are done and every accumulator
// that is handed over: the parities of their barriers.  (A count that the loading
// warp keeps in shared memory cost the weights' gradients 2%.)
__device__ __forceinline__ uint32_t progress(const Control& c) {
  uint32_t bits = 0;
#pragma unroll 1
  for (uint32_t i = 0; i < c.stages; ++i) bits = bits << 1 | (uint32_t)mbar_test_wait(c.empty + 8u * i, 0);
  return bits << 2 | (uint32_t)mbar_test_wait(c.accf, 0) << 1 | (uint32_t)mbar_test_wait(c.accf + 8u, 0);
}

// The limit is on seeing the same so many times in a row.  (A parity that has changed
// an even number of times looks the same, but not sixteen times.)
constexpr uint32_t kGlances = 16;

template <bool CLUSTER>
__device__ __noinline__ bool wait_bar_slow(uint32_t bar, uint32_t parity, Control* c, uint64_t timeout_ns, int* status,
                                           int role, bool pair) {
  uint64_t t0 = globaltimer();
  uint32_t seen = ~0u, same = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (try_wait<CLUSTER>(bar, parity)) return true;
    if (aborting(*c)) return false;
    if (globaltimer() - t0 <= timeout_ns / kGlances) continue;
    const uint32_t now = progress(*c);
    same = now == seen ? same + 1 : 0;
    if (same == kGlances) {
      give_up(c, pair, status, role);
      return false;
    }
    seen = now;
    t0 = globaltimer();
  }
}

// Bounded wait on an mbarrier phase.  False if this CTA is aborting.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Abort& ab) {
  if (try_wait<CLUSTER>(bar, parity)) return true;
  return wait_bar_slow<CLUSTER>(bar, parity, ab.c, ab.timeout_ns, ab.status, ab.role, ab.pair);
}

// The same without a call, whose registers a warp full of sums would have to
// spill, and with its clock in shared memory: in units of 2^16 ns, read every 256
// looks.  (It waits for one segment at a time, so that any progress but its own is
// not looked at.)  A warp whose clock has run out tells its CTA's roles alone; the rest of
// give_up() follows when it has left its tiles.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_bar_lean(uint32_t bar, uint32_t parity, Control& c, uint32_t units) {
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (try_wait<CLUSTER>(bar, parity)) return true;
    if (aborting(c)) return false;
    if (i & 255) continue;
    volatile uint32_t* since = &c.since[(threadIdx.x >> 5) - 2];
    const uint32_t now = (uint32_t)(globaltimer() >> 16);
    if (i == 256) *since = now;
    else if (now - *since > units) *const_cast<volatile uint32_t*>(&c.abort) = kLate;
  }
}

// The commit behind all MMAs, whether or not a wait has run out: they may take no
// longer than what the ring holds, but a limit set short is not for them.
template <bool CLUSTER>
__device__ __noinline__ bool wait_drain(uint32_t bar, uint64_t timeout_ns) {
  const uint64_t t0 = globaltimer(), limit = timeout_ns > 100000000 ? timeout_ns : 100000000;
  while (!try_wait<CLUSTER>(bar, 0))
    if (globaltimer() - t0 > limit) return false;
  return true;
}

__device__ __noinline__ void settle(uint64_t ns) {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < ns) __nanosleep(1000);
}

// Descriptor of an MN-major operand in shared memory: chunks of 64 columns
// (128 bytes, 128-byte swizzle), `chunk` bytes apart, one row of a chunk per
// summation index.  PTX ISA, tcgen05 shared memory descriptor: the stride from
// one group of 8 summation indices to the next (1024 bytes) in bits 32-45,
// that from one chunk of columns to the next in bits 16-29.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, int chunk) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(chunk >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// What the multiplying warp has to know of a tile, in the leader's shared
// memory beside the ring stage of the tile's first block: the loading thread
// puts it there before it arrives on that stage's barrier.  Tiles without a sum
// take no stage.  (One for their note would be handed back to the peer CTA
// without its having loaded anything, and so perhaps a second time before it
// has seen the first.)
struct Note {
  int n;        // the MMA's N; 0 behind the last tile
  int sum;      // summation indices
  int empty;    // tiles without a sum before this one
  int box;      // groups of k-blocks: rows that lie between one of a stage and the next
};

// The experts' first rows (E + 1) and first row blocks (E + 2: behind the
// experts the rows of nobody) of one launch, in shared memory.
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

__device__ __forceinline__ int div_by(int n, FastDiv d) { return d.mul ? (int)(__umulhi((uint32_t)n, d.mul) >> d.shift) : n; }

// One tile: its expert (E: the rows of nobody), its rows of the output from
// row0, the MMA's N for them, its first column, and its sum's range and blocks.
struct Tile {
  int e, row0, rows, n, col0;
  int k0, k_end, num_kb;      // weights: the expert's rows; else 0 and the sum's length
};

template <int CG, int OP, bool GROUPS>
__device__ __forceinline__ Tile tile_of(int t, const ExpertsParams& p, const Table& tb) {
  constexpr int kStep = 16 * CG;
  Tile r;
  int local, blocks, first, high, each;     // the expert's row blocks, its rows, and those of a block
  if constexpr (OP == kExpertsWeights) {
    r.e = div_by(t, p.by_tiles);
    local = t - r.e * p.row_blocks * p.col_blocks;
    blocks = p.row_blocks;
    first = 0;
    high = p.rows_out;
    each = p.row_block;
    r.k0 = tb.row[r.e];
    r.k_end = tb.row[r.e + 1];
    r.num_kb = (r.k_end - r.k0 + kBlockK - 1) / kBlockK;
  } else {
    // the last entry whose first row block is not past this one; entries
    // without rows share their first block with the next
    const int b = div_by(t, p.by_cols);
    int lo = 0, hi = p.E;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tb.tile[mid] <= b) lo = mid;
      else hi = mid - 1;
    }
    r.e = lo;
    local = t - tb.tile[lo] * p.col_blocks;
    blocks = tb.tile[lo + 1] - tb.tile[lo];
    first = tb.row[lo];
    high = (lo < p.E ? tb.row[lo + 1] : p.R) - first;
    // equal blocks, a multiple of the MMA's step.  All have rows: they are at
    // most tile_rows high, and all but one are cut from more than that many each
    each = blocks == 1 ? high : ((high + blocks - 1) / blocks + kStep - 1) / kStep * kStep;
    r.k0 = 0;
    r.k_end = p.S;
    r.num_kb = lo < p.E ? (p.S + kBlockK * (GROUPS ? p.group : 1) - 1) / (kBlockK * (GROUPS ? p.group : 1)) : 0;
  }
  // strips of p.strip row blocks, row blocks fastest within a strip
  int rb, cb;
  if (blocks == 1) {
    rb = 0;
    cb = local;
  } else {
    const int strip = div_by(local, p.by_strip_tiles), s0 = strip * p.strip, sh = min(p.strip, blocks - s0);
    const int in = local - s0 * p.col_blocks;
    cb = sh == p.strip ? div_by(in, p.by_strip) : in / sh;
    rb = s0 + in - cb * sh;
  }
  r.col0 = cb * (p.col_tile * CG);
  r.row0 = first + rb * each;
  r.rows = min(each, high - rb * each);
  r.n = (r.rows + kStep - 1) / kStep * kStep;
  return r;
}

// ---------------------------------------------------------------- loads
// A stage's columns from `col`, summation indices from k, to dst.  PAIR: on
// the leader's barrier.  chunk: bytes from one chunk of 64 columns to the next.
template <int OP, bool PAIR, bool GROUPS>
__device__ __forceinline__ void load_cols(uint32_t dst, const CUtensorMap* m, bool wide, int col, int k, int e, int chunk,
                                          uint32_t bar) {
  if constexpr (OP == kExpertsForward && GROUPS) {
    if constexpr (PAIR) tma_load_4d_pair(dst, m, 0, col, k / 64, e, bar);
    else tma_load_4d(dst, m, 0, col, k / 64, e, bar);
  } else if constexpr (OP == kExpertsForward) {
    if constexpr (PAIR) tma_load_3d_pair(dst, m, k, col, e, bar);
    else tma_load_3d(dst, m, k, col, e, bar);
  } else if (wide) {
    if constexpr (OP == kExpertsRows) {
      if constexpr (PAIR) tma_load_4d_pair(dst, m, 0, k, col / 64, e, bar);
      else tma_load_4d(dst, m, 0, k, col / 64, e, bar);
    } else {
      if constexpr (PAIR) tma_load_3d_pair(dst, m, 0, k, col / 64, bar);
      else tma_load_3d(dst, m, 0, k, col / 64, bar);
    }
  } else {
    for (int i = 0; i < 2; ++i) {
      if constexpr (OP == kExpertsRows) {
        if constexpr (PAIR) tma_load_3d_pair(dst + i * chunk, m, col + 64 * i, k, e, bar);
        else tma_load_3d(dst + i * chunk, m, col + 64 * i, k, e, bar);
      } else {
        if constexpr (PAIR) tma_load_2d_pair(dst + i * chunk, m, col + 64 * i, k, bar);
        else tma_load_2d(dst + i * chunk, m, col + 64 * i, k, bar);
      }
    }
  }
}

// The same for the rows from `row`; chunks: of 64 rows (weights).
template <int OP, bool PAIR, bool GROUPS>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* m, bool wide, int row, int k, int chunk,
                                          int chunks, uint32_t bar) {
  if constexpr (GROUPS) {
    if constexpr (PAIR) tma_load_3d_pair(dst, m, 0, row, k / 64, bar);
    else tma_load_3d(dst, m, 0, row, k / 64, bar);
  } else if constexpr (OP != kExpertsWeights) {
    if constexpr (PAIR) tma_load_2d_pair(dst, m, k, row, bar);
    else tma_load_2d(dst, m, k, row, bar);
  } else if (wide) {
    if constexpr (PAIR) tma_load_3d_pair(dst, m, 0, k, row / 64, bar);
    else tma_load_3d(dst, m, 0, k, row / 64, bar);
  } else {
    for (int i = 0; i < chunks; ++i) {
      if constexpr (PAIR) tma_load_2d_pair(dst + i * chunk, m, row + 64 * i, k, bar);
      else tma_load_2d(dst + i * chunk, m, row + 64 * i, k, bar);
    }
  }
}

// ---------------------------------------------------------------- epilogue
// The logistic activations for a result that is rounded to bf16: __expf, whose
// error grows with its argument (2^-22 of the value for each unit of it, below
// 2^-15 up to 89, where it is infinite), instead of expf.  Far below the rounding's 2^-9, and
// less work beside the MMAs.
template <int NR>
__device__ __forceinline__ void logistic_rows(float (&v)[NR], bool gelu) {
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const float t = gelu ? -1.5957691216057308f * fmaf(0.044715f * v[j], v[j] * v[j], v[j]) : -v[j];
    v[j] = __fdividef(v[j], 1.0f + __expf(t));
  }
}

template <int NR>
__device__ __forceinline__ void activate_rows(float (&v)[NR], int act, bool f32) {
  if (!f32 && act == kActSilu) logistic_rows(v, false);
  else if (!f32 && act == kActGeluTanh) logistic_rows(v, true);
  else activate_chunk(v, act);
}

// Values of NR rows of one column per lane, lane l on column `col` + l, to or
// from a row-major matrix at `base` (its element (first row, col)).  fp32 rows
// are 128 contiguous bytes of a warp.  bf16: in pairs, where the addresses
// allow: an even lane moves both columns of its pair in one row, the odd lane
// in the next, so that a step moves two rows of 64 bytes.
//
// For short sums these instructions are the kernel's time (with a select, a
// shuffle and two more selects a pair and a compare at each store 61 matrices
// of 1000 x 2000 took 64 us), so all words are made before the stores, and rows
// that are all there are stored without a look at each.
template <int NR>
__device__ __forceinline__ void store_rows_f32(float* at, long long ld, int rows, bool mine, const float (&v)[NR]) {
  if (!mine) return;
  if (rows >= NR) {
#pragma unroll
    for (int j = 0; j < NR; ++j, at += ld) *at = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < NR; ++j, at += ld)
      if (j < rows) *at = v[j];
  }
}

template <int NR>
__device__ __forceinline__ void store_rows_bf16(uint16_t* at, long long ld, int rows, bool mine, bool pairs,
                                                const float (&v)[NR]) {
  const int odd = threadIdx.x & 1;
  if (pairs) {
    uint32_t w[NR / 2];
#pragma unroll
    for (int j = 0; j < NR; j += 2) {
      const uint32_t own = pack_bf16x2(v[j], v[j + 1]);      // rows j and j + 1 of this column
      const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
      // even: both low halves (row j), odd: both high halves (row j + 1)
      w[j / 2] = __byte_perm(own, other, odd ? 0x3276 : 0x5410);
    }
    if (!mine) return;
    uint32_t* to = reinterpret_cast<uint32_t*>(at - odd + odd * ld);
    if (rows >= NR) {
#pragma unroll
      for (int j = 0; j < NR / 2; ++j, to += ld) *to = w[j];
    } else {
#pragma unroll
      for (int j = 0; j < NR / 2; ++j, to += ld)
        if (2 * j + odd < rows) *to = w[j];
    }
  } else if (mine) {
#pragma unroll
    for (int j = 0; j < NR; ++j, at += ld)
      if (j < rows) *at = (uint16_t)(pack_bf16x2(v[j], 0.0f) & 0xFFFFu);
  }
}

__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&x)[32]) { tmem_ld_32x32b_x32(taddr, x); }
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&x)[16]) { tmem_ld_32x32b_x16(taddr, x); }

// C's raw words, of the rows and columns that store_rows_* writes; add_c makes values of them.
template <int N, typename T>
__device__ __forceinline__ void load_words(const T* at, long long step, int count, bool mine, uint32_t* x) {
  if (mine && count >= N) {
#pragma unroll
    for (int j = 0; j < N; ++j, at += step) x[j] = *at;
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j, at += step) x[j] = mine && j < count ? *at : 0;
  }
}

template <int NR>
__device__ __forceinline__ void load_c(const void* base, long long ld, int rows, bool mine, bool f32, bool pairs,
                                       uint32_t (&x)[NR]) {
  const int odd = threadIdx.x & 1;
  const uint16_t* half = static_cast<const uint16_t*>(base);
  if (f32) load_words<NR>(static_cast<const uint32_t*>(base), ld, rows, mine, x);
  else if (pairs) load_words<NR / 2>(reinterpret_cast<const uint32_t*>(half - odd + odd * ld), ld, (rows + 1 - odd) / 2, mine, x);
  else load_words<NR>(half, ld, rows, mine, x);
}

template <int NR>
__device__ __forceinline__ void add_c(const uint32_t (&x)[NR], float beta, bool f32, bool pairs, float (&v)[NR]) {
  const int odd = threadIdx.x & 1;
  if (f32) {
#pragma unroll
    for (int j = 0; j < NR; ++j) v[j] = fmaf(beta, __uint_as_float(x[j]), v[j]);
  } else if (pairs) {
#pragma unroll
    for (int j = 0; j < NR / 2; ++j) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, x[j], 1);
      const float a = __uint_as_float(odd ? o & 0xFFFF0000u : x[j] << 16);      // row 2j, this lane's column
      const float b = __uint_as_float(odd ? x[j] & 0xFFFF0000u : o << 16);      // row 2j + 1
      v[2 * j] = fmaf(beta, a, v[2 * j]);
      v[2 * j + 1] = fmaf(beta, b, v[2 * j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NR; ++j) v[j] = fmaf(beta, __uint_as_float(x[j] << 16), v[j]);
  }
}

template <int CG, int OP, bool GROUPS, bool LONG>
__global__ void __launch_bounds__(Shape<OP, LONG>::kThreads, 1)
    gemm_experts_kernel(const __grid_constant__ ExpertsMaps maps, const __grid_constant__ ExpertsParams p) {
  using S_ = Shape<OP, LONG>;
  constexpr int kEpiWarps = S_::kEpiWarps, kRowsAtOnce = S_::kRowsAtOnce;
  constexpr bool kPair = CG == 2;
  constexpr int kMaxStages = max_stages(S_::kWeights), kBars = bars_of(S_::kWeights), kAccBars = kBars - 5;
  __shared__ Control ctl;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sC = smem_u32(smem);                       // the columns' operand
  const uint32_t sR = sC + p.stages * p.group * kColBytes;            // the rows' operand
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * p.group * (kColBytes + p.row_bytes));
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tail_bar = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };    // this CTA's bytes of a ragged block
  auto ready_bar = [&](int s) { return bar0 + 8u * (3 * kMaxStages + s); };   // leader: every CTA has zeroed it
  auto accf_bar = [&](int b) { return bar0 + 8u * (kAccBars + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (kAccBars + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (kAccBars + 4);
  Note* notes = reinterpret_cast<Note*>(bars + kBars);      // one per stage
  Table tb;
  tb.row = reinterpret_cast<int*>(notes + kMaxStages);
  tb.tile = tb.row + p.E + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const int first_tile = blockIdx.x / CG, step = gridDim.x / CG;
  const int group = GROUPS ? p.group : 1;      // k-blocks per stage

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      if constexpr (S_::kWeights) {
        mbar_init(tail_bar(s), 1);
        mbar_init(ready_bar(s), CG);
      }
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), (LONG ? kEpiWarps : kEpiWarps / 2) * CG);
    }
    mbar_init(drain_bar, 1);
    ctl.abort = 0;
    ctl.stages = (uint32_t)p.stages;
    ctl.empty = empty_bar(0);
    ctl.accf = accf_bar(0);
    fence_mbar_init();
    fence_proxy_async_smem();
    if (p.has_ab) {
      tma_prefetch_desc(&maps.cols);
      tma_prefetch_desc(&maps.rows);
      if (S_::kWeights) tma_prefetch_desc(&maps.cols_part);
      for (int i = 0; i < (S_::kWeights ? 1 : p.row_box < 64 ? 0 : 3); ++i) tma_prefetch_desc(&maps.rows_part[i]);
    }
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(&ctl.tmem), 2 * p.acc_cols);
  // Inputs may come from the previous kernel on the stream: no global memory
  // access before this point.
  griddep_wait();
  griddep_launch_dependents();
  for (int e = threadIdx.x; e <= p.E; e += S_::kThreads) tb.row[e] = min(max(p.offsets[e], 0), p.R);
  __syncthreads();
  if (warp == 2) fill_table(p, tb, S_::kWeights ? 0 : p.tile_rows);
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = ctl.tmem;
  const int num_tiles = (S_::kWeights ? p.E * p.row_blocks : tb.tile[p.E + 1]) * p.col_blocks;
  // the rows of an expert's last block that are not its own, when the MMA would take some of them
  auto ragged = [](const Tile& r) { return S_::kWeights && ((r.k_end - r.k0) & 15) != 0; };

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    // (the whole warp, one elected lane of which issues, as below)
    Abort ab{&ctl, p.timeout_ns, p.status, kRoleProducer, kPair};
    auto wait_empty = [&](int s, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_bar<kPair>(empty_bar(s), parity, ab)) != 0;
    };
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;
    auto advance = [&] {
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    };
    int empty = 0;          // tiles without a sum since the last note
    for (int t = first_tile; t < num_tiles && ok; t += step) {
      Tile r = tile_of<CG, OP, GROUPS>(t, p, tb);
      if (r.num_kb == 0) {
        ++empty;
        continue;
      }
      const int e = __shfl_sync(0xffffffffu, r.e, 0), n = __shfl_sync(0xffffffffu, r.n, 0);
      const int k0 = __shfl_sync(0xffffffffu, r.k0, 0), sum = __shfl_sync(0xffffffffu, r.k_end, 0) - k0;
      const int share = n / CG;              // this CTA's share of the tile's rows
      const int c_at = __shfl_sync(0xffffffffu, r.col0, 0) + (int)rank * p.col_tile;
      const int r_at = __shfl_sync(0xffffffffu, r.row0, 0) + (int)rank * share;
      // the smallest box that holds the share: whole, 3/4, 1/2 or 1/4 (of at least 64 rows, else whole)
      const int box = S_::kWeights || p.row_box < 64 ? 3 : (4 * share - 1) / p.row_box;
      const int chunks = p.wide_rows ? p.row_bytes / kChunkBytes : (share + 63) / 64;    // weights
      const int box_rows = box == 3 ? p.row_box : (box + 1) * (p.row_box / 4);
      const uint32_t tx =
          (uint32_t)(group * (p.col_tile * 128 + (S_::kWeights ? chunks * kChunkBytes : box_rows * 128)));
      const CUtensorMap* row_map = box == 3 ? &maps.rows : &maps.rows_part[box];
      const int blocks = (sum + kBlockK * group - 1) / (kBlockK * group), whole = S_::kWeights ? sum / kBlockK : blocks;
      // (tests: the block of the first tile whose copies CTA 0 leaves out)
      const int dropped = p.fault && blockIdx.x == 0 && t == 0 ? (p.fault & kFaultSkipTmaOnce ? 0 : blocks - 1) : -1;
      for (int kb = 0; kb < whole; ++kb) {
        ok = wait_empty(stage, phase ^ 1);
        if (!ok) break;
        const int k = k0 + kb * kBlockK * group;
        const uint32_t c = sC + stage * group * kColBytes, b = sR + stage * group * p.row_bytes;
        const uint32_t fb = full_bar(stage);
        const uint32_t to = kPair ? mapa_shared(fb, 0) : fb;    // a pair's bytes all count on its leader's barrier
        if (elect_one()) {
          if (kb == 0) notes[stage] = Note{n, sum, empty, box_rows};
          if (leader) mbar_arrive_expect_tx(fb, tx * CG);
          if (kb != dropped) {
            load_cols<OP, kPair, GROUPS>(c, &maps.cols, p.wide_cols, c_at, k, e, kChunkBytes, to);
            load_rows<OP, kPair, GROUPS>(b, row_map, p.wide_rows, r_at, k, kChunkBytes, chunks, to);
          }
        }
        advance();
      }
      if (S_::kWeights && ok && whole < blocks) {
        // the rest of the expert's rows, 16 at a time.  Where the last are not
        // all its own, the bytes count on each CTA's own barrier, for the warp
        // that zeroes
        ok = wait_empty(stage, phase ^ 1);
        if (!ok) break;
        const int parts = (sum - whole * kBlockK + 15) / 16;
        const uint32_t part_tx = (uint32_t)(parts * (2 + chunks) * kPartBytes);
        const bool own = (sum & 15) != 0;
        const uint32_t fb = full_bar(stage), tail = tail_bar(stage);
        const uint32_t to = kPair ? mapa_shared(fb, 0) : fb;
        if (elect_one()) {
          if (whole == 0) notes[stage] = Note{n, sum, empty, 0};
          if (leader) {
            if (own) mbar_arrive(fb);
            else mbar_arrive_expect_tx(fb, part_tx * CG);
          }
          if (own) mbar_arrive_expect_tx(tail, part_tx);
          for (int i = whole == dropped ? parts : 0; i < parts; ++i) {
            const uint32_t ci = sC + stage * kColBytes + i * (kColBytes / 4), bi = sR + stage * p.row_bytes + i * (p.row_bytes / 4);
            const int k = k0 + whole * kBlockK + 16 * i;
            if (own) {
              load_cols<OP, false, false>(ci, &maps.cols_part, p.wide_cols, c_at, k, e, kPartBytes, tail);
              load_rows<OP, false, false>(bi, &maps.rows_part[0], p.wide_rows, r_at, k, kPartBytes, chunks, tail);
            } else {
              load_cols<OP, kPair, GROUPS>(ci, &maps.cols_part, p.wide_cols, c_at, k, e, kPartBytes, to);
              load_rows<OP, kPair, GROUPS>(bi, &maps.rows_part[0], p.wide_rows, r_at, k, kPartBytes, chunks, to);
            }
          }
        }
        advance();
      }
      empty = 0;
    }
    if (ok && leader && wait_empty(stage, phase ^ 1) && elect_one()) {
      notes[stage] = Note{0, 0, empty, 0};
      mbar_arrive(full_bar(stage));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    // The whole warp runs this, and one elected lane issues: with one lane in
    // here alone each MMA took 69 cycles to issue and each block 590, whatever its N.
    if (leader) {
      Abort ab{&ctl, p.timeout_ns, p.status, kRoleMma, kPair};
      // (the whole warp leaves, or none of it)
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_bar<kPair>(bar, parity, ab)) != 0;
      };
      int stage = 0;
      uint32_t phase = 0, ready_phase = 0;      // ready: one bit per stage
      int acc = 0;
      uint32_t acc_phase = 0;
      auto commit = [&](uint32_t bar) {
        if constexpr (kPair) mma_commit_pair(bar, 0x3);
        else mma_commit(bar);
      };
      auto advance = [&] {
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      };
      // the accumulator goes to the warps that store it, the other is next
      auto hand_over = [&] {
        if (elect_one()) commit(accf_bar(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      };
      while (true) {
        if (!wait_all(full_bar(stage), phase)) break;
        const int n = __shfl_sync(0xffffffffu, notes[stage].n, 0), sum = __shfl_sync(0xffffffffu, notes[stage].sum, 0);
        const int empty = __shfl_sync(0xffffffffu, notes[stage].empty, 0), box = __shfl_sync(0xffffffffu, notes[stage].box, 0);
        bool ok = true;
        for (int i = 0; i < empty && ok; ++i) {       // their zeros are stored without a look at the accumulator
          ok = wait_all(acce_bar(acc), acc_phase ^ 1);
          if (ok) hand_over();
        }
        if (!ok || n == 0) break;
        const uint32_t idesc =
            instr_desc_bf16_f32(128 * CG, n) | (S_::kMnCols ? 1u << 15 : 0u) | (S_::kMnRows ? 1u << 16 : 0u);
        if (!wait_all(acce_bar(acc), acc_phase ^ 1)) break;
        auto d_tmem = [&] { return tmem_base + (uint32_t)(acc * p.acc_cols); };
        // Whole blocks; the last, shorter one apart: with the two in one loop,
        // and so its steps and strides in registers, the MMAs came with pauses
        // (2048 rows for each of 8 matrices of 8192 x 4096: 747 us, apart 625).
        const int blocks = (sum + kBlockK * group - 1) / (kBlockK * group), whole = S_::kWeights ? sum / kBlockK : blocks;
        // blocks of one segment into the current accumulator
        auto multiply = [&](int kb0, int kb1) {
          const uint32_t d = d_tmem();
          for (int kb = kb0; kb < kb1; ++kb) {
            if (kb > 0) ok = wait_all(full_bar(stage), phase);
            if (!ok) break;
            tc_fence_after();
            const uint32_t c = sC + stage * group * kColBytes, b = sR + stage * group * p.row_bytes;
            const uint64_t c0 = S_::kMnCols ? desc_mn(c, kChunkBytes) : smem_desc_sw128(c);
            const uint64_t b0 = S_::kMnRows ? desc_mn(b, kChunkBytes) : smem_desc_sw128(b);
            // 16 summation indices are 32 bytes of a K-major operand's rows, 16 rows of each chunk of an MN-major one
            constexpr uint64_t kStepC = S_::kMnCols ? kPartBytes / 16 : 2, kStepR = S_::kMnRows ? kPartBytes / 16 : 2;
            if (elect_one()) {
              if constexpr (GROUPS) {
                for (int j = 0; j < group; ++j)
#pragma unroll
                  for (int i = 0; i < kBlockK / 16; ++i)
                    mma_issue<CG, kKindF16>(d, c0 + (uint64_t)(j * p.col_tile * 8 + 2 * i), b0 + (uint64_t)(j * box * 8 + 2 * i),
                                            idesc, (kb != kb0 || j != 0 || i != 0) ? 1u : 0u);
              } else {
#pragma unroll
                for (int i = 0; i < kBlockK / 16; ++i)
                  mma_issue<CG, kKindF16>(d, c0 + kStepC * i, b0 + kStepR * i, idesc, (kb != kb0 || i != 0) ? 1u : 0u);
              }
              commit(empty_bar(stage));
            }
            advance();
          }
        };
        if constexpr (LONG) {
          const int segment = kSegmentBlocks / group;
          for (int kb = 0; kb < whole && ok; kb += segment) {
            if (kb > 0) {
              hand_over();
              ok = wait_all(acce_bar(acc), acc_phase ^ 1);
              if (!ok) break;
            }
            multiply(kb, min(whole, kb + segment));
          }
        } else {
          multiply(0, whole);
        }
        if (S_::kWeights && ok && whole < blocks) {
          if (whole > 0) ok = wait_all(full_bar(stage), phase);
          if (ok && (sum & 15) != 0) {
            ok = wait_all(ready_bar(stage), (ready_phase >> stage) & 1u);
            ready_phase ^= 1u << stage;
          }
          if (!ok) break;
          tc_fence_after();
          // parts of 16 rows, each with its chunks together
          const int parts = (sum - whole * kBlockK + 15) / 16;
          if (elect_one()) {
            for (int i = 0; i < parts; ++i)
              mma_issue<CG, kKindF16>(d_tmem(), desc_mn(sC + stage * kColBytes + i * (kColBytes / 4), kPartBytes),
                                      desc_mn(sR + stage * p.row_bytes + i * (p.row_bytes / 4), kPartBytes), idesc,
                                      (whole != 0 || i != 0) ? 1u : 0u);
            commit(empty_bar(stage));
          }
          advance();
        }
        if (!ok) break;
        hand_over();
      }
      // All MMAs that were issued complete before TMEM is released.
      if (elect_one()) commit(drain_bar);
      if (!wait_drain<kPair>(drain_bar, p.timeout_ns)) give_up(&ctl, kPair, p.status, kRoleMma);
    }
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                   // TMEM lane quarter this warp may access
    // Half of the warps take the tiles of one accumulator, half those of the other:
    // while some store, the others wait for sums, read and convert.  LONG: all take
    // all of them, as the next segment's accumulator is the other one.
    constexpr int kGroups = LONG ? 1 : 2;
    [[maybe_unused]] int done = 0;            // LONG: segments taken
    const int acc = LONG ? 0 : (warp - 2) / (kEpiWarps / 2);
    constexpr int kRowStep = kEpiWarps / (4 * kGroups) * kRowsAtOnce;
    Abort ab{&ctl, p.timeout_ns, p.status, kRoleEpilogue, kPair};
    const bool f32 = LONG || p.out_f32, pairs = p.pairs;
    const int esize = f32 ? 4 : 2;
    uint32_t acc_phase = 0;
    const uint32_t acce_target = kPair ? mapa_shared(acce_bar(acc), 0) : acce_bar(acc);
    // accumulator read, its values in registers: it goes back to the MMA warp.
    // Relaxed: a release across the cluster waits for the stores before it, 1000 to
    // 9000 cycles (9003 rows of 61 of 5000 x 2000 in fp32: 258 us, relaxed 248).
    auto hand_back = [&](int a) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair) mbar_arrive_relaxed_cluster(acce_target + 8u * (a - acc));
        else mbar_arrive_relaxed(acce_bar(a));
      }
    };
    for (int t = first_tile + acc * step; t < num_tiles; t += kGroups * step) {
      const Tile r = tile_of<CG, OP, GROUPS>(t, p, tb);
      const int col = r.col0 + (int)rank * p.col_tile + q * 32 + lane;
      const bool mine = q * 32 + lane < p.col_tile && col < p.cols_out;
      auto element = [&](const void* base, long long ld, long long stride, int row) {
        return const_cast<uint8_t*>(static_cast<const uint8_t*>(base)) +
               ((OP == kExpertsWeights ? (long long)r.e * stride : 0) + (long long)row * ld + col) * esize;
      };
      // segments of this tile's sum (weights: of its own expert's rows)
      const int whole = S_::kWeights ? (r.k_end - r.k0) / kBlockK : r.num_kb;
      [[maybe_unused]] const int segments = max(1, (whole * group + kSegmentBlocks - 1) / kSegmentBlocks);
      if (LONG && !(S_::kWeights && segments == 1)) {
        // this warp's rows of every segment, added up in fp32 registers (with
        // GROUPS a tile has 128 rows at most)
        constexpr int kMine = GROUPS ? 32 : 64;
        const int part = (warp - 2) / 4 * kMine;
        float sum[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) sum[j] = 0.0f;
        if (S_::kWeights && p.has_c && r.col0 + (int)rank * p.col_tile + q * 32 < p.cols_out)
          // C, which no registers are left for, on its way to L2: 128 bytes of rows lane and lane + 32
          // (32 matrices of 2048 x 2048 with C, 1000 rows each: 342 us without, 298 with; 285 now)
#pragma unroll
          for (int j = 0; j < kMine; j += 32)
            if (part + lane + j < r.rows)
              prefetch_l2(static_cast<const uint8_t*>(element(p.C, p.ldc, p.stride_c, r.row0 + part + lane + j)) - lane * esize);
        bool ok = true;
        for (int i = 0; i < segments && ok; ++i, ++done) {
          const int a = done & 1;
          ok = __all_sync(0xffffffffu, wait_bar_lean<kPair>(accf_bar(a), (uint32_t)(done >> 1) & 1u, ctl, p.timeout_units)) != 0;
          if (!ok) break;
          tc_fence_after();
          if (r.num_kb > 0) {
#pragma unroll
            for (int j = 0; j < kMine; j += 16)
              if (part + j < r.rows) {
                uint32_t x[16];
                tmem_ld_rows(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * p.acc_cols + part + j), x);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) sum[j + k] += __uint_as_float(x[k]);
              }
          }
          hand_back(a);
        }
        if (!ok) break;
        // Where it goes is worked out only now: in registers during the sum it
        // spilled, and behind a full memory system a spilled word takes microseconds.
        int again = t;
        asm volatile("" : "+r"(again));
        const Tile o = tile_of<CG, OP, GROUPS>(again, p, tb);
        const int o_col = o.col0 + (int)rank * p.col_tile + q * 32 + lane;
        const bool o_mine = q * 32 + lane < p.col_tile && o_col < p.cols_out;
        auto place = [&](void* base, long long ld, long long stride, int row) {
          return static_cast<float*>(base) + ((OP == kExpertsWeights ? (long long)o.e * stride : 0) + (long long)row * ld + o_col);
        };
#pragma unroll
        for (int j = 0; j < kMine; j += 8)
          if (part + j < o.rows) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = p.alpha * sum[j + k];
            if constexpr (OP == kExpertsForward) activate_rows(v, p.act, true);
            if constexpr (OP == kExpertsWeights)
              if (p.has_c) {
                uint32_t xc[8];
                load_c(place(const_cast<void*>(p.C), p.ldc, p.stride_c, o.row0 + part + j), p.ldc, o.rows - part - j, o_mine, true, false, xc);
                add_c(xc, p.beta, true, false, v);
              }
            store_rows_f32(place(p.D, p.ldd, p.stride_d, o.row0 + part + j), p.ldd,
                           o.rows - part - j, o_mine, v);
          }
        if (__any_sync(0xffffffffu, aborting(ctl))) break;
        continue;
      }
      // LONG: nothing that this path needs may be held in a register during the
      // other's long sums, neither what follows from these (the rows' distances from
      // one another, the same for all tiles) nor an undefined C.
      int own = warp;
      long long ldc = p.ldc, ldd = p.ldd;
      if constexpr (LONG) asm volatile("" : "+r"(own), "+l"(ldc), "+l"(ldd));
      const int c_first = (own - 2) / 4 % (kEpiWarps / (4 * kGroups)) * kRowsAtOnce;
      [[maybe_unused]] uint32_t xc[kRowsAtOnce] = {};
      if constexpr (OP == kExpertsWeights)
        if (p.has_c)
          load_c(element(p.C, ldc, p.stride_c, r.row0 + c_first), ldc, r.rows - c_first, mine, f32, pairs, xc);
      const int a = LONG ? done & 1 : acc;
      if constexpr (LONG) acc_phase = (uint32_t)(done++ >> 1) & 1u;
      // (the whole warp leaves, or none of it: what follows is warp-wide)
      if constexpr (LONG) {
        if (!__all_sync(0xffffffffu, wait_bar_lean<kPair>(accf_bar(a), acc_phase, ctl, p.timeout_units))) break;
      } else {
        if (!__all_sync(0xffffffffu, wait_bar<kPair>(accf_bar(a), acc_phase, ab))) break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int c = c_first; c < r.rows; c += kRowStep) {
        float v[kRowsAtOnce];
        if (r.num_kb > 0) {
          uint32_t x[kRowsAtOnce];
          tmem_ld_rows(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * p.acc_cols + c), x);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < kRowsAtOnce; ++j) v[j] = __uint_as_float(x[j]);
          if (p.alpha != 1.0f) {
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j) v[j] *= p.alpha;
          }
        } else {
#pragma unroll
          for (int j = 0; j < kRowsAtOnce; ++j) v[j] = 0.0f;
        }
        if constexpr (OP == kExpertsForward) activate_rows(v, p.act, f32);
        if constexpr (OP == kExpertsWeights) {
          if (p.has_c) {
            add_c(xc, p.beta, f32, pairs, v);
            // the next rows of C are on their way while these are stored
            const int next = c + kRowStep;
            if (next < r.rows)
              load_c(element(p.C, ldc, p.stride_c, r.row0 + next), ldc, r.rows - next, mine, f32, pairs, xc);
          }
        }
        uint8_t* to = element(p.D, ldd, p.stride_d, r.row0 + c);
        if (f32) store_rows_f32(reinterpret_cast<float*>(to), ldd, r.rows - c, mine, v);
        else store_rows_bf16(reinterpret_cast<uint16_t*>(to), ldd, r.rows - c, mine, pairs, v);
      }
      hand_back(a);
      if (__any_sync(0xffffffffu, aborting(ctl))) break;
      acc_phase ^= 1;
    }
    if (LONG && *const_cast<volatile uint32_t*>(&ctl.abort) == kLate) give_up(&ctl, kPair, p.status, kRoleEpilogue);
  } else if constexpr (S_::kWeights) {
    // ------------------------------------------------------------ ragged blocks
    Abort ab{&ctl, p.timeout_ns, p.status, kRoleProducer, kPair};
    int stage = 0;
    uint32_t tail_phase = 0;            // one bit per stage
    const int chunks = p.row_bytes / kChunkBytes;
    for (int t = first_tile; t < num_tiles; t += step) {
      const Tile r = tile_of<CG, OP, GROUPS>(t, p, tb);
      const int last = (stage + r.num_kb - 1) % p.stages;      // (a tile without a sum is not ragged)
      stage = (stage + r.num_kb) % p.stages;
      if (!ragged(r)) continue;
      if (!__all_sync(0xffffffffu, wait_bar<false>(tail_bar(last), (tail_phase >> last) & 1u, ab))) break;
      tail_phase ^= 1u << last;
      // of the last 16 rows those from `valid` on, in every chunk of both operands
      const int part = (r.k_end - r.k0 - 1) % kBlockK / 16, valid = (r.k_end - r.k0) & 15, bad = 16 - valid;
      const uint32_t c = sC + last * kColBytes + part * (kColBytes / 4);
      const uint32_t b = sR + last * p.row_bytes + part * (p.row_bytes / 4);
      for (int i = lane; i < (2 + chunks) * bad * 8; i += 32) {
        const int chunk = i / (bad * 8), in = i - chunk * (bad * 8);
        const uint32_t base = chunk < 2 ? c + chunk * kPartBytes : b + (chunk - 2) * kPartBytes;
        st_shared_v4(base + (valid + in / 8) * 128 + (in % 8) * 16, 0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair) mbar_arrive_cluster(mapa_shared(ready_bar(last), 0));
        else mbar_arrive(ready_bar(last));
      }
    }
  }

  __syncthreads();
  // Both CTAs of a pair wait for the last commit: those before it arrive on both, and
  // none may come after a CTA has left its shared memory to the next.  (The one
  // without MMAs only now, when its other roles are done, or the call's time would count.)
  if (kPair && !leader && warp == 1 && !wait_drain<kPair>(drain_bar, p.timeout_ns)) give_up(&ctl, kPair, p.status, kRoleMma);
  // Whatever wait ran out: copies already on their way, into this CTA or by it, land
  // before either CTA gives its shared memory to the next.
  if (aborting(ctl)) settle(kSettleNs);
  if constexpr (kPair) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<CG>(tmem_base, 2 * p.acc_cols);
  }
}

// 0: products on single k-blocks, 1: on groups, 2: rows, 3: weights on single
// CTAs, 4: on pairs; from 5 on the same with long sums in fp32
constexpr int kKernels = 10;

int kernel_index(const ExpertsParams& p) {
  return (p.op == kExpertsForward ? (p.group > 1 ? 1 : 0) : p.op == kExpertsRows ? 2 : p.cg + 2) + (p.long_sum ? 5 : 0);
}

template <bool LONG>
const void* kernel_of(int index) {
  static const void* const table[5] = {
      (const void*)gemm_experts_kernel<2, kExpertsForward, false, LONG>,
      (const void*)gemm_experts_kernel<2, kExpertsForward, true, LONG>,
      (const void*)gemm_experts_kernel<2, kExpertsRows, false, LONG>,
      (const void*)gemm_experts_kernel<1, kExpertsWeights, false, LONG>,
      (const void*)gemm_experts_kernel<2, kExpertsWeights, false, LONG>};
  return table[index];
}

const void* kernel_at(int index) { return index < 5 ? kernel_of<false>(index) : kernel_of<true>(index - 5); }

int threads_of(int index) {
  return index >= 5   ? (index >= 8 ? Shape<kExpertsWeights, true>::kThreads : Shape<kExpertsForward, true>::kThreads)
         : index >= 3 ? Shape<kExpertsWeights, false>::kThreads
                      : Shape<kExpertsForward, false>::kThreads;
}

constexpr int kSmemMax = 232448 - (int)sizeof(Control);      // beside what is static

int smem_bytes(const ExpertsParams& p) {
  return 1024 + p.stages * p.group * (kColBytes + p.row_bytes) + bars_of(p.op == kExpertsWeights) * 8 +
         max_stages(p.op == kExpertsWeights) * (int)sizeof(Note) + table_bytes(p.E);
}

}  // namespace

void experts_geometry(ExpertsParams* p, int sms) {
  const bool weights = p->op == kExpertsWeights;
  const int active = p->E < p->R ? p->E : p->R;       // experts that can have rows
  const int average = active > 0 ? p->R / active : 0;
  // Pairs halve what a CTA loads of the other operand.  Weights of few rows,
  // where the output's memory decides: single CTAs, which need not wait for each
  // other.  64 matrices of 2048 x 2048, single / pairs, us, by the rows of each:
  //   bf16          64: 97 / 98,    128: 109 / 107,  256: 143 / 127,  512: 225 / 184
  //   bf16 with C   256: 284 / 288, 384: 309 / 302,  512: 328 / 321,  768: 370 / 355
  //   fp32          64: 199 / 192,  128: 205 / 200,  384: 261 / 201,  512: 300 / 246
  //   fp32 with C   256: 373 / 416, 512: 388 / 433, 1024: 531 / 530, 1536: 705 / 591
  // Routed unevenly: bf16, 150 on average: 135 / 136; with C, 500: 361 / 344; fp32 with C, 1000: 299 / 298.
  // LONG for weights wherever an expert can have more rows than a segment: how
  // many each has is known on the device only, and every tile goes by its own.
  p->long_sum = p->out_f32 && (weights ? p->R : p->S) > kSegmentBlocks * kBlockK;
  p->cg = weights && average < (!p->has_c ? 192 : p->out_f32 ? 768 : 320) ? 1 : 2;
  const int step = 16 * p->cg;
  const int most = average < 16 ? 32 : average > 128 ? 256 : 2 * average;
  p->tile_rows = weights ? 256 : (most + 31) / 32 * 32;
  if (!weights && p->tile_rows > (p->R + step - 1) / step * step) p->tile_rows = (p->R + step - 1) / step * step;
  const int share = p->tile_rows / p->cg;
  p->row_box = share;
  p->row_bytes = weights ? share / 64 * kChunkBytes : (share * 128 + 1023) / 1024 * 1024;
  // Few rows: W's bytes decide, and each CTA takes the same number of them when
  // the tiles' columns are chosen so that the rounds of tiles are full (16
  // tokens through 2 of 8 matrices of 4096 x 4096: 128 tiles of 256 columns on 76
  // pairs take two rounds; 152 tiles of 224 columns too).
  p->col_tile = 128;
  if (p->op == kExpertsForward && average < 64) {
    long long best = 0;
    for (int c = 128; c >= 96; c -= 16) {
      const long long tiles = (long long)active * ((p->cols_out + 2 * c - 1) / (2 * c)), time = (tiles + sms / 2 - 1) / (sms / 2) * c;
      if (!best || time < best) {
        best = time;
        p->col_tile = c;
      }
    }
  }
  p->acc_cols = 32;
  while (p->acc_cols < p->tile_rows) p->acc_cols *= 2;
  // Boxes of four or two k-blocks, where three stages of them fit: an SM asks
  // for the bytes of few rows sooner (one token through 2 of 8 matrices of 4096 x
  // 4096: 17.4, with two 16.1, with four 13.3 us; 16 rows each for 64 of 4096 x
  // 2048: 171, 163, 160; 32 rows each 172, 163, with four and two stages 173).
  // With long tiles the code for it costs (a prompt 696, 725).
  p->stages = 0;
  p->group = 1;
  const int room = kSmemMax - smem_bytes(*p);
  if (p->op == kExpertsForward && average < 64 && p->S % kBlockK == 0)
    for (int g = 4; g > 1 && p->group == 1; g /= 2)
      if (p->S >= g * kBlockK && room >= 3 * g * (kColBytes + p->row_bytes)) p->group = g;
  p->stages = room / (p->group * (kColBytes + p->row_bytes));
  if (p->stages > max_stages(weights)) p->stages = max_stages(weights);
}

FastDiv fast_div(uint32_t d) {
  FastDiv r = {0, 0};
  if (d <= 1) return r;
  uint32_t s = 0;
  while ((1u << s) < d) ++s;
  r.mul = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
  r.shift = s - 1;
  return r;
}

cudaError_t launch_experts(const ExpertsMaps& maps, ExpertsParams p, int sms, cudaStream_t stream, LaunchInfo* info) {
  static DeviceOnce configured;
  static int pairs[DeviceOnce::kDevices][kKernels] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  e = configured.run(dev, [&] {
    for (int i = 0; i < kKernels; ++i) {
      cudaError_t err = cudaFuncSetAttribute(kernel_at(i), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
      if (err != cudaSuccess) return err;
      cfg.gridDim = dim3(2);
      cfg.blockDim = dim3(threads_of(i));
      cfg.dynamicSmemBytes = kSmemMax;
      cfg.numAttrs = 1;
      if (i % 5 != 3 && (err = cudaOccupancyMaxActiveClusters(&pairs[dev][i], kernel_at(i), &cfg))) return err;
    }
    return cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  const int index = kernel_index(p);
  const int most = p.cg == 2 ? pairs[dev][index] : sms;
  if (most < 1) return cudaErrorInvalidConfiguration;
  // Tiles: known for the weights' gradient; else the most that the rows can
  // make, each expert and the rows of nobody ending with one part tile.
  const long long blocks = p.op == kExpertsWeights ? (long long)p.E * p.row_blocks
                                                   : (long long)p.R / p.tile_rows + (p.E + 1 < p.R ? p.E + 1 : p.R);
  const int units = (int)(blocks * p.col_blocks < most ? blocks * p.col_blocks : most);
  attr[0].val.clusterDim.x = p.cg;
  cfg.gridDim = dim3(units * p.cg);
  cfg.blockDim = dim3(threads_of(index));
  cfg.dynamicSmemBytes = smem_bytes(p);
  cfg.stream = stream;
  cfg.numAttrs = 2;
  *info = LaunchInfo{};
  info->grid = units * p.cg;
  info->cluster = p.cg;
  info->block = cfg.blockDim.x;
  info->tile_m = p.tile_rows;
  info->tile_n = 128 * p.cg;
  info->stages = p.stages;
  info->smem_bytes = cfg.dynamicSmemBytes;
  info->k_parts = 1;
  info->scheduler = 1;
  static const char* const names[kKernels] = {
      "gemm_experts_kernel<forward>",         "gemm_experts_kernel<forward, groups>",
      "gemm_experts_kernel<rows>",            "gemm_experts_kernel<weights, 1>",
      "gemm_experts_kernel<weights, 2>",      "gemm_experts_kernel<forward, long>",
      "gemm_experts_kernel<forward, groups, long>", "gemm_experts_kernel<rows, long>",
      "gemm_experts_kernel<weights, 1, long>", "gemm_experts_kernel<weights, 2, long>"};
  info->kernel = names[index];
  p.timeout_units = (uint32_t)std::min<uint64_t>((p.timeout_ns >> 16) + 1, 1u << 31);
  p.by_cols = fast_div(p.col_blocks);
  p.by_tiles = fast_div(p.row_blocks * p.col_blocks);
  p.by_strip = fast_div(p.strip);
  p.by_strip_tiles = fast_div(p.strip * p.col_blocks);
  void* args[2] = {const_cast<ExpertsMaps*>(&maps), &p};
  return cudaLaunchKernelExC(&cfg, kernel_at(index), args);
}

}  // namespace gtn
