// Tokens to expert order and back: the two ends of a mixture-of-experts MLP
// around the grouped products (gemm_expert_* in include/gemm_tn.h).
//
//   dispatch            slot s = t k + j goes to row offsets[e] + #{s' < s : id(s') = e}, e = id(s);
//                       Xs[row] = X[t]
//   dispatch backward   dX[t]   = sum_j dXs[slot_row[t, j]]            (combine with weights of one)
//   combine             out[t]  = sum_j w[t, j] Y[slot_row[t, j]]
//   combine backward    dY[slot_row[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], Y[slot_row[t, j]]>
//
// All of them are bound by memory.  Every kernel works token by token, so
// that the token's row is read (or written) once and only the k expert rows
// move per slot; walking the expert rows instead would read X k times.  (The
// combine's gradient reads dout's row once for every eight slots.)  Sums
// run over j in order in fp32 and are rounded once, with no atomics on data,
// so results do not change from run to run.  Rows that no slot fills (dropped
// slots) are set to zero by the token loop, T rows apart.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace gtn {
namespace {

constexpr int kRowThreads = 256;

// ---------------------------------------------------------------- sorting
__device__ __forceinline__ int load_id(const ExpertParams& p, int s) {
  long long at = s;
  if (p.ld_ids != p.k) {   // rows apart: no division where they are not
    const int t = s / p.k;
    at = (long long)t * p.ld_ids + (s - t * p.k);
  }
  const long long v = p.ids64 ? static_cast<const long long*>(p.ids)[at] : static_cast<const int*>(p.ids)[at];
  return v >= 0 && v < p.E ? (int)v : p.E;   // E = dropped
}

// Histogram of one chunk of slots: hist[chunk][e].
__global__ void __launch_bounds__(1024) expert_hist_kernel(ExpertParams p) {
  extern __shared__ int h[];
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) h[e] = 0;
  griddep_wait();
  // More blocks than this hold so many SMs that the ranking's, let in now, settle
  // two on one: 500000 x 4 slots of 1024 experts 87 us, 65 if they come at the end.
  if (gridDim.x <= 64) griddep_launch_dependents();
  __syncthreads();
  const int lo = blockIdx.x * p.chunk, hi = min(p.n, lo + p.chunk);
  for (int s = lo + threadIdx.x; s < hi; s += blockDim.x) {
    const int e = load_id(p, s);
    if (e < p.E) atomicAdd(&h[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[(long long)blockIdx.x * p.E + e] = h[e];
}

// Exclusive sum of h[0..n) in shared memory, in place, by the block's first
// warp (by the whole block it took 2100 cycles for 129 values, most of them
// its barriers).
__device__ void exclusive_scan(int* h, int n) {
  if (threadIdx.x < 32) {
    const int per = (n + 31) / 32, lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
    int sum = 0;
    for (int i = lo; i < hi; ++i) sum += h[i];
    int x = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (threadIdx.x >= d) x += y;
    }
    x -= sum;
    for (int i = lo; i < hi; ++i) {
      const int v = h[i];
      h[i] = x;
      x += v;
    }
  }
  __syncthreads();
}

// Ranks of up to S * blockDim.x slots from `base` on among those of the same
// expert, in slot order: wh[warp][e] = slots of e before the warp's, and
// count[e] = all of them.  A warp takes S * 32 consecutive slots; a step costs
// about 1000 cycles, most of them the match, so S is as small as it can be.
template <int S>
__device__ __forceinline__ void rank_slots(const int (&id)[S], int (&rank)[S], int E, uint16_t* wh, int* count) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  for (int i = tid; i < warps * E; i += blockDim.x) wh[i] = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < S; ++q) {
    const unsigned same = __match_any_sync(0xFFFFFFFFu, id[q]);
    const int prior = id[q] < E ? wh[warp * E + id[q]] : 0;
    rank[q] = prior + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (id[q] < E && lane == __ffs(same) - 1) wh[warp * E + id[q]] = (uint16_t)(prior + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) {
    int x = 0;
#pragma unroll 16
    for (int w = 0; w < warps; ++w) {
      const int v = wh[w * E + e];
      wh[w * E + e] = (uint16_t)x;
      x += v;
    }
    count[e] = x;
  }
  __syncthreads();
}

template <int S>
__device__ __forceinline__ void load_ids(const ExpertParams& p, int base, int hi, int (&id)[S]) {
#pragma unroll
  for (int q = 0; q < S; ++q) {
    const int s = base + ((int)(threadIdx.x >> 5) * S + q) * 32 + (threadIdx.x & 31);
    id[q] = s < hi ? load_id(p, s) : p.E;
  }
}

// Writes the slots' rows, and the rows' tokens to row_token where it is given.
template <int S>
__device__ __forceinline__ void store_rows(const ExpertParams& p, const int (&id)[S], const int (&rank)[S], int base, int hi,
                                           const int* start, const uint16_t* wh, int* row_token = nullptr) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int q = 0; q < S; ++q) {
    const int s = base + (warp * S + q) * 32 + lane;
    if (s >= hi) continue;
    int row = -1;
    if (id[q] < p.E) {
      row = start[id[q]] + wh[warp * p.E + id[q]] + rank[q];
      if (row_token) row_token[row] = s / p.k;
    }
    p.slot_row[s] = row;
  }
}

// The whole sort of at most S * blockDim.x slots, in one block.  The rows'
// tokens are put together in shared memory: stored one by one they take a
// cycle each.
template <int S>
__global__ void __launch_bounds__(1024) expert_sort_kernel(ExpertParams p) {
  extern __shared__ int sm[];
  int* start = sm;                                           // E + 1
  int* token = sm + p.E + 1;                                 // n
  uint16_t* wh = reinterpret_cast<uint16_t*>(token + p.n);   // warps x E
  griddep_wait();
  griddep_launch_dependents();
  int id[S], rank[S];
  load_ids(p, 0, p.n, id);
  if (threadIdx.x == 0) start[p.E] = 0;
  rank_slots(id, rank, p.E, wh, start);
  exclusive_scan(start, p.E + 1);
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) p.offsets[e] = start[e];
  store_rows(p, id, rank, 0, p.n, start, wh, token);
  __syncthreads();
  for (int r = threadIdx.x; r < p.n; r += blockDim.x) p.row_token[r] = r < start[p.E] ? token[r] : -1;
}

// Rows of one chunk's slots, S * blockDim.x at a time.  Every block adds up the histograms before its
// own chunk (and all of them, for the experts' offsets), ranks its slots in
// slot order, and writes their rows.  The histograms lie in row_token, which
// other blocks may still be reading, so the next kernel fills that.
template <int S>
__global__ void __launch_bounds__(1024) expert_rank_kernel(ExpertParams p) {
  extern __shared__ int sm[];
  const int E = p.E, tid = threadIdx.x;
  int* start = sm;                                          // E + 1: next row of each expert
  int* total = sm + E + 1;                                  // E + 1
  uint16_t* wh = reinterpret_cast<uint16_t*>(total + E + 1);   // warps x E
  const int lo = blockIdx.x * p.chunk, hi = min(p.n, lo + p.chunk);
  int id[S], rank[S];
  // The histogram's kernel waited for everything before it, so the ids are
  // there before it has ended.
  load_ids(p, lo, hi, id);
  for (int e = tid; e < 2 * (E + 1); e += blockDim.x) sm[e] = 0;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  // parts of the chunks added by different threads, joined by integer adds
  const int parts = max(1, (int)blockDim.x / E);
  for (int i = tid; i < parts * E; i += blockDim.x) {
    const int e = i % E, part = i / E;
    int before = 0, all = 0;
#pragma unroll 8
    for (int c = part; c < p.chunks; c += parts) {
      const int v = p.hist[(long long)c * E + e];
      all += v;
      if (c < (int)blockIdx.x) before += v;
    }
    atomicAdd(&start[e], before);
    atomicAdd(&total[e], all);
  }
  __syncthreads();
  exclusive_scan(total, E + 1);
  for (int e = tid; e < E; e += blockDim.x) start[e] += total[e];
  if (blockIdx.x == 0)
    for (int e = tid; e <= E; e += blockDim.x) p.offsets[e] = total[e];
  for (int base = lo; base < hi; base += S * (int)blockDim.x) {
    if (base > lo) load_ids(p, base, hi, id);
    __syncthreads();
    rank_slots(id, rank, E, wh, total);
    store_rows(p, id, rank, base, hi, start, wh);
    __syncthreads();
    for (int e = tid; e < E; e += blockDim.x) start[e] += total[e];
  }
}

// Number of rows that slots fill.
__device__ __forceinline__ int rows_filled(const ExpertParams& p) { return min(max(p.offsets[p.E], 0), p.n); }

// The rows' tokens, from the slots' rows (a plan of many slots without rows to copy).
constexpr int kTokenSlots = 4;   // per thread
__global__ void __launch_bounds__(kRowThreads) expert_token_kernel(ExpertParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int V = rows_filled(p), s0 = blockIdx.x * (kTokenSlots * kRowThreads) + threadIdx.x;   // below 2^31: n ends 4096 before
  int r[kTokenSlots];
#pragma unroll
  for (int q = 0; q < kTokenSlots; ++q) r[q] = s0 + q * kRowThreads < p.n ? p.slot_row[s0 + q * kRowThreads] : -1;
#pragma unroll
  for (int q = 0; q < kTokenSlots; ++q) {
    const int s = s0 + q * kRowThreads;
    if (r[q] >= 0 && r[q] < p.n) p.row_token[r[q]] = s / p.k;
    if (s >= V && s < p.n) p.row_token[s] = -1;
  }
}

// ---------------------------------------------------------------- rows
// A chunk of CH bytes of a row: 16 where every row allows it, else 4 (one fp32
// or two bf16 elements), else one bf16 element.
template <int CH> struct Raw;
template <> struct Raw<16> { using T = uint4; };
template <> struct Raw<4> { using T = unsigned int; };
template <> struct Raw<2> { using T = unsigned short; };

template <int CH>
__device__ __forceinline__ typename Raw<CH>::T zero_raw() {
  if constexpr (CH == 16) return make_uint4(0, 0, 0, 0);
  else return 0;
}

// CH bytes <-> fp32 values (ES = element size).
template <int ES, int CH>
__device__ __forceinline__ void unpack(typename Raw<CH>::T v, float (&x)[CH / ES]) {
  if constexpr (CH == 16 && ES == 2) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else if constexpr (CH == 16) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  } else if constexpr (ES == 4) {
    x[0] = __uint_as_float(v);
  } else if constexpr (CH == 4) {
    x[0] = __uint_as_float(v << 16);
    x[1] = __uint_as_float(v & 0xFFFF0000u);
  } else {
    x[0] = __uint_as_float((uint32_t)v << 16);
  }
}

template <int ES, int CH>
__device__ __forceinline__ typename Raw<CH>::T pack(const float (&x)[CH / ES]) {
  if constexpr (CH == 16 && ES == 2) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  } else if constexpr (CH == 16) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  } else if constexpr (ES == 4) {
    return __float_as_uint(x[0]);
  } else if constexpr (CH == 4) {
    return pack_bf16x2(x[0], x[1]);
  } else {
    return (uint16_t)pack_bf16x2(x[0], 0.0f);
  }
}

// Chunks are counted without a sign: a row has fewer than 2^31, but a step past its end may pass that.
template <int CH>
__device__ __forceinline__ typename Raw<CH>::T ldc(const void* base, long long row_bytes, long long row, unsigned c) {
  return reinterpret_cast<const typename Raw<CH>::T*>(static_cast<const char*>(base) + row * row_bytes)[c];
}
template <int CH>
__device__ __forceinline__ void stc(void* base, long long row_bytes, long long row, unsigned c, typename Raw<CH>::T v) {
  reinterpret_cast<typename Raw<CH>::T*>(static_cast<char*>(base) + row * row_bytes)[c] = v;
}
// The same, marked as not used again soon.
template <int CH>
__device__ __forceinline__ typename Raw<CH>::T ldc_stream(const void* base, long long row_bytes, long long row, unsigned c) {
  return __ldcs(reinterpret_cast<const typename Raw<CH>::T*>(static_cast<const char*>(base) + row * row_bytes) + c);
}
template <int CH>
__device__ __forceinline__ void stc_stream(void* base, long long row_bytes, long long row, unsigned c, typename Raw<CH>::T v) {
  __stcs(reinterpret_cast<typename Raw<CH>::T*>(static_cast<char*>(base) + row * row_bytes) + c, v);
}

__device__ __forceinline__ float load_weight(const ExpertParams& p, int t, int j) {
  if (!p.weights) return 1.0f;
  const long long at = (long long)t * p.ld_w + j;
  if (p.w_f32) return static_cast<const float*>(p.weights)[at];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.weights)[at] << 16);
}

// Row of slot j of token t; -1 where it is dropped (or not a row at all).
__device__ __forceinline__ int load_row(const ExpertParams& p, int t, int j) {
  if (j >= p.k) return -1;
  const int r = p.slot_row[t * p.k + j];
  return r >= 0 && r < p.n ? r : -1;
}

// Chunks c0, c0 + lanes, ... of token t's row.
template <int CH, int U>
__device__ __forceinline__ void load_chunks(const ExpertParams& p, int t, unsigned c0, unsigned lanes, typename Raw<CH>::T (&x)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c0 + u * lanes < p.nch) x[u] = ldc<CH>(p.in, p.in_pitch, t, c0 + u * lanes);
}

// Copies token t's row to the rows r[0..count), from the chunks in x on; U
// chunks per lane in flight.
template <int CH, int U>
__device__ __forceinline__ void copy_row(const ExpertParams& p, int t, const int* r, int count, unsigned lane, unsigned lanes,
                                         typename Raw<CH>::T (&x)[U]) {
  const unsigned step = lanes * U * gridDim.y;
  for (unsigned c0 = lane + lanes * U * blockIdx.y; c0 < p.nch; c0 += step) {
    for (int j = 0; j < count; ++j) {
      if (r[j] < 0) continue;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * lanes < p.nch) stc<CH>(p.out, p.out_pitch, r[j], c0 + u * lanes, x[u]);
    }
    load_chunks<CH, U>(p, t, c0 + step, lanes, x);
  }
}

// Zeroes row r of p.out, by `lanes` threads of each of the gridDim.y blocks.
template <int CH>
__device__ __forceinline__ void zero_row(const ExpertParams& p, long long r, unsigned lane, unsigned lanes) {
  for (unsigned c = lane + lanes * blockIdx.y; c < p.nch; c += lanes * gridDim.y) stc<CH>(p.out, p.out_pitch, r, c, zero_raw<CH>());
}

// Rows past 16-byte chunks: the last H % (16 / ES) elements of each row go
// element by element through the same code, as a second, short "row".
template <int ES>
__device__ __forceinline__ ExpertParams tail_of(ExpertParams p, int ch) {
  const long long done = (long long)p.nch * ch;
  p.in = static_cast<const char*>(p.in) + done;
  if (p.out) p.out = static_cast<char*>(p.out) + done;
  if (p.in2) p.in2 = static_cast<const char*>(p.in2) + done;
  p.nch = p.tail;
  p.tail = 0;
  return p;
}

// The elements past the last whole chunk, where there are some.
template <int ES>
__device__ __forceinline__ void copy_tail(const ExpertParams& tail, int t, const int* r, int count, unsigned lane, unsigned lanes) {
  typename Raw<ES>::T x[1];
  load_chunks<ES, 1>(tail, t, lane + lanes * blockIdx.y, lanes, x);
  copy_row<ES, 1>(tail, t, r, count, lane, lanes, x);
}

template <int ES, int CH, int U>
__global__ void __launch_bounds__(kRowThreads) expert_gather_kernel(ExpertParams p) {
  extern __shared__ int rows[];   // (threads / lanes) x k
  const int lanes = p.lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int per = kRowThreads / lanes;
  const int t0 = blockIdx.x * per, t = t0 + group;
  // (Loading here takes 1.3 of 54 us off 8192 x 8 slots of 2048 bf16; asking
  // for X in L2 while the slots are sorted gained nothing.)  The sort's
  // kernels waited for whatever wrote X, so it is there before they end.
  typename Raw<CH>::T x[U];
  if (t < p.T) load_chunks<CH, U>(p, t, lane + lanes * U * blockIdx.y, lanes, x);
  griddep_wait();
  griddep_launch_dependents();
  const bool fill = p.tokens_left && blockIdx.y == 0;
  for (int i = threadIdx.x; i < per * p.k; i += kRowThreads) {
    const int t = t0 + i / p.k;
    rows[i] = t < p.T ? load_row(p, t, i % p.k) : -1;
    if (fill && rows[i] >= 0) p.row_token[rows[i]] = t;
  }
  const int V = rows_filled(p);
  __syncthreads();
  if (t >= p.T) return;
  copy_row<CH, U>(p, t, rows + group * p.k, p.k, lane, lanes, x);
  if (p.tail) copy_tail<ES>(tail_of<ES>(p, CH), t, rows + group * p.k, p.k, lane, lanes);
  for (long long r = (long long)V + t; r < p.n; r += p.T) {
    if (fill && lane == 0) p.row_token[r] = -1;
    zero_row<CH>(p, r, lane, lanes);
    if (p.tail) zero_row<ES>(tail_of<ES>(p, CH), r, lane, lanes);
  }
}

// The whole dispatch of few slots in one launch: every block counts its own
// slots' rows against all ids (held in shared memory), then copies.
template <int ES, int CH, int U>
__global__ void __launch_bounds__(kRowThreads) expert_dispatch_small_kernel(ExpertParams p) {
  extern __shared__ int sm[];
  const int lanes = p.lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int per = kRowThreads / lanes;
  const int t0 = blockIdx.x * per, t = t0 + group;
  int* ids = sm;               // n
  int* rows = sm + p.n;        // per * k
  __shared__ int filled;
  if (threadIdx.x == 0) filled = 0;
  griddep_wait();
  griddep_launch_dependents();
  typename Raw<CH>::T x[U];
  if (t < p.T) load_chunks<CH, U>(p, t, lane + lanes * U * blockIdx.y, lanes, x);
  __syncthreads();
  int mine = 0;
  for (int s = threadIdx.x; s < p.n; s += kRowThreads) {
    ids[s] = load_id(p, s);
    mine += ids[s] < p.E;
  }
  if (mine) atomicAdd(&filled, mine);
  __syncthreads();
  const int wl = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kRowThreads / 32;
  for (int i = warp; i < per * p.k; i += warps) {      // a warp counts one slot's row
    const int s = t0 * p.k + i;
    int row = -1;
    if (s < p.n && ids[s] < p.E) {
      const int e = ids[s];
      int c = 0;
      for (int o = wl; o < p.n; o += 32) c += ids[o] < e || (ids[o] == e && o < s);
      row = __reduce_add_sync(0xFFFFFFFFu, c);
    }
    if (wl == 0) {
      rows[i] = row;
      if (s < p.n && blockIdx.y == 0) {
        p.slot_row[s] = row;
        if (row >= 0) p.row_token[row] = s / p.k;
      }
    }
  }
  const int V = filled;
  if (blockIdx.y == 0) {
    for (int e = blockIdx.x * warps + warp; e <= p.E; e += gridDim.x * warps) {
      int c = 0;
      for (int o = wl; o < p.n; o += 32) c += ids[o] < e;
      c = __reduce_add_sync(0xFFFFFFFFu, c);
      if (wl == 0) p.offsets[e] = c;
    }
    for (int r = V + blockIdx.x * kRowThreads + threadIdx.x; r < p.n; r += gridDim.x * kRowThreads) p.row_token[r] = -1;
  }
  __syncthreads();
  if (t >= p.T) return;
  copy_row<CH, U>(p, t, rows + group * p.k, p.k, lane, lanes, x);
  if (p.tail) copy_tail<ES>(tail_of<ES>(p, CH), t, rows + group * p.k, p.k, lane, lanes);
  if (p.nch + p.tail > 0)
    for (long long r = (long long)V + t; r < p.n; r += p.T) {
      zero_row<CH>(p, r, lane, lanes);
      if (p.tail) zero_row<ES>(tail_of<ES>(p, CH), r, lane, lanes);
    }
}

// Rows and weights of the slots j0 .. j0 + KU - 1 of token t.
template <int KU>
__device__ __forceinline__ void load_slots(const ExpertParams& p, int t, int j0, int (&r)[KU], float (&w)[KU]) {
#pragma unroll
  for (int j = 0; j < KU; ++j) {
    r[j] = t < p.T ? load_row(p, t, j0 + j) : -1;
    w[j] = r[j] >= 0 ? load_weight(p, t, j0 + j) : 0.0f;
  }
}

// acc += sum_j w_j in[r_j] over the lane's chunks from c0 on, with all KU U loads in flight.
template <int ES, int CH, int KU, int U>
__device__ __forceinline__ void add_rows(const ExpertParams& p, const int (&r)[KU], const float (&w)[KU], unsigned c0, unsigned lanes,
                                         float (&acc)[U][CH / ES]) {
  constexpr int V = CH / ES;
  typename Raw<CH>::T x[KU][U];
#pragma unroll
  for (int j = 0; j < KU; ++j)
#pragma unroll
    for (int u = 0; u < U; ++u)
      x[j][u] = r[j] >= 0 && c0 + u * lanes < p.nch ? ldc<CH>(p.in, p.in_pitch, r[j], c0 + u * lanes) : zero_raw<CH>();
#pragma unroll
  for (int j = 0; j < KU; ++j)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[V];
      unpack<ES, CH>(x[j][u], f);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[u][v] = fmaf(w[j], f[v], acc[u][v]);
    }
}

// out[t] = sum_j w_j in[r_j].  AHEAD: r, w hold the first KU slots.
template <int ES, int CH, int KU, int U, bool AHEAD>
__device__ __forceinline__ void combine_row(const ExpertParams& p, int t, const int (&r)[KU], const float (&w)[KU], unsigned lane,
                                            unsigned lanes) {
  for (unsigned c0 = lane + lanes * U * blockIdx.y; c0 < p.nch; c0 += lanes * U * gridDim.y) {
    float acc[U][CH / ES] = {};
    if constexpr (AHEAD) add_rows<ES, CH, KU, U>(p, r, w, c0, lanes, acc);
    for (int j0 = AHEAD ? KU : 0; j0 < p.k; j0 += KU) {
      int more[KU];
      float weight[KU];
      load_slots<KU>(p, t, j0, more, weight);
      add_rows<ES, CH, KU, U>(p, more, weight, c0, lanes, acc);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * lanes < p.nch) stc<CH>(p.out, p.out_pitch, t, c0 + u * lanes, pack<ES, CH>(acc[u]));
  }
}

// The first KU slots are loaded before the walk along the row (8192 x 8 rows of
// 2048 bf16: 46.2 us, 0.97 of a copy, against 49.6 with the loads inside it).
// One and two slots: as many blocks as run at once walk over the tokens, each
// with the next token's rows and weights loaded ahead.  8192 rows of 4096
// bf16: one slot 24.0 us against 24.9 with a block per token, two slots 32.8
// against 36.9.  More slots lose by it (4096 tokens of four: 36.2 against 28.6).
// bf16 in smaller chunks loses by all of it, so its slots are loaded inside the
// walk along the row, a block per token: rows of 1001 with one, two, four and
// eight slots 14.9 / 31.0 / 24.7 / 23.9 us against 26.1 / 45.4 / 34.8 / 43.5, of
// 1002 8.7 / 14.4 / 12.2 / 10.5 against 9.2 / 14.5 / 13.9 / 12.5.  (Rows of 1001
// fp32 at two slots: 30.6 inside, 22.1 ahead, the others alike.)
template <int ES, int CH> constexpr bool kAhead = CH == 16 || ES == 4;
template <int ES, int CH, int KU> constexpr bool kWalk = kAhead<ES, CH> && KU <= 2;

template <int ES, int CH, int KU, int U>
__global__ void __launch_bounds__(kRowThreads) expert_combine_kernel(ExpertParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lanes = p.lanes, per = kRowThreads / lanes, lane = threadIdx.x % lanes;
  int t = blockIdx.x * per + threadIdx.x / lanes;
  int r[KU];
  float w[KU];
  if constexpr (kAhead<ES, CH>) load_slots<KU>(p, t, 0, r, w);
  while (t < p.T) {
    int next_r[KU];
    float next_w[KU];
    const int step = gridDim.x * per, next = p.T - t > step ? t + step : p.T;   // t + step may pass 2^31
    if constexpr (kWalk<ES, CH, KU>) load_slots<KU>(p, next, 0, next_r, next_w);
    combine_row<ES, CH, KU, U, kAhead<ES, CH>>(p, t, r, w, lane, lanes);
    if (p.tail) combine_row<ES, ES, KU, 1, kAhead<ES, CH>>(tail_of<ES>(p, CH), t, r, w, lane, lanes);
    if constexpr (!kWalk<ES, CH, KU>) break;
    t = next;
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      r[j] = next_r[j];
      w[j] = next_w[j];
    }
  }
}

// in = dout, in2 = Y, out = dY.  Adds the lane's part of <dout, Y_j> to dot[j].
// Three rows move for each slot and none is read again: with loads and stores
// marked so, 16384 x 4 rows of 4096 bf16 take 180 us (6.7 TB/s) against 202.
// The other kernels do not gain (combine loses 7%).
template <int ES, int CH, int KU, int U>
__device__ __forceinline__ void combine_back_row(const ExpertParams& p, int t, const int (&r)[KU], const float (&w)[KU],
                                                 float (&dot)[KU], unsigned lane, unsigned lanes) {
  using R = typename Raw<CH>::T;
  constexpr int V = CH / ES;
  for (unsigned c0 = lane; c0 < p.nch; c0 += lanes * U) {
    R d[U], y[KU][U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      d[u] = c0 + u * lanes < p.nch ? ldc_stream<CH>(p.in, p.in_pitch, t, c0 + u * lanes) : zero_raw<CH>();
    if (p.dweights) {
#pragma unroll
      for (int j = 0; j < KU; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u)
          y[j][u] = r[j] >= 0 && c0 + u * lanes < p.nch ? ldc_stream<CH>(p.in2, p.in2_pitch, r[j], c0 + u * lanes) : zero_raw<CH>();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + u * lanes >= p.nch) continue;
      float f[V];
      unpack<ES, CH>(d[u], f);
#pragma unroll
      for (int j = 0; j < KU; ++j) {
        if (r[j] < 0) continue;
        if (p.dweights) {
          float g[V];
          unpack<ES, CH>(y[j][u], g);
#pragma unroll
          for (int v = 0; v < V; ++v) dot[j] = fmaf(f[v], g[v], dot[j]);
        }
        if (p.out) {
          float o[V];
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] = w[j] * f[v];
          stc_stream<CH>(p.out, p.out_pitch, r[j], c0 + u * lanes, pack<ES, CH>(o));
        }
      }
    }
  }
}

template <int ES, int CH, int KU, int U>
__global__ void __launch_bounds__(kRowThreads) expert_combine_back_kernel(ExpertParams p) {
  __shared__ float part[KU][kRowThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int lanes = p.lanes, per = kRowThreads / lanes;    // lanes is a multiple of 32
  const int t = blockIdx.x * per + threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int wl = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int j0 = 0; j0 < p.k; j0 += KU) {
    int r[KU];
    float w[KU], dot[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      r[j] = t < p.T ? load_row(p, t, j0 + j) : -1;
      w[j] = r[j] >= 0 ? load_weight(p, t, j0 + j) : 0.0f;
      dot[j] = 0.0f;
    }
    if (t < p.T) {
      combine_back_row<ES, CH, KU, U>(p, t, r, w, dot, lane, lanes);
      if (p.tail) combine_back_row<ES, ES, KU, 1>(tail_of<ES>(p, CH), t, r, w, dot, lane, lanes);
    }
    if (p.dweights) {
#pragma unroll
      for (int j = 0; j < KU; ++j) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
        if (wl == 0) part[j][warp] = dot[j];
      }
      __syncthreads();
      const int warps = lanes / 32, tg = threadIdx.x / KU, j = threadIdx.x % KU;   // one thread per (token, slot)
      if (tg < per && blockIdx.x * per + tg < p.T && j0 + j < p.k) {
        float s = 0.0f;
        for (int i = 0; i < warps; ++i) s += part[j][tg * warps + i];
        const long long at = (long long)(blockIdx.x * per + tg) * p.ld_dw + j0 + j;
        if (p.w_f32) static_cast<float*>(p.dweights)[at] = s;
        else static_cast<uint16_t*>(p.dweights)[at] = (uint16_t)pack_bf16x2(s, 0.0f);
      }
      __syncthreads();
    }
  }
  if (p.out && t < p.T) {
    const int V = rows_filled(p);
    for (long long r = (long long)V + t; r < p.n; r += p.T) {
      zero_row<CH>(p, r, lane, lanes);
      if (p.tail) zero_row<ES>(tail_of<ES>(p, CH), r, lane, lanes);
    }
  }
}

// ---------------------------------------------------------------- launches
cudaError_t launch(const void* kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, ExpertParams& p) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[1] = {&p};
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

// Lanes per token: the power of two in [least, 256] that covers the row with
// U chunks per lane.
int lanes_for(long long nch, int U, int least) {
  int l = least;
  while (l < kRowThreads && (long long)l * U < nch) l *= 2;
  return l;
}

// Token blocks, and where they are too few for the GPU, blocks along the row.
dim3 row_grid(const ExpertParams& p, int U, int sms) {
  const int per = kRowThreads / p.lanes;
  const long long gx = ((long long)p.T + per - 1) / per;
  const long long cols = (p.nch + (long long)p.lanes * U - 1) / ((long long)p.lanes * U);
  long long gy = 1;
  while (gy * 2 <= cols && gx * gy < 2 * sms) gy *= 2;
  return dim3((unsigned)gx, (unsigned)gy);
}

// Bytes per chunk that these rows' addresses allow: 16, 4 or one element.
int chunk_bytes(int es, const void* a, long long pitch_a, const void* b, long long pitch_b, const void* c = nullptr,
                long long pitch_c = 0) {
  const unsigned long long at = reinterpret_cast<uintptr_t>(a) | (unsigned long long)pitch_a | reinterpret_cast<uintptr_t>(b) |
                                (b ? (unsigned long long)pitch_b : 0) | reinterpret_cast<uintptr_t>(c) |
                                (c ? (unsigned long long)pitch_c : 0);
  return at % 16 == 0 ? 16 : (at % 4 == 0 ? 4 : es);
}

void set_chunks(ExpertParams* p, int es, int ch) {
  p->nch = (unsigned)(p->H * es / ch);
  p->tail = (int)(p->H - (long long)p->nch * ch / es);
}

template <template <int, int> class Pick>
const void* kernel_of(int es, int ch) {
  if (es == 4) return ch == 16 ? Pick<4, 16>::get() : Pick<4, 4>::get();
  return ch == 16 ? Pick<2, 16>::get() : (ch == 4 ? Pick<2, 4>::get() : Pick<2, 2>::get());
}

}  // namespace

namespace {

// Chunks of 1024, 2048 or 4096 slots, at most 64 where that can be: every
// block of the ranking adds up all of them.  (131072 slots of 256 experts in
// 128 / 64 / 32 chunks: 11.8 / 10.4 / 12.2 us; 262144 in 128 / 64: 14.1 / 13.9.)
// Their histograms have to fit n integers.
int expert_chunks(long long n, int experts) {
  const int per = n <= 65536 ? 1024 : (n <= 131072 ? 2048 : 4096);
  long long c = (n + per - 1) / per;
  if (c > kExpertMaxChunks) c = kExpertMaxChunks;
  if (c > n / experts) c = n / experts;
  return (int)c;
}

// 8192 rows of 1002 bf16, one slot each: 15.2 / 12.6 us with 4 / 8 chunks of 4
// bytes; of 1001, 24.3 / 23.6 / 18.8 us with 2 / 4 / 8 elements.
constexpr int gather_chunks(int ch) { return ch == 16 ? 2 : 8; }
template <int ES, int CH> struct SmallDispatch {
  static const void* get() { return (const void*)expert_dispatch_small_kernel<ES, CH, gather_chunks(CH)>; }
};
template <int ES, int CH> struct Gather {
  static const void* get() { return (const void*)expert_gather_kernel<ES, CH, gather_chunks(CH)>; }
};

}  // namespace

cudaError_t launch_expert_dispatch(ExpertParams p, int es, int sms, cudaStream_t stream, LaunchInfo* info) {
  const int ch = chunk_bytes(es, p.in, p.in_pitch, p.out, p.out_pitch);
  set_chunks(&p, es, ch);
  const int U = gather_chunks(ch);
  p.lanes = lanes_for(p.nch, U, 8);
  if (p.n <= kExpertSmallSlots) {
    if (p.lanes < 32) p.lanes = 32;    // counting rows is the work here: 8 tokens a block at most
    if (p.T < 1) p.lanes = kRowThreads;
    dim3 grid = row_grid(p, U, sms);
    if (grid.x < 1) grid.x = 1;
    const size_t smem = ((size_t)p.n + (size_t)(kRowThreads / p.lanes) * p.k) * sizeof(int);
    const void* f = kernel_of<SmallDispatch>(es, ch);
    *info = LaunchInfo{};
    info->grid = grid.x * grid.y; info->cluster = 1; info->block = kRowThreads; info->smem_bytes = (int)smem;
    info->kernel = "expert_dispatch_small_kernel";
    return launch(f, grid, kRowThreads, smem, stream, p);
  }
  auto rank_bytes = [](int E) { return 2 * ((size_t)E + 1) * sizeof(int) + (size_t)32 * E * sizeof(uint16_t); };
  auto sort_bytes = [](int E, int n) { return ((size_t)E + 1 + n) * sizeof(int) + (size_t)32 * E * sizeof(uint16_t); };
  const void* ranks[3] = {(const void*)expert_rank_kernel<1>, (const void*)expert_rank_kernel<2>, (const void*)expert_rank_kernel<4>};
  const void* sorts[3] = {(const void*)expert_sort_kernel<1>, (const void*)expert_sort_kernel<2>, (const void*)expert_sort_kernel<4>};
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && !configured[dev]) {
    constexpr cudaFuncAttribute kSmem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    for (const void* f : ranks)
      if (e == cudaSuccess) e = cudaFuncSetAttribute(f, kSmem, (int)rank_bytes(kExpertMax));
    for (const void* f : sorts)
      if (e == cudaSuccess) e = cudaFuncSetAttribute(f, kSmem, (int)sort_bytes(kExpertMax, kExpertOneBlock));
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  *info = LaunchInfo{};
  if (p.n <= kExpertOneBlock) {
    const size_t bytes = sort_bytes(p.E, p.n);
    if ((e = launch(sorts[p.n <= 1024 ? 0 : (p.n <= 2048 ? 1 : 2)], dim3(1), 1024, bytes, stream, p))) return e;
    info->grid = 1; info->cluster = 1; info->block = 1024; info->smem_bytes = (int)bytes;
    info->kernel = "expert_sort_kernel";
  } else {
    p.chunks = expert_chunks(p.n, p.E);
    p.hist = p.row_token;
    p.tokens_left = 1;
    p.chunk = (int)(((long long)p.n + p.chunks - 1) / p.chunks);
    if ((e = launch((const void*)expert_hist_kernel, dim3(p.chunks), 1024, (size_t)p.E * sizeof(int), stream, p))) return e;
    if ((e = launch(ranks[p.chunk <= 1024 ? 0 : (p.chunk <= 2048 ? 1 : 2)], dim3(p.chunks), 1024, rank_bytes(p.E), stream, p))) return e;
    info->grid = p.chunks; info->cluster = 1; info->block = 1024; info->smem_bytes = (int)rank_bytes(p.E);
    info->kernel = "expert_rank_kernel";
  }
  if (p.H == 0 && !p.tokens_left) return cudaSuccess;
  if (p.H == 0) {
    // 8192 x 8 slots of 128 experts: 7.6 us with this launch, 65536 x 4 of 256: 13.5.
    const int per = kTokenSlots * kRowThreads;
    return launch((const void*)expert_token_kernel, dim3((p.n + per - 1) / per), kRowThreads, 0, stream, p);
  }
  const dim3 grid = row_grid(p, U, sms);
  const size_t smem = (size_t)(kRowThreads / p.lanes) * p.k * sizeof(int);
  const void* f = kernel_of<Gather>(es, ch);
  info->grid = grid.x * grid.y; info->block = kRowThreads; info->smem_bytes = (int)smem;
  info->kernel = "expert_gather_kernel";
  return launch(f, grid, kRowThreads, smem, stream, p);
}

namespace {

// Chunks per lane in flight, for KU slots at once.  Measured in us with rows of
// 4096 bf16 in 16-byte chunks and of 1002 and 1001 bf16 in 4- and 2-byte ones,
// 400 MB of them in rotation, 8192 tokens of one and two slots, 4096 of four,
// 2048 of eight, for U = 1 / 2 / 4 / 8:
//                    16-byte                      4-byte                       2-byte
//   combine, KU = 1   26.4 / 29.4 / 24.6 / 24.7    19.1 / 14.9 /  9.9 /  8.6    29.2 / 25.6 / 23.8 / 14.9
//            KU = 2   32.3 / 32.6 / 33.2 / 44.3    21.0 / 17.5 / 14.4 / 17.3    32.2 / 23.5 / 31.0 / 31.2
//            KU = 4   27.4 / 30.9 / 46.7 / 38.0    15.9 / 12.2 / 11.2 / 13.5    24.3 / 24.7 / 25.7 / 34.1
//            KU = 8   24.5 / 29.2 / 34.6 /  187    12.6 / 10.6 / 11.6 / 11.3    28.4 / 23.9 / 34.7 / 43.0
//   gradient KU = 1   36.1 / 34.3 / 32.5 / 33.8    22.1 / 18.9 / 14.2 / 13.2    29.7 / 27.2 / 26.4 / 21.9
//            KU = 2   54.6 / 53.4 / 55.5 / 64.4    30.8 / 26.2 / 19.8 / 18.3    43.1 / 39.6 / 36.3 / 29.2
//            KU = 4   47.5 / 52.2 / 47.5 / 54.8    26.1 / 19.9 / 17.1 / 20.4    40.2 / 30.3 / 28.1 / 32.7
//            KU = 8   47.9 / 45.6 / 52.3 / 89.3    28.9 / 24.6 / 19.6 / 19.6    41.6 / 38.4 / 32.4 / 31.4
// Both small chunks share a rule.  Not the best here: combine's KU = 2 in 2-byte
// chunks and KU = 4 in 4-byte ones, and the gradient's 16-byte chunks with one
// and eight slots, which earlier measurements with less in rotation preferred.
constexpr int combine_chunks(int ku, int ch) { return ch == 16 ? (ku >= 4 ? 1 : 4 / ku) : (ku >= 4 ? 2 : 8 / ku); }
constexpr int back_chunks(int ku, int ch) { return ch == 16 ? (ku >= 4 ? 1 : 2) : (ku >= 4 ? 4 : 8); }

template <int KU> struct ForSlots {
  template <int ES, int CH> struct Combine {
    static const void* get() { return (const void*)expert_combine_kernel<ES, CH, KU, combine_chunks(KU, CH)>; }
  };
  template <int ES, int CH> struct Back {
    static const void* get() { return (const void*)expert_combine_back_kernel<ES, CH, KU, back_chunks(KU, CH)>; }
  };
};
int slots_unrolled(int k) { return k <= 1 ? 1 : (k <= 2 ? 2 : (k <= 4 ? 4 : 8)); }

}  // namespace

cudaError_t launch_expert_combine(ExpertParams p, int es, int sms, cudaStream_t stream, LaunchInfo* info) {
  const int ch = chunk_bytes(es, p.in, p.in_pitch, p.out, p.out_pitch);
  set_chunks(&p, es, ch);
  const int ku = slots_unrolled(p.k);
  const int U = combine_chunks(ku, ch);
  p.lanes = lanes_for(p.nch, U, 1);
  dim3 grid = row_grid(p, U, sms);
  const void* f = ku == 1   ? kernel_of<ForSlots<1>::Combine>(es, ch)
                  : ku == 2 ? kernel_of<ForSlots<2>::Combine>(es, ch)
                  : ku == 4 ? kernel_of<ForSlots<4>::Combine>(es, ch)
                            : kernel_of<ForSlots<8>::Combine>(es, ch);
  if (ku <= 2 && (ch == 16 || es == 4)) {
    static int resident[64][2][3] = {};   // blocks per SM by slots and chunk
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int& blocks = resident[dev][ku - 1][es == 2 ? 0 : (ch == 16 ? 1 : 2)];
    if (blocks == 0) {
      int got = 0;
      if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&got, f, kRowThreads, 0))) return e;
      blocks = got > 0 ? got : 1;
    }
    if (grid.x > (unsigned)(blocks * sms)) grid.x = blocks * sms;
  }
  *info = LaunchInfo{};
  info->grid = grid.x * grid.y; info->cluster = 1; info->block = kRowThreads;
  info->kernel = "expert_combine_kernel";
  return launch(f, grid, kRowThreads, 0, stream, p);
}

cudaError_t launch_expert_combine_back(ExpertParams p, int es, int sms, cudaStream_t stream, LaunchInfo* info) {
  const int ch = chunk_bytes(es, p.in, p.in_pitch, p.out, p.out_pitch, p.in2, p.in2_pitch);
  set_chunks(&p, es, ch);
  const int ku = slots_unrolled(p.k);
  const int U = back_chunks(ku, ch);
  p.lanes = lanes_for(p.nch, U, 32);
  const int per = kRowThreads / p.lanes;
  const dim3 grid((p.T + per - 1) / per);
  const void* f = ku == 1   ? kernel_of<ForSlots<1>::Back>(es, ch)
                  : ku == 2 ? kernel_of<ForSlots<2>::Back>(es, ch)
                  : ku == 4 ? kernel_of<ForSlots<4>::Back>(es, ch)
                            : kernel_of<ForSlots<8>::Back>(es, ch);
  *info = LaunchInfo{};
  info->grid = grid.x; info->cluster = 1; info->block = kRowThreads;
  info->kernel = "expert_combine_back_kernel";
  return launch(f, grid, kRowThreads, 0, stream, p);
}

}  // namespace gtn
