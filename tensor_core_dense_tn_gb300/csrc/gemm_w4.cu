// Products with 4-bit weights for few tokens (gemm_w4_tn, gemm_w4_tn_experts):
//
//   D[m, n] = act(alpha * sum_g s[n, g] * sum_{k in g} A[m, k] (q[n, k] - z[n, g]))
//
// Bound by the read of the codes (half a byte per weight) and the scales.
// The differences q - z are whole numbers below 256 in magnitude, so they are
// exact in bf16: a group's products run on the tensor cores (fp32 sums) with
// no rounding of the weights, and the scale multiplies the group's fp32 sum.
//
// Two CTAs per SM work through items, each a tile of 128 weight rows and the
// rows of A of one matrix, or a part of their K: the parts of a tile are the
// CTAs of a cluster, which add their fp32 sums through distributed shared
// memory in part order (no workspace, no atomics).  Four copying warps keep a
// ring of stages of 256 k ahead, across items: codes by TMA (128 x 128-byte
// boxes, 16 KiB), activations by asynchronous copies, scales and zero points
// through registers, a slab of eight groups ahead.  Eight warps multiply: two
// sets, each half of a stage's k, of four warps with 32 rows each.
//
// Measured (replayed in a graph, weights larger than L2 in rotation, against
// the time of a copy of the same bytes):
//    1 token  x 8192 x 8192,  groups of 128                    12.5 us   5.1
//   16 tokens x 28672 x 4096, groups of 128, zero points       27.6 us   9.2
//    5 tokens x 5000 x 2000,  groups of 32, fp32 result         8.6 us   0.9
//    1 token through 8 of 64 experts of 4096 x 2048            12.9 us   5.1
//   32 tokens, 2 of 16 experts of 8192 x 4096, groups of 64    65.6 us  42.9
// What bounds it is the multiplying warps' dependent chain (code word, unpacking,
// two mma into the same sums) with four of them per scheduler, more than memory:
// with the ring alone (nothing multiplied) the same calls take 8.8, 13.7, 6.4,
// 9.0 and 48.5 us, with two stages instead of three or four the first four take
// no longer, and with the weights in L2 they gain 1.5 us.  Nor is it the issue
// of instructions or the tensor pipe: counters show 38-52% of the issue slots
// and 11-18% of the pipe in use, and unpacking without the fma took longer.  A
// stage is about 3500 warp instructions; its four steps take a warp 1250 cycles
// where one CTA has the SM and 1650 where two do.  Removing the unpacking or the
// mma alone gains 10%, both 45%.  The ring alone is short of the copy too: its
// thread 0 asks for a stage's codes only after its warp has stored the scales of
// the one before.  Slower or equal: one CTA per SM with 16 multiplying warps;
// three CTAs; 96-row tiles; ranges of equal length across tiles, joined in
// memory (24.3 us for 16 tokens, but 13.9 us for one and 76.7 for 32; no rule
// chooses between the two); activations by bulk copies; a first copy of codes
// before the scales' loads.
//
// mma.sync and not tcgen05.mma: the latter takes at least 27 ns whatever its
// number of columns up to 64, so that 128 x 256 weights hold the tensor core
// 0.44 us and more, and 16 KiB arrive every 0.37 us.  With the weights
// unpacked into Tensor Memory as its A operand it was right and slower: 103
// us for the last of these calls.
//
// Fragments.  mma.m16n8k16 sums over k, so k may be permuted as long as both
// operands agree.  A lane (row r = lane / 4, q = lane % 4) reads the word that
// holds k = 8 q .. 8 q + 7 of its row in a block of 32.  Masking the word
// leaves the nibbles i and i + 4 in the two halves of a register, either at
// bits 0-3 or at bits 4-7.  Read as bf16, a half with only its low eight bits
// set is that whole number times 2^-133 (below 128 it is subnormal, and the
// first normal binade continues the same spacing), so one packed fma with
// 2^127 or 2^123 and -z 2^-6 gives (q - z) 2^-6, exactly, with one shift per
// eight weights.  The 2^6 is put back with alpha.  The activations are staged
// as they are and take the same pairs (0,4) (1,5) (2,6) (3,7) when a fragment is read.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace gtn {
namespace {

constexpr int kWarps = 8;                           // warps that multiply
constexpr int kAuxThreads = 128;                    // one per weight row: copies, scales
constexpr int kThreads = 32 * kWarps + kAuxThreads;
constexpr int kStageBytes = kW4TileRows * 128;
constexpr int kStepK = 32;                          // k per step: two mma
constexpr int kSteps = kW4StageK / kStepK;          // steps per stage
constexpr int kSets = 2;                            // halves of a stage's steps, each with warps for all rows
constexpr int kWarpSteps = kSteps / kSets;
constexpr int kErrTimeout = -5;
constexpr int kCtasPerSm = 2;
constexpr int kMaxSplit = 8;

// Waits (bounded) for a phase; false if it gave up or another warp did.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint64_t timeout_ns,
                                       int* status, int role) {
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer() - t0 > timeout_ns) {
      *abort_flag = 1;
      if (atomicCAS(&status[0], 0, kErrTimeout) == 0) status[1] = (role << 24) | (int)(blockIdx.x & 0xFFFFFF);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                         uint64_t timeout_ns, int* status, int role) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, abort_flag, timeout_ns, status, role);
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with no sum to add to.
__device__ __forceinline__ void mma_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

constexpr uint32_t kTwo127 = 0x7F007F00u, kTwo123 = 0x7D007D00u, kMinusTwo127 = 0xFF00FF00u;   // bf16 pairs
constexpr float kUnit = 64.0f;                                      // fragments hold (q - z) / 64

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The eight codes of `word` as bf16 pairs (0,4) (1,5) (2,6) (3,7) of (q - z) / 64.
__device__ __forceinline__ void differences(uint32_t word, uint32_t minus_z, uint32_t (&d)[4]) {
  const uint32_t high = word >> 8;
  d[0] = fma_bf16x2(word & 0x000F000Fu, kTwo127, minus_z);
  d[1] = fma_bf16x2(word & 0x00F000F0u, kTwo123, minus_z);
  d[2] = fma_bf16x2(high & 0x000F000Fu, kTwo127, minus_z);
  d[3] = fma_bf16x2(high & 0x00F000F0u, kTwo123, minus_z);
}

// Asynchronous 16-byte copy of which the first `bytes` are read, zeros after them.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}
// Arrives on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Sum of one token's column: [token][row], padded so that a warp's fragment
// stores (8 rows x 4 token pairs) fall in different banks.
constexpr int kRedPitch = kW4TileRows + 4;

__host__ __device__ constexpr int act_bytes(int nt) { return kSteps * nt * 512; }                              // per stage
__host__ __device__ constexpr int scale_bytes(int fl) { return kSteps / fl * kW4TileRows * (int)sizeof(uint2); }   // per stage
__host__ __device__ constexpr int red_bytes(int nt) { return 8 * nt * kRedPitch * 4; }
__host__ __device__ constexpr int ring_bytes(int nt, int fl, int stages) {
  return 1024 + stages * (kStageBytes + act_bytes(nt) + scale_bytes(fl)) + red_bytes(nt);
}
// As many stages, up to four, as leave room for two CTAs on an SM (and 7 KiB for the list of experts).
__host__ __device__ constexpr int ring_stages(int nt, int fl) { return ring_bytes(nt, fl, 4) <= 105 * 1024 ? 4 : 3; }
__host__ __device__ constexpr int smem_for(int nt, int fl) { return ring_bytes(nt, fl, ring_stages(nt, fl)); }
__host__ __device__ constexpr int list_bytes(int experts) { return experts ? (experts + 1) * 4 + experts * 2 : 0; }

// A block's shared memory, and the work of its cluster: items of one weight
// tile and the rows of one matrix (an expert's, or one block of tokens).
struct W4Block {
  int items, tiles, active;  // active: matrices with rows, or blocks of tokens
  int first, step;           // this cluster's items
  int kb0, count_kb;         // this part's stages
  const int* list_lo;        // experts: first row of the y-th matrix that has rows, and one past the last row
  const uint16_t* list_id;   // experts: that matrix
  uint32_t ring;             // codes, 16 KiB a stage
  uint32_t acts;             // a stage: [k / 32][token][32 k]
  unsigned char* base;       // = ring
  unsigned char* act_base;   // = acts
  uint2* scales;             // a stage: [group][row] of s, -z / 64 twice
  float* red;
  uint32_t full, empty;      // a barrier per stage
  volatile uint32_t* abort_flag;
};

struct W4Item {
  int expert, lo, hi, n0;    // matrix, rows of A, first weight row
};

template <int NT>
__device__ __forceinline__ W4Item item_of(const W4Params& p, const W4Block& k, int item) {
  W4Item w;
  if (p.offsets) {           // an expert's tiles follow one another
    const int y = item / k.tiles;
    w.n0 = (item - y * k.tiles) * kW4TileRows;
    w.expert = k.list_id[y];
    w.lo = k.list_lo[y];
    w.hi = k.list_lo[y + 1];
  } else {                   // a tile's blocks of tokens follow one another, so that its codes are in L2
    const int tile = item / k.active;
    w.n0 = tile * kW4TileRows;
    w.expert = 0;
    w.lo = (item - tile * k.active) * 8 * NT;
    w.hi = min(p.M, w.lo + 8 * NT);
  }
  return w;
}

// Lists the matrices that have rows; returns their number.  The rows of the
// y-th are lo[y] .. lo[y + 1]: offsets[e] .. offsets[e + 1] of a plan in order,
// and for offsets that decrease up to the next one's first, which may be none.
// The last one's end at offsets[E], where the rows of zeros begin.
__device__ int list_experts(const W4Params& p, int* lo, uint16_t* id) {
  __shared__ int warp_count[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int before = 0;
  for (int e0 = 0; e0 < p.E; e0 += kThreads) {
    const int e = e0 + tid;
    int a = 0, b = 0;
    if (e < p.E) {
      a = min(max(p.offsets[e], 0), p.M);
      b = min(max(p.offsets[e + 1], a), p.M);
    }
    const unsigned some = __ballot_sync(0xFFFFFFFFu, b > a);
    if (lane == 0) warp_count[warp] = __popc(some);
    __syncthreads();
    int at = before;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += warp_count[w];
      before += warp_count[w];
    }
    // One writer per entry: in a caller's own plan the next one's lo may be another row than b, and the
    // CTAs of a cluster have to come to the same list (they meet once for each block of its rows).
    if (tid == 0) lo[before] = min(max(p.offsets[p.E], 0), p.M);
    if (b > a) {
      at += __popc(some & ((1u << lane) - 1));
      id[at] = (uint16_t)e;
      lo[at] = a;
    }
    __syncthreads();
  }
  return before;
}

template <bool S_F32>
struct RawScales {           // eight groups' scales and zero points of a row, as loaded
  uint32_t s[S_F32 ? 8 : 4];
  uint32_t z[2];
};

// The copying half: keeps the ring ahead of the multiplying warps, across
// items.
template <int NT, int FL, bool SPLIT, bool S_F32>
__device__ __forceinline__ void w4_copy(const CUtensorMap* tm, const W4Params& p, const W4Block& k) {
  constexpr int kTok = 8 * NT, kFlushes = kSteps / FL, kStages = ring_stages(NT, FL);
  constexpr int kSlab = FL == kSteps ? 1 : FL;            // stages whose scales are loaded together
  constexpr int kGroups = kFlushes * kSlab;               // 8, or 1 where a group is a stage or longer
  const int tid = threadIdx.x - 32 * kWarps, lane = tid & 31;
  const int tok = (tid >> 2) % kTok;                      // this thread's token and weight row of an item
  int slot = 0, phase = 1, fetched = 0;                   // phase: of the empty barriers (the first round passes)
  bool ok = true;                                         // false after a wait that gave up: nothing more is copied

  for (int item = k.first; item < k.items; item += k.step) {
    const W4Item w = item_of<NT>(p, k, item);
    const int n = w.n0 + tid;
    const bool has_row = n < p.N;
    const char* s_row = static_cast<const char*>(p.scales) + (w.expert * p.stride_s + n * p.ld_s) * (S_F32 ? 4 : 2);
    const uint8_t* z_row = p.zeros && has_row ? p.zeros + w.expert * p.stride_z + n * p.ld_z : nullptr;

    auto load_scales = [&](int stage, RawScales<S_F32>& r) {
      const int kb = k.kb0 + stage;
      const int g0 = FL == kSteps ? kb / (p.group / kW4StageK) : kb * kFlushes;
      const int count = has_row ? min(max(p.ngroups - g0, 0), kGroups) : 0;
      r.z[0] = r.z[1] = 0x08080808u;
      if (z_row) {
        const uint8_t* z = z_row + g0;
        if (count == 8 && (reinterpret_cast<uintptr_t>(z) & 7) == 0) {
          const uint2 v = *reinterpret_cast<const uint2*>(z);
          r.z[0] = v.x;
          r.z[1] = v.y;
        } else {
#pragma unroll
          for (int j = 0; j < kGroups; ++j)
            if (j < count) r.z[j / 4] = __byte_perm(r.z[j / 4], z[j], 0x3210 + ((4 - j % 4) << (4 * (j % 4))));
        }
      }
      const char* sp = s_row + (long long)g0 * (S_F32 ? 4 : 2);
      if (count == 8 && (reinterpret_cast<uintptr_t>(sp) & 15) == 0) {
#pragma unroll
        for (int j = 0; j < (S_F32 ? 2 : 1); ++j) {
          const uint4 v = reinterpret_cast<const uint4*>(sp)[j];
          r.s[4 * j] = v.x; r.s[4 * j + 1] = v.y; r.s[4 * j + 2] = v.z; r.s[4 * j + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < (S_F32 ? 8 : 4); ++j) r.s[j] = 0;
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          if (j >= count) continue;
          if constexpr (S_F32) r.s[j] = reinterpret_cast<const uint32_t*>(sp)[j];
          else r.s[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(sp)[j] << (16 * (j & 1));
        }
      }
    };

    for (int m0 = w.lo; m0 < w.hi; m0 += kTok) {
      const int count = min(kTok, w.hi - m0);
      const uint16_t* a_row = static_cast<const uint16_t*>(p.A);
      int a_len = 0;   // elements of the row; 0 = a row of zeros
      if (tok < count) {
        const long long r = p.a_rows ? p.a_rows[m0 + tok] : m0 + tok;
        if (r >= 0 && r < p.a_count) {
          a_row += r * p.lda;
          a_len = p.K;
        }
      }
      RawScales<S_F32> next;
      if (k.count_kb > 0 && ok) load_scales(0, next);
      for (int i0 = 0; i0 < k.count_kb && ok; i0 += kSlab) {
        const RawScales<S_F32> cur = next;
        if (i0 + kSlab < k.count_kb) load_scales(i0 + kSlab, next);
#pragma unroll
        for (int u = 0; u < kSlab; ++u) {
          const int i = i0 + u;
          if (i >= k.count_kb || !ok) break;
          ok = __all_sync(0xFFFFFFFFu, wait_bar(k.empty + 8 * slot, phase, k.abort_flag, p.timeout_ns, p.status, kRoleProducer));
          if (!ok) break;
          // Codes by TMA, activations by 16-byte asynchronous copies that arrive on the same barrier.
          if (tid == 0) {
            mbar_arrive_expect_tx(k.full + 8 * slot, kStageBytes);
            tma_load_3d(k.ring + slot * kStageBytes, tm, (k.kb0 + i) * 128, w.n0, w.expert, k.full + 8 * slot);
          }
          ++fetched;
          if (tok < count) {
#pragma unroll
            for (int t = 0; t < kSteps * kTok * 4 / kAuxThreads; ++t) {
              const int k32 = (tid + t * kAuxThreads) / (4 * kTok), at = (k.kb0 + i) * kW4StageK + k32 * kStepK + (tid & 3) * 8;
              const int bytes = min(max(a_len - at, 0), 8) * 2;
              cp_async_16(k.acts + slot * act_bytes(NT) + (k32 * kTok + tok) * 64 + (tid & 3) * 16, bytes > 0 ? a_row + at : a_row,
                          bytes);
            }
          }
          cp_async_arrive(k.full + 8 * slot);
          uint2* to = k.scales + slot * kFlushes * kW4TileRows + tid;
#pragma unroll
          for (int f = 0; f < kFlushes; ++f) {
            const int j = u * kFlushes + f;
            const uint32_t sv = S_F32 ? cur.s[j] : (j & 1 ? cur.s[j / 2] & 0xFFFF0000u : cur.s[j / 2] << 16);
            const uint32_t zz = __byte_perm(cur.z[j / 4], 0, 0x4040 + 0x0101 * (j % 4));    // the byte in both halves
            to[f * kW4TileRows] = make_uint2(sv, fma_bf16x2(zz, kMinusTwo127, 0));          // -z / 64, exact
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(k.full + 8 * slot);
          if (++slot == kStages) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if constexpr (SPLIT) {   // a cluster's barrier counts every thread: these two are the multiplying warps'
        cluster_sync();
        cluster_sync();
      }
    }
  }
  cp_async_wait_all();
  __syncthreads();
  // After a wait that gave up, copies may still be in flight: they land
  // (bounded) before the shared memory is given back.
  if (tid == 0 && *k.abort_flag) {
    const uint64_t t0 = globaltimer();
    for (int i = 0; i < min(kStages, fetched); ++i) {
      const int at = fetched - 1 - i;
      while (!mbar_try_wait(k.full + 8 * (at % kStages), (at / kStages) & 1) && globaltimer() - t0 < p.timeout_ns) {
      }
    }
  }
}

// The multiplying half.
template <int NT, int FL, bool SPLIT>
__device__ __forceinline__ void w4_multiply(const W4Params& p, const W4Block& k, int part) {
  constexpr int kTok = 8 * NT, kFlushes = kSteps / FL, kStages = ring_stages(NT, FL);
  constexpr int kSeg = FL < kWarpSteps ? FL : kWarpSteps;   // steps of one scale
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = lane >> 2, q = lane & 3;
  const int r0 = (warp % (kWarps / kSets)) * 32 + row, set = warp / (kWarps / kSets);   // rows r0, + 8, + 16, + 24
  const int col = ((row ^ (set * kWarpSteps)) << 4) | (q << 2);

  int slot = 0, phase = 0;
  bool ok = true;   // false after a wait that gave up: the results are undefined, the barriers are still met
  for (int item = k.first; item < k.items; item += k.step) {
    const W4Item w = item_of<NT>(p, k, item);
    for (int m0 = w.lo; m0 < w.hi; m0 += kTok) {   // the weights are streamed once for each block of tokens
      const int count = min(kTok, w.hi - m0);
      float tot[2][NT][4];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) tot[s][t][j] = 0.0f;

      // Lanes of tokens that are not there read the last one's: a column of B
      // only reaches its own column of the result, which is not stored.
      int act_at[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
        act_at[t] = set * kWarpSteps * kTok * 64 + (t * 8 + min(row, max(count - 8 * t, 1) - 1)) * 64 + q * 16;

      for (int i = 0; i < k.count_kb && ok; ++i) {
        // one answer per warp: its lanes go on together
        ok = __all_sync(0xFFFFFFFFu, wait_bar(k.full + 8 * slot, phase, k.abort_flag, p.timeout_ns, p.status, kRoleMma));
        if (!ok) break;
        const unsigned char* codes = k.base + slot * kStageBytes + r0 * 128;
        const uint2* sc = k.scales + slot * kFlushes * kW4TileRows + (FL == kSteps ? 0 : set * (kWarpSteps / kSeg)) * kW4TileRows + r0;
        const unsigned char* act = k.act_base + slot * act_bytes(NT);
#pragma unroll
        for (int f = 0; f < kWarpSteps / kSeg; ++f) {
          uint2 sz[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) sz[j] = sc[f * kW4TileRows + 8 * j];
          float acc[2][NT][4];
          // two tiles of tokens: all four steps at once spill registers (28.4 against 27.4 us)
          constexpr int kUnroll = NT == 2 && kSeg > 2 ? 2 : kSeg;
          if constexpr (kUnroll < kSeg) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[s][t][j] = 0.0f;
          }
#pragma unroll (kUnroll)
          for (int h = 0; h < kSeg; ++h) {
            const int step = f * kSeg + h;
            // 128-byte swizzle: the 16-byte column c of row r sits at c ^ (r % 8)
            const unsigned char* at = codes + (col ^ (step << 4));
            uint4 b[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint4 w = *reinterpret_cast<const uint4*>(act + act_at[t] + step * kTok * 64);
              b[t] = make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632),    // (0,4) (1,5)
                                __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));   // (2,6) (3,7)
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              uint32_t da[4], db[4];
              differences(*reinterpret_cast<const uint32_t*>(at + 16 * s * 128), sz[2 * s].y, da);
              differences(*reinterpret_cast<const uint32_t*>(at + (16 * s + 8) * 128), sz[2 * s + 1].y, db);
              const uint32_t a0[4] = {da[0], db[0], da[1], db[1]}, a1[4] = {da[2], db[2], da[3], db[3]};
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                if (kUnroll == kSeg && h == 0) mma_16816_first(acc[s][t], a0, b[t].x, b[t].y);
                else mma_16816(acc[s][t], a0, b[t].x, b[t].y);
                mma_16816(acc[s][t], a1, b[t].z, b[t].w);
              }
            }
          }
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tot[s][t][j] = fmaf(__uint_as_float(sz[2 * s + j / 2].x), acc[s][t][j], tot[s][t][j]);
        }
        // The stage's codes were read as ordinary memory and are next written by
        // a TMA copy: without this fence a late read of the last step's words
        // met the next codes (a few rows in half a million, in calls of
        // several items per CTA).
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k.empty + 8 * slot);
        if (++slot == kStages) {
          slot = 0;
          phase ^= 1;
        }
      }
      // The second set's sums go through shared memory to the first, whose
      // warps hold the same rows; then, with several parts, each finishes its
      // share of the tile's elements, adding the parts in order.
      auto each = [&](auto f) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) f(k.red[(t * 8 + 2 * q + (j & 1)) * kRedPitch + r0 + 16 * s + 8 * (j >> 1)], tot[s][t][j]);
      };
      if (set == 1) each([](float& at, float v) { at = v; });
      named_bar_sync(1, 32 * kWarps);
      if (set == 0) each([](float& at, float v) { at += v; });
      if constexpr (SPLIT) cluster_sync();
      else named_bar_sync(1, 32 * kWarps);
      auto store = [&](int m, int rr, float v) {
        const long long d = (long long)(m0 + m) * p.ldd + w.n0 + rr;
        if (p.out_f32) static_cast<float*>(p.D)[d] = v;
        else static_cast<uint16_t*>(p.D)[d] = (uint16_t)pack_bf16x2(v, 0.0f);
      };
      if constexpr (SPLIT) {
        const int total = count * kW4TileRows, share = (total + p.split - 1) / p.split, end = min(total, (part + 1) * share);
        for (int i = part * share + tid; i < end; i += 32 * kWarps) {
          const int m = i / kW4TileRows, rr = i % kW4TileRows;
          const uint32_t at = smem_u32(k.red + m * kRedPitch + rr);
          float y[kMaxSplit], v = 0.0f;
#pragma unroll
          for (int j = 0; j < kMaxSplit; ++j) y[j] = j < p.split ? ld_cluster_f32(mapa_shared(at, j)) : 0.0f;
#pragma unroll
          for (int j = 0; j < kMaxSplit; ++j) v += y[j];
          if (w.n0 + rr < p.N) store(m, rr, activate(p.alpha * (kUnit * v), p.act));
        }
      } else {
        for (int i = tid; i < count * kW4TileRows; i += 32 * kWarps) {
          const int m = i / kW4TileRows, rr = i % kW4TileRows;
          if (w.n0 + rr < p.N) store(m, rr, activate(p.alpha * (kUnit * k.red[m * kRedPitch + rr]), p.act));
        }
      }
      if constexpr (SPLIT) cluster_sync();   // the sums are read: no part leaves or writes again before
      else named_bar_sync(1, 32 * kWarps);
    }
  }
  __syncthreads();
}

// NT: token tiles of 8.  FL: steps of 32 k per scale group (8 = whole stage).
// SPLIT: a tile's k has several parts (apart, because the registers that this
// takes slow the other form: 72 against 64 us for 32 tokens through experts).
template <int NT, int FL, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 2) gemm_w4_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ W4Params p) {
  extern __shared__ unsigned char smem_raw[];
  constexpr int kStages = ring_stages(NT, FL);
  __shared__ __align__(8) uint64_t bars[2 * kStages];
  __shared__ uint32_t abort_word;
  W4Block k;
  k.ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  k.base = smem_raw + (k.ring - smem_u32(smem_raw));
  k.act_base = k.base + kStages * kStageBytes;
  k.acts = k.ring + kStages * kStageBytes;
  k.scales = reinterpret_cast<uint2*>(k.act_base + kStages * act_bytes(NT));
  k.red = reinterpret_cast<float*>(k.scales + kStages * (kSteps / FL) * kW4TileRows);
  int* list_lo = reinterpret_cast<int*>(k.red + 8 * NT * kRedPitch);
  uint16_t* list_id = reinterpret_cast<uint16_t*>(list_lo + p.E + 1);
  k.list_lo = list_lo;
  k.list_id = list_id;
  k.full = smem_u32(bars);
  k.empty = k.full + 8 * kStages;
  k.abort_flag = &abort_word;

  const int tid = threadIdx.x;
  const int split = SPLIT ? p.split : 1, part = (int)(blockIdx.x % split);
  k.tiles = (p.N + kW4TileRows - 1) / kW4TileRows;
  k.first = (int)(blockIdx.x / split);
  k.step = (int)(gridDim.x / split);
  k.kb0 = (int)((long long)part * p.num_kb / split);
  k.count_kb = (int)((long long)(part + 1) * p.num_kb / split) - k.kb0;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(k.full + 8 * s, 1 + kAuxThreads + kAuxThreads / 32);
      mbar_init(k.empty + 8 * s, kWarps);
    }
    fence_mbar_init();
    abort_word = 0;
    if (p.num_kb > 0) tma_prefetch_desc(&tm);
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  if (p.offsets) {
    k.active = list_experts(p, list_lo, list_id);
    // the rows past the last expert's
    const int V = min(max(p.offsets[p.E], 0), p.M);
    if (part == 0)
      for (int tile = k.first; tile < k.tiles; tile += k.step)
        for (long long i = tid; i < (long long)(p.M - V) * kW4TileRows; i += kThreads) {
          const long long m = V + i / kW4TileRows;
          const int n = tile * kW4TileRows + (int)(i % kW4TileRows);
          if (n >= p.N) continue;
          if (p.out_f32) static_cast<float*>(p.D)[m * p.ldd + n] = 0.0f;
          else static_cast<uint16_t*>(p.D)[m * p.ldd + n] = 0;
        }
  } else {
    k.active = (p.M + 8 * NT - 1) / (8 * NT);
  }
  k.items = k.tiles * k.active;

  if (tid >= 32 * kWarps) {
    if (p.s_f32) w4_copy<NT, FL, SPLIT, true>(&tm, p, k);
    else w4_copy<NT, FL, SPLIT, false>(&tm, p, k);
  } else {
    w4_multiply<NT, FL, SPLIT>(p, k, part);
  }
}

const void* kernel_for(int nt, int fl, bool split) {
  static const void* const table[2][4][2] = {
      {{(const void*)gemm_w4_kernel<1, 1, false>, (const void*)gemm_w4_kernel<1, 1, true>},
       {(const void*)gemm_w4_kernel<1, 2, false>, (const void*)gemm_w4_kernel<1, 2, true>},
       {(const void*)gemm_w4_kernel<1, 4, false>, (const void*)gemm_w4_kernel<1, 4, true>},
       {(const void*)gemm_w4_kernel<1, 8, false>, (const void*)gemm_w4_kernel<1, 8, true>}},
      {{(const void*)gemm_w4_kernel<2, 1, false>, (const void*)gemm_w4_kernel<2, 1, true>},
       {(const void*)gemm_w4_kernel<2, 2, false>, (const void*)gemm_w4_kernel<2, 2, true>},
       {(const void*)gemm_w4_kernel<2, 4, false>, (const void*)gemm_w4_kernel<2, 4, true>},
       {(const void*)gemm_w4_kernel<2, 8, false>, (const void*)gemm_w4_kernel<2, 8, true>}}};
  return table[nt - 1][fl == 1 ? 0 : fl == 2 ? 1 : fl == 4 ? 2 : 3][split];
}

}  // namespace

// The smallest number of parts for which the longest is shortest, as long as
// all of them run at once.  (1 token x 10157 x 7866, 80 tiles of 31 stages: three
// parts take 20.1 us, two 25.5.)
int w4_split(long long items, int num_kb, int sms) {
  int best = 1;
  for (int s = 2; s <= kMaxSplit && s <= num_kb && items * s <= kCtasPerSm * sms; ++s)
    if ((num_kb + s - 1) / s < (num_kb + best - 1) / best) best = s;
  return best;
}

cudaError_t launch_w4(const CUtensorMap& tm, W4Params p, int active, int sms, cudaStream_t stream, LaunchInfo* info) {
  const int fl = p.group >= kW4StageK ? kSteps : p.group / kStepK;
  // Two token tiles where one would stream the weights twice.
  const int nt = p.offsets ? (p.M > 4LL * active ? 2 : 1) : (p.M > 8 ? 2 : 1);
  const int smem = smem_for(nt, fl) + list_bytes(p.E);
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && !configured[dev]) {
    for (int i = 0; i < 16; ++i) {
      const int n = 1 + i / 8, f = 1 << (i / 2 % 4);
      if ((e = cudaFuncSetAttribute(kernel_for(n, f, i % 2), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    smem_for(n, f) + list_bytes(kExpertMax))))
        return e;
    }
    configured[dev] = true;
  }
  const long long tiles = (p.N + kW4TileRows - 1) / kW4TileRows;
  const long long items = tiles * (p.offsets ? active : (p.M + 8 * nt - 1) / (8 * nt));
  p.split = w4_split(items, p.num_kb, sms);
  const long long clusters = kCtasPerSm * sms / p.split;
  const int grid = (int)(items < clusters ? items : clusters) * p.split;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  *info = LaunchInfo{};
  info->grid = grid;
  info->cluster = p.split;
  info->block = kThreads;
  info->tile_m = kW4TileRows;
  info->tile_n = 8 * nt;
  info->stages = ring_stages(nt, fl);
  info->smem_bytes = smem;
  info->k_parts = p.split;
  info->kernel = p.offsets ? "gemm_w4_kernel<experts>" : "gemm_w4_kernel";
  void* args[2] = {const_cast<CUtensorMap*>(&tm), &p};
  return cudaLaunchKernelExC(&cfg, kernel_for(nt, fl, p.split > 1), args);
}

}  // namespace gtn
