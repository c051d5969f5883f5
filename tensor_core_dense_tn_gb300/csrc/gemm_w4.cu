// Products with 4-bit weights for few tokens (gemm_w4_tn, gemm_w4_tn_experts):
//
//   D[m, n] = act(alpha * sum_g s[n, g] * sum_{k in g} A[m, k] (q[n, k] - z[n, g]))
//
// Bound by the read of the codes (half a byte per weight) and the scales.
// The differences q - z are whole numbers below 256 in magnitude, so they are
// exact in bf16: a group's products run on the tensor cores (fp32 sums) with
// no rounding of the weights, and the scale multiplies the group's fp32 sum.
//
// A CTA holds 128 rows of the weights and a part of K; the parts of a tile
// are the CTAs of a cluster, which add their fp32 sums through distributed
// shared memory in part order (no workspace, no atomics).  One warp streams
// the codes by TMA (128 x 128-byte boxes, 16 KiB) through an mbarrier ring;
// eight warps of 16 rows each turn them into mma fragments.
//
// Fragments.  mma.m16n8k16 sums over k, so k may be permuted as long as both
// operands agree.  A lane (row r = lane / 4, q = lane % 4) reads the word that
// holds k = 8 q .. 8 q + 7 of its row in a block of 32; masking the word
// shifted by 4 i leaves the nibbles i and i + 4 as the two halves of a
// register, 0x4300 | nibble is the bf16 value 128 + nibble, and one packed
// subtraction of 128 + z gives the exact difference.  The activations are
// staged in the same order (0, 4, 1, 5, 2, 6, 3, 7) per block of 8.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace gtn {
namespace {

constexpr int kMmaWarps = 8;
constexpr int kThreads = 32 * (kMmaWarps + 1);
constexpr int kStageBytes = kW4TileRows * 128;
constexpr int kStepK = 32;                          // k per step: two mma
constexpr int kSteps = kW4StageK / kStepK;          // steps per stage
constexpr int kErrTimeout = -5;
constexpr int kMaxStages = 6;

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

// Nibbles i and i + 4 of `word` as bf16 differences from the zero point:
// (128 + q) - (128 + z), both exact.
__device__ __forceinline__ uint32_t nibbles(uint32_t word, int i, uint32_t magic_z) {
  const uint32_t v = ((word >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  __nv_bfloat162 a, z;
  memcpy(&a, &v, 4);
  memcpy(&z, &magic_z, 4);
  a = __hsub2(a, z);
  uint32_t r;
  memcpy(&r, &a, 4);
  return r;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Sum of one token's column: [token][row], padded so that a warp's fragment
// stores (8 rows x 4 token pairs) fall in different banks.
constexpr int kRedPitch = kW4TileRows + 4;

__host__ __device__ constexpr int act_bytes(int nt, int slab) { return slab * kW4StageK * 8 * nt * 2; }
__host__ __device__ constexpr int scale_bytes(int slab, int per_stage) { return slab * per_stage * kW4TileRows * 8; }
__host__ __device__ constexpr int red_bytes(int nt) { return 8 * nt * kRedPitch * 4; }

// NT: token tiles of 8.  FL: steps of 32 k per scale group (8 = whole stage).
template <int NT, int FL>
__global__ void __launch_bounds__(kThreads, 2) gemm_w4_kernel(const __grid_constant__ CUtensorMap tm, W4Params p) {
  extern __shared__ unsigned char smem_raw[];
  constexpr int kTok = 8 * NT, kFlushes = kSteps / FL;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* base = smem_raw + (ring - smem_u32(smem_raw));
  unsigned char* acts = base + p.stages * kStageBytes;
  uint2* scales = reinterpret_cast<uint2*>(acts + act_bytes(NT, p.slab));   // [stage][flush][row]: scale, 128 + z twice
  float* red = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(scales) + scale_bytes(p.slab, kFlushes));
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages];
  __shared__ uint32_t abort_word;
  __shared__ int found[2];
  __shared__ int warp_count[kMmaWarps + 1];
  volatile uint32_t* abort_flag = &abort_word;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = (int)(blockIdx.x % p.split);
  const int n0 = (int)(blockIdx.x / p.split) * kW4TileRows;
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  auto empty = [&](int s) { return smem_u32(&bars[kMaxStages + s]); };
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kMmaWarps);
    }
    fence_mbar_init();
    abort_word = 0;
    found[0] = found[1] = 0;
    if (p.num_kb > 0) tma_prefetch_desc(&tm);
  }
  griddep_wait();
  griddep_launch_dependents();

  // Rows [lo, hi) of this block: the blockIdx.y-th matrix that has rows, or
  // the dense form's blockIdx.y-th block of tokens.
  int expert = 0, lo, hi;
  __syncthreads();
  if (p.offsets) {
    int before = 0;
    lo = hi = 0;
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
      for (int w = 0; w <= kMmaWarps; ++w) {
        if (w < warp) at += warp_count[w];
        before += warp_count[w];
      }
      if (b > a && at + __popc(some & ((1u << lane) - 1)) == (int)blockIdx.y) {
        found[0] = e + 1;
        found[1] = a;
      }
      __syncthreads();
    }
    expert = found[0] - 1;
    // rows after the last expert's are zeroed by the first row of blocks
    if (blockIdx.y == 0 && part == 0) {
      const int V = min(max(p.offsets[p.E], 0), p.M);
      for (long long i = (long long)tid; i < (long long)(p.M - V) * kW4TileRows; i += kThreads) {
        const long long m = V + i / kW4TileRows;
        const int n = n0 + (int)(i % kW4TileRows);
        if (n >= p.N) continue;
        if (p.out_f32) static_cast<float*>(p.D)[m * p.ldd + n] = 0.0f;
        else static_cast<uint16_t*>(p.D)[m * p.ldd + n] = 0;
      }
    }
    if (expert < 0) return;   // the same for the whole cluster
    lo = found[1];
    hi = min(max(p.offsets[expert + 1], lo), p.M);
  } else {
    lo = (int)blockIdx.y * kTok;
    hi = min(p.M, lo + kTok);
  }

  const int kb0 = (int)((long long)part * p.num_kb / p.split), kb1 = (int)((long long)(part + 1) * p.num_kb / p.split);
  const int blocks = (hi - lo + kTok - 1) / kTok;   // token blocks: the weights are streamed once for each

  const uint16_t* A = static_cast<const uint16_t*>(p.A);
  const int row = lane >> 2, q = lane & 3;
  int stage = 0, phase = 0, issued = 0;
  bool ok = true;
  for (int tb = 0; tb < blocks; ++tb) {
    const int m0 = lo + tb * kTok, count = min(kTok, hi - m0);
    if (warp == kMmaWarps) {
      if (lane == 0)
        for (int kb = kb0; kb < kb1 && ok; ++kb) {
          ok = wait_bar(empty(stage), phase ^ 1, abort_flag, p.timeout_ns, p.status, kRoleProducer);
          if (!ok) break;
          mbar_arrive_expect_tx(full(stage), kStageBytes);
          tma_load_3d(ring + stage * kStageBytes, &tm, kb * 128, n0, expert, full(stage));
          ++issued;
          if (++stage == p.stages) { stage = 0; phase ^= 1; }
        }
      __syncwarp();
    }
    float tot[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[t][i] = 0.0f;

    for (int s0 = kb0; s0 < kb1 && warp < kMmaWarps; s0 += p.slab) {
      const int s1 = min(kb1, s0 + p.slab);
      if (s0 > kb0) named_bar_sync(1, 32 * kMmaWarps);   // the last slab's readers are done
      {
        // activations: 16 bytes (8 k) per thread and turn, k permuted for the fragments
        const int chunks = (s1 - s0) * (kW4StageK / 8) * kTok;
        for (int i = tid; i < chunks; i += 32 * kMmaWarps) {
          const int cq = i & 3, tok8 = (i >> 2) & 7, rest = i >> 5;   // lane order of the fragment
          const int t = rest % NT, k32 = rest / NT, m = t * 8 + tok8;
          if (m >= count) continue;
          const int k = s0 * kW4StageK + k32 * kStepK + cq * 8;
          long long r = m0 + m;
          if (p.a_rows) r = p.a_rows[r];
          uint32_t w[4] = {0, 0, 0, 0};
          if (r >= 0 && r < p.a_count) {
            const uint16_t* src = A + r * p.lda + k;
            if (k + 8 <= p.K) {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (k + j < p.K) w[j / 2] |= (uint32_t)src[j] << (16 * (j & 1));
            }
          }
          uint4 o;   // (0,4) (1,5) (2,6) (3,7)
          o.x = __byte_perm(w[0], w[2], 0x5410);
          o.y = __byte_perm(w[0], w[2], 0x7632);
          o.z = __byte_perm(w[1], w[3], 0x5410);
          o.w = __byte_perm(w[1], w[3], 0x7632);
          *reinterpret_cast<uint4*>(acts + ((k32 * NT + t) * 32 + tok8 * 4 + cq) * 16) = o;
        }
        // scales and zero points
        const int entries = (s1 - s0) * kFlushes * kW4TileRows;
        for (int i = tid; i < entries; i += 32 * kMmaWarps) {
          const int rr = i % kW4TileRows, f = i / kW4TileRows;
          const int n = n0 + rr;
          const long long g = ((long long)s0 * kW4StageK + (long long)f * FL * kStepK) / p.group;
          float sc = 0.0f;
          uint32_t z = 8;
          if (n < p.N && g < p.ngroups) {
            const long long at = expert * p.stride_s + n * p.ld_s + g;
            sc = p.s_f32 ? static_cast<const float*>(p.scales)[at]
                         : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.scales)[at] << 16);
            if (p.zeros) z = p.zeros[expert * p.stride_z + n * p.ld_z + g];
          }
          // 128 + z in bf16: exact for z up to 127, the low seven bits
          scales[i] = make_uint2(__float_as_uint(sc), (0x4300u + (z & 0x7Fu)) * 0x00010001u);
        }
      }
      named_bar_sync(1, 32 * kMmaWarps);
      {
        for (int kb = s0; kb < s1 && ok; ++kb) {
          // one answer per warp: its lanes leave together
          ok = __all_sync(0xFFFFFFFFu, wait_bar(full(stage), phase, abort_flag, p.timeout_ns, p.status, kRoleMma));
          if (!ok) break;
          const unsigned char* codes = base + stage * kStageBytes;
          const int ra = warp * 16 + row, rb = ra + 8;
          const uint2* sc = scales + (kb - s0) * kFlushes * kW4TileRows;
          const unsigned char* act = acts + (kb - s0) * kSteps * NT * 512 + lane * 16;
#pragma unroll
          for (int f = 0; f < kFlushes; ++f) {
            const uint2 sa = sc[f * kW4TileRows + ra], sb = sc[f * kW4TileRows + rb];
            float acc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
#pragma unroll
            for (int h = 0; h < FL; ++h) {
              const int step = f * FL + h;
              // 128-byte swizzle: 16-byte column c of row r sits at c ^ (r % 8)
              const int col = ((step ^ row) << 4) | (q << 2);
              const uint32_t wa = *reinterpret_cast<const uint32_t*>(codes + ra * 128 + col);
              const uint32_t wb = *reinterpret_cast<const uint32_t*>(codes + rb * 128 + col);
              uint32_t lo4[4], hi4[4];
              lo4[0] = nibbles(wa, 0, sa.y); lo4[1] = nibbles(wb, 0, sb.y);
              lo4[2] = nibbles(wa, 1, sa.y); lo4[3] = nibbles(wb, 1, sb.y);
              hi4[0] = nibbles(wa, 2, sa.y); hi4[1] = nibbles(wb, 2, sb.y);
              hi4[2] = nibbles(wa, 3, sa.y); hi4[3] = nibbles(wb, 3, sb.y);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                uint4 b = make_uint4(0, 0, 0, 0);
                if (t * 8 + row < count) b = *reinterpret_cast<const uint4*>(act + (step * NT + t) * 512);
                mma_16816(acc[t], lo4, b.x, b.y);
                mma_16816(acc[t], hi4, b.z, b.w);
              }
            }
            const float fa = __uint_as_float(sa.x), fb = __uint_as_float(sb.x);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              tot[t][0] = fmaf(fa, acc[t][0], tot[t][0]);
              tot[t][1] = fmaf(fa, acc[t][1], tot[t][1]);
              tot[t][2] = fmaf(fb, acc[t][2], tot[t][2]);
              tot[t][3] = fmaf(fb, acc[t][3], tot[t][3]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty(stage));
          if (++stage == p.stages) { stage = 0; phase ^= 1; }
        }
      }
    }

    // The parts' sums meet in shared memory; part j finishes rows
    // [128 j / split, 128 (j + 1) / split), adding the parts in order.
    if (warp < kMmaWarps) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[(t * 8 + 2 * q + (i & 1)) * kRedPitch + warp * 16 + row + 8 * (i >> 1)] = tot[t][i];
    }
    if (p.split > 1) cluster_sync();
    else __syncthreads();
    const int rows = kW4TileRows / p.split;
    for (int i = tid; i < count * rows; i += kThreads) {
      const int m = i / rows, rr = part * rows + i % rows, n = n0 + rr;
      const uint32_t at = smem_u32(red + m * kRedPitch + rr);
      float v = 0.0f;
      if (p.split > 1) {
        for (int j = 0; j < p.split; ++j) v += ld_cluster_f32(mapa_shared(at, j));
      } else {
        v = red[m * kRedPitch + rr];
      }
      if (n < p.N) {
        v = activate(p.alpha * v, p.act);
        const long long d = (m0 + m) * p.ldd + n;
        if (p.out_f32) static_cast<float*>(p.D)[d] = v;
        else static_cast<uint16_t*>(p.D)[d] = (uint16_t)pack_bf16x2(v, 0.0f);
      }
    }
    if (p.split > 1) cluster_sync();   // no part leaves or writes again while another reads its sums
    else __syncthreads();
  }

  // After a wait that gave up, the copies still in flight land (bounded)
  // before the shared memory is given back.
  if (warp == kMmaWarps && lane == 0 && *abort_flag) {
    const uint64_t t0 = globaltimer();
    for (int i = 0; i < min(issued, p.stages); ++i) {
      const int at = issued - 1 - i, s = at % p.stages, ph = (at / p.stages) & 1;
      while (!mbar_try_wait(full(s), ph) && globaltimer() - t0 < p.timeout_ns) {
      }
    }
  }
}

int smem_for(int nt, int fl, int stages, int slab) {
  return 1024 + stages * kStageBytes + act_bytes(nt, slab) + scale_bytes(slab, kSteps / fl) + red_bytes(nt);
}

template <int NT>
const void* kernel_for(int fl) {
  return fl == 1 ? (const void*)gemm_w4_kernel<NT, 1> : fl == 2 ? (const void*)gemm_w4_kernel<NT, 2>
         : fl == 4 ? (const void*)gemm_w4_kernel<NT, 4> : (const void*)gemm_w4_kernel<NT, 8>;
}

}  // namespace

int w4_split(long long tiles, int num_kb, int sms) {
  int s = 1;
  while (s < 8 && s * 2 <= num_kb && tiles * s * 2 <= 4 * sms) s *= 2;
  return s;
}

cudaError_t launch_w4(const CUtensorMap& tm, W4Params p, int active, cudaStream_t stream, LaunchInfo* info) {
  const int fl = p.group >= kW4StageK ? kSteps : p.group / kStepK;
  // Two token tiles where one would stream the weights twice.
  const int nt = p.offsets ? (p.M > 4LL * active ? 2 : 1) : (p.M > 8 ? 2 : 1);
  const int kb_part = (p.num_kb + p.split - 1) / p.split;
  p.stages = 4;
  p.slab = kb_part < 1 ? 1 : kb_part;
  const int budget = 112 * 1024;    // two CTAs per SM
  while (p.slab > 1 && smem_for(nt, fl, p.stages, p.slab) > budget) --p.slab;
  const int smem = smem_for(nt, fl, p.stages, p.slab);
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && !configured[dev]) {
    for (int f = 1; f <= kSteps; f *= 2) {
      if ((e = cudaFuncSetAttribute(kernel_for<1>(f), cudaFuncAttributeMaxDynamicSharedMemorySize, budget))) return e;
      if ((e = cudaFuncSetAttribute(kernel_for<2>(f), cudaFuncAttributeMaxDynamicSharedMemorySize, budget))) return e;
    }
    configured[dev] = true;
  }
  const int tiles = (p.N + kW4TileRows - 1) / kW4TileRows;
  const int gy = p.offsets ? active : (p.M + 8 * nt - 1) / (8 * nt);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(tiles * p.split, gy);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  *info = LaunchInfo{};
  info->grid = tiles * p.split * gy;
  info->cluster = p.split;
  info->block = kThreads;
  info->tile_m = kW4TileRows;
  info->tile_n = 8 * nt;
  info->stages = p.stages;
  info->smem_bytes = smem;
  info->k_parts = p.split;
  info->kernel = p.offsets ? "gemm_w4_kernel<experts>" : "gemm_w4_kernel";
  void* args[2] = {const_cast<CUtensorMap*>(&tm), &p};
  return cudaLaunchKernelExC(&cfg, nt == 2 ? kernel_for<2>(fl) : kernel_for<1>(fl), args);
}

}  // namespace gtn
