// The norm of many gradient tensors, and clipping by it (sm_103a).
//
//   norm = sqrt(sum over all tensors and values of x^2)
//   clip: y = x * c,  c = max_norm / norm where norm > max_norm, else 1
//
// Memory bounds both: the norm reads every value once, a clip that has to
// scale reads it again and writes it once (between the two lies the sum of all
// of them).  So:
// - The tensors' addresses travel in the kernel's parameters (a list of 64, or
//   of 960 for longer ones), no table is copied to the GPU, and one launch
//   takes all of them: work is cut into chunks of 32 KB, and a block takes every
//   G-th chunk of the whole list, with the next one's loads in flight.
// - The clip's second pass runs through the chunks backwards: some 60 MB that
//   the first pass read last are still in L2 (132 MB of fp32 values into bf16: 48
//   us, forwards 57; 400 MB 151, 158).  Its stores are streaming, so that they do
//   not push them out.
// - Sums.  A thread adds 32 squares (16 of fp32 values) in fp32, in four chains
//   (an error of at most 11 steps of 2^-24), and these sums in fp64: one fp64 addition per 32
//   values is within what the SMs can do at the memory's rate, one per value
//   is not.  Where the fp32 sum overflowed, or is so small that squares may
//   have been lost, the values are squared again in fp64.  So the norm is
//   right over the whole range of values, and infinite or NaN only if a value is.
// - No atomics: a block's sum goes to its place in the workspace, and each
//   block that needs the total adds all places in the same order.
//
// Measured (graph-replayed): 1.07 GB of bf16 values 161 us, 0.98 of the copy
// bandwidth; 1.07 GB of fp32 values clipped into bf16 400 us for 2.68 GB, 0.99 of it;
// 16 small tensors of 4 MB 5.5 us, 40 of 6 MB clipped 9.2 us, each two launches
// that wait for one another.  In fp64, of which an SM does two operations a cycle, every
// step that all threads took together showed: a tree over 512 threads 2.5 us,
// a root and a quotient in each of them 4.5, squares of the zeros behind a
// tensor's end 3.6.

#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace gtn {

namespace {

constexpr int kThreads = 512;
constexpr int kBlocksPerSm = 2;
constexpr int kVectors = 4;              // 16-byte vectors per thread and chunk
constexpr int kChunkVectors = kThreads * kVectors;
constexpr int kSmallList = 64;

template <int CAP>
struct List {
  GradTensor t[CAP];
  int count;           // tensors in this launch
  int chunks;          // of all of them
};

struct Task {
  double* partial;     // sums of the blocks of this launch (squares), or of all launches (finish, clip)
  int partials;
  float max_norm;
  float* norm;         // finish, and the first block of a clip
};

// The values of a vector, 4 fp32 or 8 bf16.
template <bool F32>
__device__ __forceinline__ void unpack(uint4 a, float (&v)[F32 ? 4 : 8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ float load1(const void* base, bool f32, long long i) {
  return f32 ? static_cast<const float*>(base)[i]
             : __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[i] << 16);
}

__device__ __forceinline__ void store1(void* base, bool f32, long long i, float v) {
  if (f32) static_cast<float*>(base)[i] = v;
  else static_cast<uint16_t*>(base)[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
}

// The tensors' first chunks in shared memory, where a search does not wait for
// the parameters at every step.
template <int CAP>
__device__ __forceinline__ void copy_firsts(const List<CAP>& l, int* firsts) {
  for (int i = threadIdx.x; i < l.count; i += kThreads) firsts[i] = l.t[i].first;
  __syncthreads();
}

// The tensor of a chunk: the last whose first chunk is not past it, in [lo, hi].
__device__ __forceinline__ int tensor_of(const int* firsts, int chunk, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (firsts[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A chunk's place: its tensor, this thread's first vector and how many there are from it on.
struct Place {
  long long at;
  int left, tensor;
};

__device__ __forceinline__ long long vectors_of(const GradTensor& t) { return (t.count - t.head) * (t.in_f32 ? 4 : 2) / 16; }

template <int CAP>
__device__ __forceinline__ Place place_in(const List<CAP>& l, int chunk, int tensor) {
  Place r;
  const GradTensor& t = l.t[tensor];
  r.tensor = tensor;
  r.at = (long long)(chunk - t.first) * kChunkVectors + threadIdx.x;
  const long long left = vectors_of(t) - r.at;
  r.left = left < kChunkVectors ? (int)left : kChunkVectors;
  return r;
}

template <int CAP>
__device__ __forceinline__ void load_vectors(const List<CAP>& l, const Place& r, uint4 (&x)[kVectors]) {
  const GradTensor& t = l.t[r.tensor];
  const uint4* in = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(t.in) + t.head * (t.in_f32 ? 4 : 2)) + r.at;
#pragma unroll
  for (int u = 0; u < kVectors; ++u) x[u] = u * kThreads < r.left ? in[u * kThreads] : make_uint4(0, 0, 0, 0);
}

// The values of a tensor before its first vector and behind its last, one per
// thread of the first 16: calls f(index).
template <typename F>
__device__ __forceinline__ void for_ends(const GradTensor& t, F f) {
  if (threadIdx.x < 16) {
    const long long i =
        threadIdx.x < 8 ? threadIdx.x : t.head + vectors_of(t) * (t.in_f32 ? 4 : 8) + (threadIdx.x - 8);
    if (threadIdx.x < 8 ? i < t.head : i < t.count) f(i);
  }
}

// The sum over the block, in every thread; the order is fixed.  One warp adds
// what all threads put down: an SM does two fp64 additions a cycle, and a tree
// over all threads with a last step in each of them took 5000 cycles.
struct Sums {
  double of_thread[kThreads];
  double all;
};

__device__ __forceinline__ double block_sum(double v, Sums& shared) {
  __syncthreads();
  shared.of_thread[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    double a[4] = {};
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) a[i & 3] += shared.of_thread[i * 32 + threadIdx.x];
    double s = (a[0] + a[1]) + (a[2] + a[3]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (threadIdx.x == 0) shared.all = s;
  }
  __syncthreads();
  return shared.all;
}

// The squares of vectors in fp64, for fp32 sums that hold too little or too much.
template <bool F32>
__device__ __noinline__ double squares64(uint4 a, uint4 b, uint4 c, uint4 d) {
  double s = 0.0;
#pragma unroll 1
  for (int u = 0; u < kVectors; ++u) {
    const uint4 x = u == 0 ? a : u == 1 ? b : u == 2 ? c : d;
    float v[F32 ? 4 : 8];
    unpack<F32>(x, v);
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 8); ++i) s += (double)v[i] * (double)v[i];
  }
  return s;
}

template <bool F32>
__device__ __forceinline__ double squares(const uint4 (&x)[kVectors]) {
  float s[kVectors] = {};
#pragma unroll
  for (int u = 0; u < kVectors; ++u) {
    float v[F32 ? 4 : 8];
    unpack<F32>(x[u], v);
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 8); ++i) s[u] = fmaf(v[i], v[i], s[u]);
  }
  const float all = (s[0] + s[1]) + (s[2] + s[3]);
  // Squares below 2^-126 lose bits, or all: with a sum above 2^-80 what is
  // lost is below 2^-41 of it.
  if (all >= 0x1p-80f && all <= 0x1p127f) return (double)all;
  uint32_t any = 0;      // zeros (also those behind a tensor's end) take no fp64 work
#pragma unroll
  for (int u = 0; u < kVectors; ++u) any |= x[u].x | x[u].y | x[u].z | x[u].w;
  if ((any & (F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0) return 0.0;
  return squares64<F32>(x[0], x[1], x[2], x[3]);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_squares_kernel(const __grid_constant__ List<CAP> l, const Task k) {
  __shared__ Sums shared;
  __shared__ int firsts[CAP];
  copy_firsts(l, firsts);
  griddep_wait();
  griddep_launch_dependents();
  double sum = 0.0;
  int chunk = blockIdx.x;
  Place r = place_in(l, chunk, tensor_of(firsts, chunk, 0, l.count - 1));
  uint4 x[kVectors];
  load_vectors(l, r, x);
  while (true) {
    // the next chunk's vectors are on their way while these are summed
    const int next = chunk + gridDim.x;
    const bool more = next < l.chunks;
    Place rn = r;
    uint4 y[kVectors];
    if (more) {
      const bool same = r.tensor + 1 == l.count || firsts[r.tensor + 1] > next;
      rn = place_in(l, next, same ? r.tensor : tensor_of(firsts, next, r.tensor + 1, l.count - 1));
      load_vectors(l, rn, y);
    }
    const GradTensor& t = l.t[r.tensor];
    sum += t.in_f32 ? squares<true>(x) : squares<false>(x);
    if (chunk == t.first)
      for_ends(t, [&](long long i) {
        const double v = load1(t.in, t.in_f32, i);
        sum += v * v;
      });
    if (!more) break;
    chunk = next;
    r = rn;
#pragma unroll
    for (int u = 0; u < kVectors; ++u) x[u] = y[u];
  }
  sum = block_sum(sum, shared);
  if (threadIdx.x == 0) k.partial[blockIdx.x] = sum;
}

// The sum of all squares, in every thread.
__device__ __forceinline__ double total(const Task& k, Sums& shared) {
  double s = 0.0;
  for (int i = threadIdx.x; i < k.partials; i += kThreads) s += k.partial[i];
  return block_sum(s, shared);
}

// A vector's values times both factors, `at` vectors behind `out`; `valid`: the
// vector is there.  All lanes of a warp call it: bf16 to fp32, a vector becomes
// 32 bytes, which one lane would store in halves of sectors (210 million values
// clipped: 1017 us), so a pair of lanes stores first the even lane's, then the
// odd lane's (273 us).
template <bool F32>
__device__ __forceinline__ void store_scaled(uint8_t* out, int at, bool valid, uint4 x, float first, float c, bool out_f32) {
  constexpr int kPer = F32 ? 4 : 8;
  float v[kPer];
  unpack<F32>(x, v);
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = v[i] * first * c;
  if constexpr (F32) {
    if (!valid) return;
    if (out_f32) __stcs(reinterpret_cast<float4*>(out) + at, make_float4(v[0], v[1], v[2], v[3]));
    else __stcs(reinterpret_cast<uint2*>(out) + at, make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])));
  } else if (!out_f32) {
    if (valid)
      __stcs(reinterpret_cast<uint4*>(out) + at, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
  } else {
    const int odd = threadIdx.x & 1;
    // the other lane's half of its own vector that this lane stores, into the half it does not need
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[4 + i], 1);
      if (odd) v[i] = got;
      else v[4 + i] = got;
    }
    const bool other = __shfl_xor_sync(0xffffffffu, (int)valid, 1);
    float4* to = reinterpret_cast<float4*>(out) + at * 2 - odd;
    if (odd ? other : valid) __stcs(to, make_float4(v[0], v[1], v[2], v[3]));              // the even lane's vector
    if (odd ? valid : other) __stcs(to + 2, make_float4(v[4], v[5], v[6], v[7]));          // the odd lane's
  }
}

__global__ void __launch_bounds__(kThreads) grad_finish_kernel(const Task k) {
  __shared__ Sums shared;
  griddep_wait();
  griddep_launch_dependents();
  const double sum = total(k, shared);
  if (threadIdx.x == 0) *k.norm = (float)sqrt(sum);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grad_clip_kernel(const __grid_constant__ List<CAP> l, const Task k, bool in_place) {
  __shared__ Sums shared;
  __shared__ int firsts[CAP];
  copy_firsts(l, firsts);
  griddep_wait();
  griddep_launch_dependents();
  const double sum = total(k, shared);
  // One thread takes the root and the quotient: in fp64, all threads' would
  // take 4 us.  Two factors, the first a power of two: a single one below 2^-126
  // (a norm beyond fp32) would lose bits.  A norm that is not finite leaves the
  // values alone.
  __shared__ float factors[2];
  __shared__ int scaled;
  if (threadIdx.x == 0) {
    const double norm = sqrt(sum);
    if (k.norm && blockIdx.x == 0) *k.norm = (float)norm;
    scaled = norm > (double)k.max_norm && norm <= 1.7976931348623157e308;
    const double exact = scaled ? (double)k.max_norm / norm : 1.0;
    const bool tiny = exact < 0x1p-100;
    factors[0] = tiny ? 0x1p-64f : 1.0f;
    factors[1] = (float)(tiny ? exact * 0x1p64 : exact);
  }
  __syncthreads();
  if (!scaled && in_place) return;
  const float first = factors[0], c = factors[1];
  // backwards through the chunks, the next one's vectors on their way while these are scaled
  int chunk = l.chunks - 1 - (int)blockIdx.x;
  Place r = place_in(l, chunk, tensor_of(firsts, chunk, 0, l.count - 1));
  uint4 x[kVectors];
  if (l.t[r.tensor].vector) load_vectors(l, r, x);
  while (true) {
    const int next = chunk - (int)gridDim.x;
    Place rn = r;
    uint4 y[kVectors];
    if (next >= 0) {
      rn = place_in(l, next, firsts[r.tensor] <= next ? r.tensor : tensor_of(firsts, next, 0, r.tensor - 1));
      if (l.t[rn.tensor].vector) load_vectors(l, rn, y);
    }
    const GradTensor& t = l.t[r.tensor];
    const bool in_f32 = t.in_f32, out_f32 = t.out_f32;
    if (t.vector) {
      const int per = in_f32 ? 4 : 8;
      uint8_t* out = static_cast<uint8_t*>(t.out) + (t.head + r.at * per) * (out_f32 ? 4 : 2);
#pragma unroll
      for (int u = 0; u < kVectors; ++u) {
        if (in_f32) store_scaled<true>(out, u * kThreads, u * kThreads < r.left, x[u], first, c, out_f32);
        else store_scaled<false>(out, u * kThreads, u * kThreads < r.left, x[u], first, c, out_f32);
      }
    } else {
      // out does not lie as in does: value by value, neighbours by neighbouring threads
      const int per = in_f32 ? 4 : 8;
      const long long begin = t.head + (r.at - threadIdx.x) * per;
      const long long end = min(begin + (long long)kChunkVectors * per, t.head + vectors_of(t) * per);
      for (long long j = begin + threadIdx.x; j < end; j += kThreads)
        store1(t.out, out_f32, j, load1(t.in, in_f32, j) * first * c);
    }
    if (chunk == t.first)
      for_ends(t, [&](long long j) { store1(t.out, out_f32, j, load1(t.in, in_f32, j) * first * c); });
    if (next < 0) break;
    chunk = next;
    r = rn;
#pragma unroll
    for (int u = 0; u < kVectors; ++u) x[u] = y[u];
  }
}

int blocks_for(int chunks, int sms) {
  const int most = kBlocksPerSm * sms < kGradMaxBlocks ? kBlocksPerSm * sms : kGradMaxBlocks;
  return chunks < most ? chunks : most;
}

template <typename... Args>
cudaError_t launch(const void* kernel, int grid, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* pointers[] = {const_cast<void*>(static_cast<const void*>(args))...};
  return cudaLaunchKernelExC(&cfg, kernel, pointers);
}

// One pass of a kernel over `count` tensors, kGradMaxTensors per launch.
// `first_partial` gets each launch's place in the workspace.
template <typename Fill>
cudaError_t passes(const GradTensor* tensors, int count, bool clip, bool in_place, int sms, cudaStream_t stream, Fill fill,
                   LaunchInfo* info) {
  static thread_local List<kGradMaxTensors> list;
  for (int at = 0; at < count; at += kGradMaxTensors) {
    const int n = count - at < kGradMaxTensors ? count - at : kGradMaxTensors;
    long long chunks = 0;
    for (int i = 0; i < n; ++i) {
      GradTensor& t = list.t[i];
      t = tensors[at + i];
      t.first = (int)chunks;
      const long long vectors = (t.count - t.head) * (t.in_f32 ? 4 : 2) / 16;
      chunks += vectors > 0 ? (vectors + kChunkVectors - 1) / kChunkVectors : 1;
      if (chunks >= (1ll << 31) - 4096) return cudaErrorInvalidValue;
    }
    list.count = n;
    list.chunks = (int)chunks;
    const int grid = blocks_for((int)chunks, sms);
    Task task = fill(at / kGradMaxTensors, grid);
    cudaError_t e;
    if (n <= kSmallList) {
      static thread_local List<kSmallList> small;
      for (int i = 0; i < n; ++i) small.t[i] = list.t[i];
      small.count = n;
      small.chunks = list.chunks;
      e = clip ? launch((const void*)grad_clip_kernel<kSmallList>, grid, stream, &small, &task, &in_place)
               : launch((const void*)grad_squares_kernel<kSmallList>, grid, stream, &small, &task);
    } else {
      e = clip ? launch((const void*)grad_clip_kernel<kGradMaxTensors>, grid, stream, &list, &task, &in_place)
               : launch((const void*)grad_squares_kernel<kGradMaxTensors>, grid, stream, &list, &task);
    }
    if (e != cudaSuccess) return e;
    info->grid = grid;
  }
  return cudaSuccess;
}

}  // namespace

long long grad_partials(int count) {
  return (long long)kGradMaxBlocks * ((count + kGradMaxTensors - 1) / kGradMaxTensors);
}

cudaError_t launch_grad_norm(const GradTensor* tensors, int count, bool clip, bool in_place, float max_norm, float* norm,
                             double* workspace, int sms, cudaStream_t stream, LaunchInfo* info) {
  *info = LaunchInfo{};
  info->cluster = 1;
  info->block = kThreads;
  info->kernel = clip ? "grad_clip_kernel" : "grad_squares_kernel";
  // the launches' sums, one behind the other without gaps
  int used = 0;
  cudaError_t e = passes(tensors, count, false, false, sms, stream, [&](int, int grid) {
    Task t = {workspace + used, 0, 0.0f, nullptr};
    used += grid;
    return t;
  }, info);
  if (e != cudaSuccess) return e;
  if (!clip || count == 0) {
    Task t = {workspace, used, 0.0f, norm};
    return launch((const void*)grad_finish_kernel, 1, stream, &t);
  }
  return passes(tensors, count, true, in_place, sms, stream, [&](int launch_index, int) {
    return Task{workspace, used, max_norm, launch_index == 0 ? norm : nullptr};
  }, info);
}

}  // namespace gtn
