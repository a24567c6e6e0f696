// Small device helpers shared by the CUDA kernels of this library.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <vector>

#include "../../include/mla_chunked_context.h"

namespace mla {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
  return __float2half_rn(x);
}

__device__ __forceinline__ bool is_neg_inf(float x) {
  return x == -__int_as_float(0x7f800000);
}

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }

// Smallest magnitude that rounds to infinity in fp16 (round to nearest even:
// the largest finite value is 65504, the midpoint to 2^16 is 65520).
constexpr float kF16Overflow = 65520.f;
template <typename T>
__host__ __device__ constexpr bool is_bf16() {
  return false;
}
template <>
__host__ __device__ constexpr bool is_bf16<__nv_bfloat16>() {
  return true;
}

// Index of the sequence that owns position `x`: the largest i in [0, n) with
// loc[i] <= x, for a non-decreasing loc[0..n].
__device__ __forceinline__ int find_seq(const int32_t *loc, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(loc + mid) <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// n / d for 0 <= n < 2^31 without a division, which takes some 200 clocks: with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (n + floor(m n
// / 2^32)) >> l (Granlund and Montgomery, Division by invariant integers using
// multiplication, 1994).
struct Divider {
  uint32_t mul = 0, shift = 0;
  explicit Divider(int32_t d) {
    while ((uint64_t(1) << shift) < uint64_t(d)) ++shift;
    mul = uint32_t((uint64_t(1) << 32) * ((uint64_t(1) << shift) - uint64_t(d)) / uint64_t(d) + 1);
  }
  __device__ __forceinline__ int quotient(int n) const {
    return int((__umulhi(mul, uint32_t(n)) + uint32_t(n)) >> shift);
  }
};

// Keys of a sequence of `len` tokens in a block table row of `stride` blocks of
// bs: the row ends them (and, far off, what 31 bits hold with room for a tile).
__device__ __forceinline__ int keys_of(int len, int stride, int bs) {
  const long long row = (long long)stride * bs, most = 0x7fff0000;
  return int(min((long long)len, row < most ? row : most));
}

// Which of its sequence's new tokens each new token sees, as bits: [T][words],
// new token j of the sequence in bit j % 64 of word j / 64.  Without bits the
// attention is causal or full.
struct TreeMask {
  const uint64_t *bits = nullptr;
  int words = 0;
};
__device__ __forceinline__ bool tree_bit(const uint64_t *row, int words, int j) {
  return (j >> 6) < words && (__ldg(row + (j >> 6)) >> (j & 63) & 1) != 0;
}
// 32 bits of a row from new token `from` on (in bit 0); tokens before the
// first (from < 0) are cached ones, which all see.
__device__ __forceinline__ uint32_t tree_bits(const uint64_t *row, int words, int from) {
  if (from <= -32) return ~0u;
  const int w = from >> 6, sh = from & 63;  // (from < 0: word -1, which is all ones)
  uint64_t v = w < 0 ? ~uint64_t(0) : w < words ? __ldg(row + w) : 0;
  v >>= sh;
  if (sh > 32 && w + 1 < words) v |= __ldg(row + w + 1) << (64 - sh);
  return uint32_t(v);
}

// Kernels this library has enqueued since it was loaded (every launcher
// calls launch_status() once, right after its launch).
inline std::atomic<unsigned long long> g_kernel_launches{0};

// Per-launch timing of one host thread, between mla_profile_begin() and
// mla_profile_end(): every launcher calls launch_begin(s) right before its
// launch and launch_status(s, name) right after it; while profiling is on
// these record a CUDA event on the launching stream on either side of the
// kernel, tagged with the step of the method the caller is in (ProfRole).
// Off (the default), launch_begin does nothing.  Events come from a pool
// that lives as long as the thread.
struct ProfRecord {
  const char *name, *role;
  cudaStream_t stream;
  cudaEvent_t start, stop;
};
struct ProfState {
  bool on = false;
  const char *role = "";
  cudaEvent_t pending = nullptr;  // start event of the launch being enqueued
  std::vector<ProfRecord> recs;
  std::vector<cudaEvent_t> pool;  // recorded-and-read events, for reuse
  cudaEvent_t take() {
    if (!pool.empty()) {
      cudaEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    cudaEvent_t e = nullptr;
    return cudaEventCreate(&e) == cudaSuccess ? e : nullptr;
  }
};
inline thread_local ProfState g_prof;

// Tags the launches enqueued while it lives with a step of the method.
struct ProfRole {
  const char *saved;
  explicit ProfRole(const char *role) : saved(g_prof.role) { g_prof.role = role; }
  ~ProfRole() { g_prof.role = saved; }
};

inline void launch_begin(cudaStream_t s) {
  if (!g_prof.on) return;
  cudaEvent_t e = g_prof.take();
  if (e && cudaEventRecord(e, s) == cudaSuccess) g_prof.pending = e;
}

inline int launch_status(cudaStream_t s, const char *name) {
  g_kernel_launches.fetch_add(1, std::memory_order_relaxed);
  const cudaError_t err = cudaGetLastError();
  if (g_prof.on && g_prof.pending) {
    cudaEvent_t e = g_prof.take();
    if (e && cudaEventRecord(e, s) == cudaSuccess)
      g_prof.recs.push_back({name, g_prof.role, s, g_prof.pending, e});
    g_prof.pending = nullptr;
  }
  return err == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

// Programmatic dependent launch, for the chains of short decode kernels: a
// kernel launched with launch_chained may start while the one before it on the
// stream is still running (once all of that one's blocks have called
// chain_release or exited), and calls chain_wait before it reads or writes any
// global memory: there it waits until the kernels before it have completed and
// their writes are visible.  (Before it the head products only ask for their
// weights in L2, where a write of the kernel before would find them.)  A kernel
// that allocates tensor memory calls chain_release (one call counts for its
// block) only once it has: else a block of a kernel behind it, resident beside
// it, could hold the columns that it still needs.
__device__ __forceinline__ void chain_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void chain_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... Params, typename... Args>
inline int launch_chained(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                          int cluster, cudaStream_t s, const char *name, Args &&...args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  launch_begin(s);
  if (cudaLaunchKernelEx(&cfg, kernel, Params(args)...) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return launch_status(s, name);
}

inline int elem_bytes(int32_t dtype) { return dtype == MLA_DTYPE_F32 ? 4 : 2; }

// storage types of the inputs and of the final output
inline bool valid_dtype(int32_t dtype) {
  return dtype == MLA_DTYPE_BF16 || dtype == MLA_DTYPE_F32;
}
// storage types of the up-projected K/V workspace
inline bool valid_kv_dtype(int32_t dtype) {
  return dtype == MLA_DTYPE_BF16 || dtype == MLA_DTYPE_F32 || dtype == MLA_DTYPE_F16;
}

// Scratch of the key-split attention: `slots` partials of [H][128][Dv] f32
// (O) and [H][128] f32 (LSE); a launch splits its longest (sequence, query
// tile) units over their keys until it has about `target_ctas` CTAs.
struct SplitScratch {
  float *o = nullptr, *lse = nullptr;
  int slots = 0, target_ctas = 0;
};

// The keys a context attention launch appends to each sequence's context
// keys: the sequence's own new tokens (rows q_loc[i] .. q_loc[i+1] of kv
// [T, H, 256] fp16 and latent [T, latent_ld] bf16, k_pe at column 512),
// attended causally.
struct NewKeySource {
  const void *kv = nullptr, *latent = nullptr;
  int64_t latent_ld = 0;
};

inline int num_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

}  // namespace mla
