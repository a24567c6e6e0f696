// Writing new tokens into the paged latent cache (mla_append_latent): RMS
// norm of the latent part, rotation of the rope part, both stored to the
// token's cache slot and (optionally) as a dense row, and the rotation of the
// queries' rope columns, in one launch.
//
//   row[0:L)   = x / sqrt(mean(x^2) + eps) * w
//   row[L:L+P) = (a cos - b sin, b cos + a sin) per rotated pair (a, b)
//
// Every value is read once and written once (the row twice, when the dense
// copy is asked for), so the kernel is bound by HBM when there are many
// tokens and by the chain of dependent loads (sequence, length, block id)
// when there are few.  A block serves one token: warp 0 of its first block
// the row, all other warps the heads of the queries, 32 lanes over 16-byte
// pieces.  Few tokens spread their heads over several blocks.
#include "common.cuh"

namespace mla {
namespace {

constexpr int WARPS = 8;

struct AppendArgs {
  const void *kv_a, *norm_weight, *q;
  void *kv_cache, *new_latent, *q_pe;
  const int32_t *qsl, *seq_lens, *positions, *block_table;
  const float *rope;
  int32_t *status;
  int64_t kv_a_ld, q_pe_ld;
  int T, R, H, L, P, Dn, bs, num_blocks, bt_stride, max_pos, interleaved;
  float eps;
  int vec_row, vec_q;  // rows / queries move as 16-byte pieces
};

// Largest r in [0, n) with loc[r] <= x, by the whole warp: each round narrows
// the range 32-fold with one load per lane (two dependent loads for 1024
// sequences, where a binary search has ten).
__device__ __forceinline__ int find_seq_warp(const int32_t *loc, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < len && __ldg(loc + i) <= x;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;  // loc is non-decreasing: the last lane that holds
    lo += k * step;
    len = min(step, len - k * step);
  }
  return lo;
}

// 16 bytes of T as floats
template <typename T>
struct Piece {
  static constexpr int N = 16 / sizeof(T);
  float v[N];
  __device__ __forceinline__ void load(const T *p) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32(e[i]);
  }
  __device__ __forceinline__ void store(T *p) const {
    uint4 u;
    T *e = reinterpret_cast<T *>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<uint4 *>(p) = u;
  }
};

// Rotates pair number `pair` of the P rope columns at `src`; the results go to
// the same columns of up to two destinations.
template <typename T>
__device__ __forceinline__ void rotate_pair(const T *src, T *d0, T *d1, const float *rope, int P,
                                            int pair, bool interleaved) {
  const int half = P / 2;
  const int i = interleaved ? 2 * pair : pair, j = interleaved ? 2 * pair + 1 : pair + half;
  const float a = to_f32(src[i]), b = to_f32(src[j]);
  const float c = __ldg(rope + pair), s = __ldg(rope + half + pair);
  const T x = from_f32<T>(a * c - b * s), y = from_f32<T>(b * c + a * s);
  if (d0) {
    d0[i] = x;
    d0[j] = y;
  }
  if (d1) {
    d1[i] = x;
    d1[j] = y;
  }
}

// The same for the 16-byte pieces of piece number `k`: interleaved, one piece
// holds N/2 pairs; half-split, piece k goes with piece k + P/(2N).
template <typename T>
__device__ __forceinline__ void rotate_piece(const T *src, T *d0, T *d1, const float *rope, int P,
                                             int k, bool interleaved) {
  constexpr int N = Piece<T>::N;
  const int half = P / 2;
  if (interleaved) {
    Piece<T> x;
    x.load(src + k * N);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const float c = __ldg(rope + k * (N / 2) + e), s = __ldg(rope + half + k * (N / 2) + e);
      const float a = x.v[2 * e], b = x.v[2 * e + 1];
      x.v[2 * e] = a * c - b * s;
      x.v[2 * e + 1] = b * c + a * s;
    }
    if (d0) x.store(d0 + k * N);
    if (d1) x.store(d1 + k * N);
  } else {
    Piece<T> x, y;
    x.load(src + k * N);
    y.load(src + half + k * N);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float c = __ldg(rope + k * N + e), s = __ldg(rope + half + k * N + e);
      const float a = x.v[e], b = y.v[e];
      x.v[e] = a * c - b * s;
      y.v[e] = b * c + a * s;
    }
    if (d0) {
      x.store(d0 + k * N);
      y.store(d0 + half + k * N);
    }
    if (d1) {
      x.store(d1 + k * N);
      y.store(d1 + half + k * N);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * WARPS) append_kernel(AppendArgs a) {
  constexpr int N = Piece<T>::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x;
  // the token's sequence and position
  const int first = max(__ldg(a.qsl), 0);
  if (t < first || t >= min(__ldg(a.qsl + a.R), a.T)) return;
  const int r = find_seq_warp(a.qsl, a.R, t);
  const int q0 = max(__ldg(a.qsl + r), 0), q1 = min(__ldg(a.qsl + r + 1), a.T);
  if (t >= q1) return;  // locations that decrease
  const int pos = __ldg(a.seq_lens + r) - (q1 - q0) + (t - q0);
  if (pos < 0) return;
  const int rpos = a.positions ? __ldg(a.positions + t) : pos;
  if (a.rope && (rpos < 0 || rpos >= a.max_pos)) {
    if (a.status && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, MLA_STATUS_BAD_POSITION);
    return;
  }
  const float *rope = a.rope ? a.rope + int64_t(rpos) * a.P : nullptr;

  if (blockIdx.y == 0 && warp == 0) {
    // ---- the row
    const int blk_i = pos / a.bs;
    const int blk = blk_i < a.bt_stride ? __ldg(a.block_table + int64_t(r) * a.bt_stride + blk_i) : -1;
    const bool good = blk >= 0 && blk < a.num_blocks;
    if (!good && lane == 0 && a.status) atomicOr(a.status, MLA_STATUS_BAD_BLOCK);
    const int LP = a.L + a.P;
    const T *x = static_cast<const T *>(a.kv_a) + t * a.kv_a_ld;
    const T *w = static_cast<const T *>(a.norm_weight);
    T *d0 = good ? static_cast<T *>(a.kv_cache) + (int64_t(blk) * a.bs + pos % a.bs) * LP : nullptr;
    T *d1 = a.new_latent ? static_cast<T *>(a.new_latent) + int64_t(t) * LP : nullptr;
    float ss = 0.f;
    if (w) {
      if (a.vec_row) {
        for (int k = lane; k < a.L / N; k += 32) {
          Piece<T> p;
          p.load(x + k * N);
#pragma unroll
          for (int e = 0; e < N; ++e) ss = fmaf(p.v[e], p.v[e], ss);
        }
      } else {
        for (int k = lane; k < a.L; k += 32) {
          const float v = to_f32(x[k]);
          ss = fmaf(v, v, ss);
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    }
    const float inv = w ? 1.f / sqrtf(ss / float(a.L) + a.eps) : 1.f;
    if (a.vec_row) {
      for (int k = lane; k < a.L / N; k += 32) {
        Piece<T> p, g;
        p.load(x + k * N);
        if (w) {
          g.load(w + k * N);
#pragma unroll
          for (int e = 0; e < N; ++e) p.v[e] = p.v[e] * inv * g.v[e];
        }
        if (d0) p.store(d0 + k * N);
        if (d1) p.store(d1 + k * N);
      }
    } else {
      for (int k = lane; k < a.L; k += 32) {
        float v = to_f32(x[k]);
        if (w) v = v * inv * to_f32(w[k]);
        const T o = from_f32<T>(v);
        if (d0) d0[k] = o;
        if (d1) d1[k] = o;
      }
    }
    T *p0 = d0 ? d0 + a.L : nullptr, *p1 = d1 ? d1 + a.L : nullptr;
    if (!rope) {
      for (int k = lane; k < a.P; k += 32) {
        const T v = x[a.L + k];
        if (p0) p0[k] = v;
        if (p1) p1[k] = v;
      }
    } else {
      for (int k = lane; k < a.P / 2; k += 32)
        rotate_pair<T>(x + a.L, p0, p1, rope, a.P, k, a.interleaved);
    }
    return;
  }
  if (!a.q) return;
  // ---- the queries' rope columns: this block's share of the heads
  const int h0 = int(int64_t(a.H) * blockIdx.y / gridDim.y);
  const int h1 = int(int64_t(a.H) * (blockIdx.y + 1) / gridDim.y);
  const T *q = static_cast<const T *>(a.q) + int64_t(t) * a.H * (a.Dn + a.P) + a.Dn;
  T *o = static_cast<T *>(a.q_pe) + int64_t(t) * a.H * a.q_pe_ld;
  const int units = !rope ? a.P : a.vec_q ? a.P / (a.interleaved ? N : 2 * N) : a.P / 2;
  const int skip = blockIdx.y == 0 ? 32 : 0;  // warp 0 of the first block has the row
  for (int u = threadIdx.x - skip; u < (h1 - h0) * units; u += int(blockDim.x) - skip) {
    const int h = h0 + u / units, k = u % units;
    const T *src = q + int64_t(h) * (a.Dn + a.P);
    T *dst = o + h * a.q_pe_ld;
    if (!rope)
      dst[k] = src[k];
    else if (a.vec_q)
      rotate_piece<T>(src, dst, nullptr, rope, a.P, k, a.interleaved);
    else
      rotate_pair<T>(src, dst, nullptr, rope, a.P, k, a.interleaved);
  }
}

}  // namespace

int launch_append(const mla_dims_t &d, const void *kv_a, int64_t kv_a_ld, const void *norm_weight,
                  float eps, int T, int R, const int32_t *qsl, const int32_t *seq_lens,
                  const int32_t *positions, const float *rope, int max_pos, int interleaved,
                  void *kv_cache, int num_blocks, const int32_t *block_table, int bt_stride,
                  void *new_latent, const void *q, void *q_pe, int64_t q_pe_ld, int32_t *status,
                  cudaStream_t s) {
  const int es = elem_bytes(d.dtype), L = d.kv_lora_rank, P = d.qk_rope_dim;
  auto al = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  AppendArgs a{kv_a, norm_weight, q, kv_cache, new_latent, q_pe, qsl, seq_lens, positions,
               block_table, rope, status, kv_a_ld, q_pe_ld, T, R, d.num_heads, L, P,
               d.qk_nope_dim, d.block_size, num_blocks, bt_stride, max_pos, interleaved, eps, 0, 0};
  // cache rows are multiples of 16 bytes from an aligned base; the rest is checked here
  a.vec_row = (L * es) % 16 == 0 && (kv_a_ld * es) % 16 == 0 && al(kv_a) && al(norm_weight) &&
              al(kv_cache) && al(new_latent);
  const int pair_bytes = interleaved ? P * es : P / 2 * es;  // a rotation's 16-byte pieces
  a.vec_q = q && pair_bytes % 16 == 0 && (d.qk_nope_dim * es) % 16 == 0 && (q_pe_ld * es) % 16 == 0 &&
            al(q) && al(q_pe);
  // enough blocks for every SM where there are heads to share out
  const int want = 2 * num_sms();
  const int most = q ? (d.num_heads + 7) / 8 : 1;
  int ys = T >= want ? 1 : (want + T - 1) / T;
  if (ys > most) ys = most;
  launch_begin(s);
  const dim3 grid(T, ys);
  const int threads = q ? 32 * WARPS : 32;
  if (d.dtype == MLA_DTYPE_BF16)
    append_kernel<__nv_bfloat16><<<grid, threads, 0, s>>>(a);
  else
    append_kernel<float><<<grid, threads, 0, s>>>(a);
  return launch_status(s, "append_kernel");
}

}  // namespace mla
