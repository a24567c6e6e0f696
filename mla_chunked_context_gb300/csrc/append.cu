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
// when there are few.  Many tokens live on warps in flight, that is on few
// registers: reading two heads at once takes 62 us where this takes 53.6, rows
// and queries before the sequence is known 60.5, one kernel for both orders of
// the rotation 55.0; nothing of it changes 16 tokens' time.  A block serves one
// token: warp 0 of its first block the row, all other threads the heads of the
// queries, each the same columns (and angles) of several heads.  Few tokens
// spread their heads over several blocks.
// Measured, 128 heads, bf16: 8192 tokens (299 MB) 53.6 us, 5.6 TB/s or 82% of
// copy bandwidth, the queries' rope columns being 128 of every 384 bytes; 16
// tokens 4.1 us in a graph.
#include "common.cuh"

namespace mla {
namespace {

// Of a block.  8192 tokens with 2, 3, 5, 8, 16 warps took 12, 1, 1, 23 and 107%
// longer.
constexpr int WARPS = 4;

struct AppendArgs {
  const void *kv_a, *norm_weight, *q;
  void *kv_cache, *new_latent, *q_pe;
  const int32_t *qsl, *seq_lens, *positions, *block_table;
  const float *rope;
  int32_t *status;
  int64_t kv_a_ld, q_pe_ld;
  int T, R, H, L, P, Dn, bs, num_blocks, bt_stride, max_pos;
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

// 16-byte pieces: interleaved, one piece holds N/2 pairs; half-split, piece k
// (x) goes with piece k + P/(2N) (y).  c, s: the pairs' cosines and sines.
template <typename T>
__device__ __forceinline__ void rotate_piece(Piece<T> &x, Piece<T> &y, const float *c,
                                             const float *s, bool interleaved) {
  constexpr int N = Piece<T>::N;
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const float a = x.v[2 * e], b = x.v[2 * e + 1];
      x.v[2 * e] = a * c[e] - b * s[e];
      x.v[2 * e + 1] = b * c[e] + a * s[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float a = x.v[e], b = y.v[e];
      x.v[e] = a * c[e] - b * s[e];
      y.v[e] = b * c[e] + a * s[e];
    }
  }
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * WARPS) append_kernel(AppendArgs a) {
  constexpr int N = Piece<T>::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x;
  const bool row_warp = blockIdx.y == 0 && warp == 0;
  chain_release();
  chain_wait();

  // ---- the token's sequence and position
  const int first = max(__ldg(a.qsl), 0);
  if (t < first || t >= min(__ldg(a.qsl + a.R), a.T)) return;
  const int r = find_seq_warp(a.qsl, a.R, t);
  const int q0 = max(__ldg(a.qsl + r), 0), q1 = min(__ldg(a.qsl + r + 1), a.T);
  if (t >= q1) return;  // locations that decrease
  const int pos = max(__ldg(a.seq_lens + r), 0) - (q1 - q0) + (t - q0);
  if (pos < 0) return;
  const int rpos = a.positions ? __ldg(a.positions + t) : pos;
  if (a.rope && (rpos < 0 || rpos >= a.max_pos)) {
    if (a.status && threadIdx.x == 0 && blockIdx.y == 0)
      atomicOr(a.status, MLA_STATUS_BAD_POSITION);
    return;
  }
  const float *rope = a.rope ? a.rope + int64_t(rpos) * a.P : nullptr;

  const T *x = static_cast<const T *>(a.kv_a) + t * a.kv_a_ld;
  if (row_warp) {
    const T *w = static_cast<const T *>(a.norm_weight);
    const int n_pieces = a.L / N;
    const int blk_i = pos / a.bs;
    const int blk =
        blk_i < a.bt_stride ? __ldg(a.block_table + int64_t(r) * a.bt_stride + blk_i) : -1;
    const bool good = blk >= 0 && blk < a.num_blocks;
    if (!good && lane == 0 && a.status) atomicOr(a.status, MLA_STATUS_BAD_BLOCK);
    const int LP = a.L + a.P;
    T *d0 = good ? static_cast<T *>(a.kv_cache) + (int64_t(blk) * a.bs + pos % a.bs) * LP : nullptr;
    T *d1 = a.new_latent ? static_cast<T *>(a.new_latent) + int64_t(t) * LP : nullptr;
    float inv = 1.f;
    if (w) {
      float ss = 0.f;
      auto square = [&](const Piece<T> &p) {
#pragma unroll
        for (int e = 0; e < N; ++e) ss = fmaf(p.v[e], p.v[e], ss);
      };
      if (a.vec_row) {
        for (int j = lane; j < n_pieces; j += 32) {
          Piece<T> p;
          p.load(x + j * N);
          square(p);
        }
      } else {
        for (int j = lane; j < a.L; j += 32) {
          const float v = to_f32(x[j]);
          ss = fmaf(v, v, ss);
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      inv = 1.f / sqrtf(ss / float(a.L) + a.eps);
    }
    if (a.vec_row) {
      for (int j = lane; j < n_pieces; j += 32) {
        Piece<T> p;
        p.load(x + j * N);
        if (w) {
          Piece<T> g;
          g.load(w + j * N);
#pragma unroll
          for (int e = 0; e < N; ++e) p.v[e] = p.v[e] * inv * g.v[e];
        }
        if (d0) p.store(d0 + j * N);
        if (d1) p.store(d1 + j * N);
      }
    } else {
      for (int j = lane; j < a.L; j += 32) {
        float v = to_f32(x[j]);
        if (w) v = v * inv * to_f32(w[j]);
        const T o = from_f32<T>(v);
        if (d0) d0[j] = o;
        if (d1) d1[j] = o;
      }
    }
    T *p0 = d0 ? d0 + a.L : nullptr, *p1 = d1 ? d1 + a.L : nullptr;
    if (!rope) {
      for (int j = lane; j < a.P; j += 32) {
        const T v = x[a.L + j];
        if (p0) p0[j] = v;
        if (p1) p1[j] = v;
      }
    } else {
      for (int j = lane; j < a.P / 2; j += 32)
        rotate_pair<T>(x + a.L, p0, p1, rope, a.P, j, INTERLEAVED);
    }
    return;
  }
  if (!a.q) return;
  // the queries: this block's share of the heads
  const int h0 = int(int64_t(a.H) * blockIdx.y / gridDim.y);
  const int h1 = int(int64_t(a.H) * (blockIdx.y + 1) / gridDim.y);
  const int q_tid = int(threadIdx.x) - (blockIdx.y == 0 ? 32 : 0);
  const int q_threads = int(blockDim.x) - (blockIdx.y == 0 ? 32 : 0);
  const int qk = a.Dn + a.P, y_off = a.P / 2;
  const T *q = static_cast<const T *>(a.q) + int64_t(t) * a.H * qk + a.Dn;
  T *qo = static_cast<T *>(a.q_pe) + int64_t(t) * a.H * a.q_pe_ld;
  if (a.vec_q) {
    // a thread has columns k of heads qh, qh + q_step, ...
    const int units = a.P / (INTERLEAVED ? N : 2 * N);  // of a head, as pieces
    const int q_step = q_threads / units, k = q_tid % units, qh = h0 + q_tid / units;
    if (q_tid >= q_step * units || qh >= h1) return;
    // the angles of this thread's columns, for all of its heads
    constexpr int NA = N;
    const int n_ang = INTERLEAVED ? N / 2 : N;
    float c[NA], sn[NA];
#pragma unroll
    for (int e = 0; e < NA; e += 2)  // (the table's rows are 8-byte aligned here)
      if (e < n_ang) {
        const float2 u = __ldg(reinterpret_cast<const float2 *>(rope + k * n_ang + e));
        const float2 v = __ldg(reinterpret_cast<const float2 *>(rope + y_off + k * n_ang + e));
        c[e] = u.x;
        c[e + 1] = u.y;
        sn[e] = v.x;
        sn[e + 1] = v.y;
      }
#pragma unroll 1
    for (int h = qh; h < h1; h += q_step) {
      const T *src = q + int64_t(h) * qk + k * N;
      T *dst = qo + h * a.q_pe_ld + k * N;
      Piece<T> px, py;
      px.load(src);
      if (!INTERLEAVED) py.load(src + y_off);
      rotate_piece<T>(px, py, c, sn, INTERLEAVED);
      px.store(dst);
      if (!INTERLEAVED) py.store(dst + y_off);
    }
    return;
  }
  const int per_head = rope ? a.P / 2 : a.P;
  for (int u = q_tid; u < (h1 - h0) * per_head; u += q_threads) {
    const int h = h0 + u / per_head, j = u % per_head;
    if (rope)
      rotate_pair<T>(q + int64_t(h) * qk, qo + h * a.q_pe_ld, nullptr, rope, a.P, j, INTERLEAVED);
    else
      qo[h * a.q_pe_ld + j] = q[int64_t(h) * qk + j];
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
               d.qk_nope_dim, d.block_size, num_blocks, bt_stride, max_pos, eps, 0, 0};
  // cache rows are multiples of 16 bytes from an aligned base; the rest is checked here
  a.vec_row = (L * es) % 16 == 0 && (kv_a_ld * es) % 16 == 0 && al(kv_a) && al(norm_weight) &&
              al(kv_cache) && al(new_latent);
  const int pair_bytes = interleaved ? P * es : P / 2 * es;  // a rotation's 16-byte pieces
  const int units = P * es / (interleaved ? 16 : 32);  // of a head
  a.vec_q = q && rope && (reinterpret_cast<uintptr_t>(rope) & 7) == 0 && units >= 1 &&
            units <= 32 * (WARPS - 1) && pair_bytes % 16 == 0 && (d.qk_nope_dim * es) % 16 == 0 &&
            (q_pe_ld * es) % 16 == 0 && al(q) && al(q_pe);
  // enough blocks for every SM where there are heads to share out
  const int want = 2 * num_sms();
  const int most = q ? (d.num_heads + 7) / 8 : 1;
  int ys = T >= want ? 1 : (want + T - 1) / T;
  if (ys > most) ys = most;
  const dim3 grid(T, ys);
  const int threads = q ? 32 * WARPS : 32;
  auto *kernel = d.dtype == MLA_DTYPE_BF16
                     ? (interleaved ? append_kernel<__nv_bfloat16, true>
                                    : append_kernel<__nv_bfloat16, false>)
                     : (interleaved ? append_kernel<float, true> : append_kernel<float, false>);
  return launch_chained(kernel, grid, threads, 0, 1, s, "append_kernel", a);
}

}  // namespace mla
