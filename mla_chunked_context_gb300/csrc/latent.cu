// CUDA-core kernels of the decode calls, for float32 storage and the head
// shapes the tensor-core kernels are not built for.  Arithmetic is float32
// throughout, rounded once at the end.
//
//  * head_gemm_simt: per head h, C[t, n] = sum_k A[t, k] B(k, n): the query
//    absorption (B = W_uk[h], n contiguous) and the output expansion (B =
//    W_uv[h]^T, k contiguous); 64x64 shared-memory tiles, 4x4 outputs a
//    thread, 32 of the contraction a step, the next step's loads in flight
//    meanwhile; the first column block copies the rope columns.  (16 a step,
//    loaded when needed: expansion of 500 tokens, 40 heads of 64 -> 32 14.4 us,
//    so 10.0; of one token 5.9 and 4.1.)
//  * latent_attn_simt: one block per (new token, head).  A group of G lanes
//    takes a key at a time (U keys in flight), each lane NC 16-byte pieces of
//    its row, so that a score costs log2 G shuffles and its weight needs none;
//    each group has its own running maximum and sum, joined over the warp by
//    shuffles and over the block in shared memory.  (A warp for a key, 32
//    lanes over its columns, kept eight rows of 4-byte loads in flight and took
//    20 us for 4 x 3 tokens, 16 heads, 700 keys of 80 floats; this 8.4.)  Every
//    head of a token reads the token's keys, all but the first from L2: 8 x 2000
//    keys of 576 floats, 16 heads 115 us (590 MB, 5.1 TB/s; the keys once would
//    take 5.5), 16 x 4096 of 288 bf16 144 us.
#include "common.cuh"

namespace mla {
namespace {

constexpr int GT = 64, GK = 32;

struct HeadGemm {
  const void *a, *b;
  void *c;
  int64_t a_row, a_head;       // strides of A in elements: token, head
  int64_t b_k, b_n, b_head;    // strides of B
  int64_t c_row, c_head;
  int M, N, K;
  int rope;  // columns of A behind its K that go to C behind its N
};

template <typename T>
__global__ void __launch_bounds__(256) head_gemm_simt(HeadGemm g) {
  __shared__ float As[GK][GT + 1];
  __shared__ float Bs[GK][GT + 1];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  chain_release();
  chain_wait();
  const int n0 = blockIdx.x * GT, m0 = blockIdx.y * GT, h = blockIdx.z;
  const T *A = static_cast<const T *>(g.a) + h * g.a_head;
  const T *B = static_cast<const T *>(g.b) + h * g.b_head;
  T *C = static_cast<T *>(g.c) + h * g.c_head;
  float acc[4][4] = {};
  // the next step's elements come while this one is multiplied
  constexpr int NE = GT * GK / 256;
  float va[NE], vb[NE];
  auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * 256 + threadIdx.x, r = e / GK, k = e % GK;
      va[i] = (m0 + r < g.M && k0 + k < g.K) ? to_f32(A[(m0 + r) * g.a_row + k0 + k]) : 0.f;
      // walk B along its contiguous dimension
      const int rb = g.b_n == 1 ? e % GT : r, kb = g.b_n == 1 ? e / GT : k;
      vb[i] = (n0 + rb < g.N && k0 + kb < g.K) ? to_f32(B[(k0 + kb) * g.b_k + (n0 + rb) * g.b_n])
                                               : 0.f;
    }
  };
  load(0);
  for (int k0 = 0; k0 < g.K; k0 += GK) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * 256 + threadIdx.x, r = e / GK, k = e % GK;
      As[k][r] = va[i];
      Bs[g.b_n == 1 ? e / GT : k][g.b_n == 1 ? e % GT : r] = vb[i];
    }
    __syncthreads();
    if (k0 + GK < g.K) load(k0 + GK);
#pragma unroll
    for (int k = 0; k < GK; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = As[k][ty + 16 * i];
        b[i] = Bs[k][tx + 16 * i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e < GT * g.rope; e += 256) {
      const int m = m0 + e / g.rope, k = e % g.rope;
      if (m < g.M) C[m * g.c_row + g.N + k] = A[m * g.a_row + g.K + k];
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < g.M && n < g.N) C[m * g.c_row + n] = from_f32<T>(acc[i][j]);
    }
}

struct LatentArgs {
  const void *q, *cache;
  void *o;
  float *lse;
  const int32_t *qsl, *seq_lens, *block_table;
  int32_t *status;
  int T, R, H, L, P, bs, num_blocks, bt_stride, causal;
  Divider by_bs;
  float scale_log2;
};

// 16 bytes of T
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ float get(int i) const {
    return to_f32(reinterpret_cast<const T *>(&raw)[i]);
  }
};

// G lanes a key, NC pieces of 16 bytes a lane (rows of at most 16 G NC bytes),
// AW warps a block, U keys of a group in flight
template <typename T, int G, int NC, int AW, int U>
__global__ void __launch_bounds__(32 * AW) latent_attn_simt(LatentArgs a) {
  extern __shared__ float sh[];  // [AW][L] partial outputs, [AW] maxima, [AW] sums
  constexpr int N = Vec<T>::N, GROUPS = AW * 32 / G, STEP = GROUPS * U;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % G, group = threadIdx.x / G;
  const int t = blockIdx.x / a.H, h = blockIdx.x % a.H;
  chain_release();
  chain_wait();
  const int lo = max(__ldg(a.qsl), 0), hi = min(__ldg(a.qsl + a.R), a.T);
  if (t < lo || t >= hi) return;
  const int r = find_seq(a.qsl, a.R, t);
  const int q0 = max(__ldg(a.qsl + r), 0), q1 = min(__ldg(a.qsl + r + 1), a.T);
  if (t >= q1) return;
  const int len = max(__ldg(a.seq_lens + r), 0);
  const int keys = keys_of(len, a.bt_stride, a.bs);
  const int nk = a.causal ? max(0, min(keys, len - (q1 - q0) + (t - q0) + 1)) : keys;
  const int LP = a.L + a.P;
  const T *q = static_cast<const T *>(a.q) + (int64_t(t) * a.H + h) * LP;
  const T *cache = static_cast<const T *>(a.cache);
  const int32_t *bt = a.block_table + int64_t(r) * a.bt_stride;
  bool bad = keys < len;
  // block ids of this group's next keys (key base + u * GROUPS + group)
  int blk[U];
  auto look_up = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = base + u * GROUPS + group;
      blk[u] = j < nk ? __ldg(bt + a.by_bs.quotient(j)) : -2;
    }
  };
  look_up(0);
  float qr[NC][N], acc[NC][N];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int d = (c * G + sub) * N + e;
      qr[c][e] = d < LP ? to_f32(q[d]) * a.scale_log2 : 0.f;
      acc[c][e] = 0.f;
    }
  float m = neg_inf(), l = 0.f;
  for (int base = 0; base < nk; base += STEP) {
    Vec<T> v[U][NC];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = base + u * GROUPS + group;
      live[u] = j < nk;
      const bool good = blk[u] >= 0 && blk[u] < a.num_blocks;
      if (live[u] && !good) bad = true;
      const T *row = cache + (int64_t(blk[u]) * a.bs + (j - a.by_bs.quotient(j) * a.bs)) * LP;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d = (c * G + sub) * N;
        v[u][c].raw = good && d < LP ? *reinterpret_cast<const uint4 *>(row + d)
                                     : make_uint4(0, 0, 0, 0);
      }
    }
    look_up(base + STEP);
    float x[U], mn = m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < N; ++e) x[u] = fmaf(qr[c][e], v[u][c].get(e), x[u]);
    }
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] += __shfl_xor_sync(0xffffffffu, x[u], off);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live[u]) x[u] = neg_inf();
      mn = fmaxf(mn, x[u]);
    }
    const float ref = is_neg_inf(mn) ? 0.f : mn;  // every score so far is -inf
    const float corr = exp2f(m - ref);
    m = mn;
    l *= corr;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < N; ++e) acc[c][e] *= corr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float p = exp2f(x[u] - ref);
      l += p;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < N; ++e) acc[c][e] = fmaf(p, v[u][c].get(e), acc[c][e]);
    }
  }
  if (bad && a.status && sub == 0) atomicOr(a.status, MLA_STATUS_BAD_BLOCK);
  // the warp's groups
  float mw = m;
#pragma unroll
  for (int off = 16; off >= G; off >>= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, off));
  const float fw = exp2f(m - (is_neg_inf(mw) ? 0.f : mw));
  l *= fw;
#pragma unroll
  for (int off = 16; off >= G; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      acc[c][e] *= fw;
#pragma unroll
      for (int off = 16; off >= G; off >>= 1)
        acc[c][e] += __shfl_xor_sync(0xffffffffu, acc[c][e], off);
      const int d = (c * G + sub) * N + e;
      if (lane < G && d < a.L) sh[warp * a.L + d] = acc[c][e];
    }
  float *sm = sh + AW * a.L, *sl = sm + AW;
  if (lane == 0) {
    sm[warp] = mw;
    sl[warp] = l;
  }
  __syncthreads();
  float mx = neg_inf(), tot = 0.f, w[AW];
#pragma unroll
  for (int i = 0; i < AW; ++i) mx = fmaxf(mx, sm[i]);
  const float ref = is_neg_inf(mx) ? 0.f : mx;
#pragma unroll
  for (int i = 0; i < AW; ++i) {
    w[i] = exp2f(sm[i] - ref);
    tot = fmaf(w[i], sl[i], tot);
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  T *o = static_cast<T *>(a.o) + (int64_t(t) * a.H + h) * a.L;
  for (int d = threadIdx.x; d < a.L; d += 32 * AW) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < AW; ++i) v = fmaf(w[i], sh[i * a.L + d], v);
    o[d] = from_f32<T>(v * inv);
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[int64_t(h) * a.T + t] =
        tot == 0.f ? neg_inf() : (ref + log2f(tot)) * 0.69314718055994531f;
}

template <typename T, int G, int NC, int AW, int U>
int launch_attn_n(const LatentArgs &a, int grid, cudaStream_t s) {
  const size_t smem = (size_t(AW) * a.L + 2 * AW) * sizeof(float);  // at most 33 KB
  return launch_chained(latent_attn_simt<T, G, NC, AW, U>, grid, 32 * AW, smem, 1, s,
                        "latent_attn_simt", a);
}

// By the 16-byte pieces of a row (at most 256: L + P <= 1024).
template <typename T>
int launch_attn_t(const LatentArgs &a, int grid, cudaStream_t s) {
  const int pieces = (a.L + a.P) * int(sizeof(T)) / 16;
  if (pieces <= 20) return launch_attn_n<T, 4, 5, 8, 2>(a, grid, s);
  if (pieces <= 40) return launch_attn_n<T, 8, 5, 8, 2>(a, grid, s);
  if (pieces <= 80) return launch_attn_n<T, 16, 5, 8, 2>(a, grid, s);
  if (pieces <= 160) return launch_attn_n<T, 32, 5, 8, 2>(a, grid, s);
  return launch_attn_n<T, 32, 8, 8, 1>(a, grid, s);
}

template <typename T>
int head_gemm(const HeadGemm &g, int H, cudaStream_t s) {
  return launch_chained(head_gemm_simt<T>, dim3((g.N + GT - 1) / GT, (g.M + GT - 1) / GT, H), 256,
                        0, 1, s, "head_gemm_simt", g);
}

}  // namespace

int launch_absorb_simt(const mla_dims_t &d, const void *q, int T, const void *w, int rope_columns,
                       void *q_latent, cudaStream_t s) {
  const int L = d.kv_lora_rank, P = d.qk_rope_dim, Dn = d.qk_nope_dim, H = d.num_heads;
  const int QK = Dn + P, LP = L + P;
  HeadGemm g{q, w, q_latent, int64_t(H) * QK, QK, L, 1, int64_t(Dn + d.v_dim) * L,
             int64_t(H) * LP, LP, T, L, Dn, rope_columns ? P : 0};
  return d.dtype == MLA_DTYPE_BF16 ? head_gemm<__nv_bfloat16>(g, H, s) : head_gemm<float>(g, H, s);
}

int launch_expand_simt(const mla_dims_t &d, const void *o_latent, int T, const void *w, void *out,
                       cudaStream_t s) {
  const int L = d.kv_lora_rank, Dn = d.qk_nope_dim, Dv = d.v_dim, H = d.num_heads;
  const int64_t off = int64_t(Dn) * L * elem_bytes(d.dtype);
  HeadGemm g{o_latent, static_cast<const char *>(w) + off, out, int64_t(H) * L, L, 1, L,
             int64_t(Dn + Dv) * L, int64_t(H) * Dv, Dv, T, Dv, L, 0};
  return d.dtype == MLA_DTYPE_BF16 ? head_gemm<__nv_bfloat16>(g, H, s) : head_gemm<float>(g, H, s);
}

bool latent_simt_ok(const mla_dims_t &d) { return d.kv_lora_rank + d.qk_rope_dim <= 1024; }

int launch_latent_attn_simt(const mla_dims_t &d, int causal, int R, const int32_t *qsl,
                            const int32_t *seq_lens, int T, const void *q, const void *cache,
                            int num_blocks, const int32_t *block_table, int bt_stride, void *o,
                            float *lse, int32_t *status, cudaStream_t s) {
  LatentArgs a{q, cache, o, lse, qsl, seq_lens, block_table, status, T, R, d.num_heads,
               d.kv_lora_rank, d.qk_rope_dim, d.block_size, num_blocks, bt_stride, causal,
               Divider(d.block_size), d.softmax_scale * 1.4426950408889634f};
  if (d.dtype == MLA_DTYPE_BF16) return launch_attn_t<__nv_bfloat16>(a, T * d.num_heads, s);
  return launch_attn_t<float>(a, T * d.num_heads, s);
}

}  // namespace mla
