// CUDA-core kernels of the decode calls, for float32 storage and the head
// shapes the tensor-core kernels are not built for.  Arithmetic is float32
// throughout, rounded once at the end.
//
//  * head_gemm_simt: per head h, C[t, n] = sum_k A[t, k] B(k, n): the query
//    absorption (B = W_uk[h], n contiguous) and the output expansion (B =
//    W_uv[h]^T, k contiguous); 64x64 shared-memory tiles, 4x4 outputs a
//    thread.
//  * latent_attn_simt: one block per (new token, head).  Its warps take the
//    keys in turn, KB at a time (the dot products' loads and reductions
//    overlap, and the next ones' block ids are on their way), each with its
//    own running maximum and sum; the warps' results are joined in shared
//    memory.  Bound by the latency of that chain: 16 warps of 8 keys took 28.7
//    to 14.4 us on 4 x 3 tokens, 16 heads, up to 700 keys of 80 floats.
#include "common.cuh"

namespace mla {
namespace {

constexpr int GT = 64, GK = 16;

struct HeadGemm {
  const void *a, *b;
  void *c;
  int64_t a_row, a_head;       // strides of A in elements: token, head
  int64_t b_k, b_n, b_head;    // strides of B
  int64_t c_row, c_head;
  int M, N, K;
};

template <typename T>
__global__ void __launch_bounds__(256) head_gemm_simt(HeadGemm g) {
  __shared__ float As[GK][GT + 1];
  __shared__ float Bs[GK][GT + 1];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int n0 = blockIdx.x * GT, m0 = blockIdx.y * GT, h = blockIdx.z;
  const T *A = static_cast<const T *>(g.a) + h * g.a_head;
  const T *B = static_cast<const T *>(g.b) + h * g.b_head;
  T *C = static_cast<T *>(g.c) + h * g.c_head;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += GK) {
    for (int e = threadIdx.x; e < GT * GK; e += 256) {
      const int r = e / GK, k = e % GK;
      As[k][r] = (m0 + r < g.M && k0 + k < g.K) ? to_f32(A[(m0 + r) * g.a_row + k0 + k]) : 0.f;
      // walk B along its contiguous dimension
      const int rb = g.b_n == 1 ? e % GT : r, kb = g.b_n == 1 ? e / GT : k;
      Bs[kb][rb] = (n0 + rb < g.N && k0 + kb < g.K)
                       ? to_f32(B[(k0 + kb) * g.b_k + (n0 + rb) * g.b_n])
                       : 0.f;
    }
    __syncthreads();
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
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < g.M && n < g.N) C[m * g.c_row + n] = from_f32<T>(acc[i][j]);
    }
}

// q_latent[row, L:L+P) = q[row, Dn:Dn+P) over rows (token, head)
template <typename T>
__global__ void __launch_bounds__(256) copy_rope_columns(const T *q, T *o, int64_t rows, int q_ld,
                                                         int q_off, int o_ld, int o_off, int P) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= rows * P) return;
  const int64_t row = i / P;
  const int k = int(i % P);
  o[row * o_ld + o_off + k] = q[row * q_ld + q_off + k];
}

struct LatentArgs {
  const void *q, *cache;
  void *o;
  float *lse;
  const int32_t *qsl, *seq_lens, *block_table;
  int32_t *status;
  int T, R, H, L, P, bs, num_blocks, bt_stride, causal;
  float scale_log2;
};

// NV: 32-element slices of a row held by a warp (L + P <= 32 * NV); AW: warps of
// a block; KB: keys a warp takes at once
template <typename T, int NV, int AW, int KB>
__global__ void __launch_bounds__(32 * AW) latent_attn_simt(LatentArgs a) {
  extern __shared__ float sh[];  // [AW][L] partial outputs, [AW] maxima, [AW] sums
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int lo = max(__ldg(a.qsl), 0), hi = min(__ldg(a.qsl + a.R), a.T);
  if (t < lo || t >= hi) return;
  const int r = find_seq(a.qsl, a.R, t);
  const int q0 = max(__ldg(a.qsl + r), 0), q1 = min(__ldg(a.qsl + r + 1), a.T);
  if (t >= q1) return;
  const int len = max(__ldg(a.seq_lens + r), 0);
  const int keys = int(min((long long)len, (long long)a.bt_stride * a.bs));
  const int nk = a.causal ? max(0, min(keys, len - (q1 - q0) + (t - q0) + 1)) : keys;
  const int LP = a.L + a.P;
  const T *q = static_cast<const T *>(a.q) + (int64_t(t) * a.H + h) * LP;
  const T *cache = static_cast<const T *>(a.cache);
  const int32_t *bt = a.block_table + int64_t(r) * a.bt_stride;
  float qr[NV], acc[NV];
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    const int d = lane + 32 * e;
    qr[e] = d < LP ? to_f32(q[d]) : 0.f;
    acc[e] = 0.f;
  }
  float m = neg_inf(), l = 0.f;
  bool bad = keys < len;
  // lane i < KB finds the cache row of key j0 + i; -1: past the end or bad
  auto find = [&](int j0) -> int64_t {
    const int j = j0 + lane;
    if (lane >= KB || j >= nk) return -1;
    const int b = j / a.bs;
    const int blk = __ldg(bt + b);
    if (blk < 0 || blk >= a.num_blocks) {
      bad = true;
      return -1;
    }
    return (int64_t(blk) * a.bs + j % a.bs) * LP;
  };
  int64_t mine = find(warp * KB);
  for (int j0 = warp * KB; j0 < nk; j0 += AW * KB) {
    const T *row[KB];
    float s[KB];
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int64_t off = __shfl_sync(0xffffffffu, mine, i);
      row[i] = off < 0 ? nullptr : cache + off;
      s[i] = 0.f;
    }
    mine = find(j0 + AW * KB);
    float c[KB][NV];
#pragma unroll
    for (int i = 0; i < KB; ++i)
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        const int d = lane + 32 * e;
        c[i][e] = (row[i] && d < LP) ? to_f32(row[i][d]) : 0.f;
        s[i] = fmaf(qr[e], c[i][e], s[i]);
      }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < KB; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], off);
    float mn = m;
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      s[i] = j0 + i < nk ? s[i] * a.scale_log2 : neg_inf();
      mn = fmaxf(mn, s[i]);
    }
    const float base = is_neg_inf(mn) ? 0.f : mn;  // every score so far is -inf
    const float corr = exp2f(m - base);
    float p[KB];
    l *= corr;
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      p[i] = exp2f(s[i] - base);
      l += p[i];
    }
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      acc[e] *= corr;
#pragma unroll
      for (int i = 0; i < KB; ++i) acc[e] = fmaf(p[i], c[i][e], acc[e]);
    }
    m = mn;
  }
  if (bad && a.status) atomicOr(a.status, MLA_STATUS_BAD_BLOCK);
  float *sm = sh + AW * a.L, *sl = sm + AW;
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    const int d = lane + 32 * e;
    if (d < a.L) sh[warp * a.L + d] = acc[e];
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float mx = neg_inf(), tot = 0.f, w[AW];
#pragma unroll
  for (int i = 0; i < AW; ++i) mx = fmaxf(mx, sm[i]);
  const float base = is_neg_inf(mx) ? 0.f : mx;
#pragma unroll
  for (int i = 0; i < AW; ++i) {
    w[i] = exp2f(sm[i] - base);
    tot = fmaf(w[i], sl[i], tot);
  }
  const float inv = tot > 0.f ? 1.f / tot : 0.f;
  T *o = static_cast<T *>(a.o) + (int64_t(t) * a.H + h) * a.L;
  for (int d = threadIdx.x; d < a.L; d += 32 * AW) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < AW; ++i) v = fmaf(w[i], sh[i * a.L + d], v);
    o[d] = from_f32<T>(v * inv);
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[int64_t(h) * a.T + t] =
        tot > 0.f ? (mx + log2f(tot)) * 0.69314718055994531f : neg_inf();
}

template <typename T, int NV, int AW, int KB>
void launch_attn_n(const LatentArgs &a, int grid, cudaStream_t s) {
  const size_t smem = (size_t(AW) * a.L + 2 * AW) * sizeof(float);  // at most 41 KB
  latent_attn_simt<T, NV, AW, KB><<<grid, 32 * AW, smem, s>>>(a);
}

template <typename T>
void launch_attn_t(const LatentArgs &a, int grid, cudaStream_t s) {
  const int LP = a.L + a.P;
  if (LP <= 128)
    launch_attn_n<T, 4, 16, 8>(a, grid, s);
  else if (LP <= 320)
    launch_attn_n<T, 10, 16, 4>(a, grid, s);
  else if (LP <= 640)
    launch_attn_n<T, 20, 16, 2>(a, grid, s);
  else
    launch_attn_n<T, 32, 8, 2>(a, grid, s);
}

template <typename T>
int head_gemm(const HeadGemm &g, int H, cudaStream_t s) {
  launch_begin(s);
  head_gemm_simt<T><<<dim3((g.N + GT - 1) / GT, (g.M + GT - 1) / GT, H), 256, 0, s>>>(g);
  return launch_status(s, "head_gemm_simt");
}

}  // namespace

int launch_absorb_simt(const mla_dims_t &d, const void *q, int T, const void *w, int rope_columns,
                       void *q_latent, cudaStream_t s) {
  const int L = d.kv_lora_rank, P = d.qk_rope_dim, Dn = d.qk_nope_dim, H = d.num_heads;
  const int QK = Dn + P, LP = L + P;
  HeadGemm g{q, w, q_latent, int64_t(H) * QK, QK, L, 1, int64_t(Dn + d.v_dim) * L,
             int64_t(H) * LP, LP, T, L, Dn};
  const bool bf = d.dtype == MLA_DTYPE_BF16;
  int rc = bf ? head_gemm<__nv_bfloat16>(g, H, s) : head_gemm<float>(g, H, s);
  if (rc || !rope_columns || P == 0) return rc;
  const int64_t rows = int64_t(T) * H;
  const unsigned blocks = unsigned((rows * P + 255) / 256);
  launch_begin(s);
  if (bf)
    copy_rope_columns<<<blocks, 256, 0, s>>>(static_cast<const __nv_bfloat16 *>(q),
                                             static_cast<__nv_bfloat16 *>(q_latent), rows, QK, Dn,
                                             LP, L, P);
  else
    copy_rope_columns<<<blocks, 256, 0, s>>>(static_cast<const float *>(q),
                                             static_cast<float *>(q_latent), rows, QK, Dn, LP, L,
                                             P);
  return launch_status(s, "copy_rope_columns");
}

int launch_expand_simt(const mla_dims_t &d, const void *o_latent, int T, const void *w, void *out,
                       cudaStream_t s) {
  const int L = d.kv_lora_rank, Dn = d.qk_nope_dim, Dv = d.v_dim, H = d.num_heads;
  const int64_t off = int64_t(Dn) * L * elem_bytes(d.dtype);
  HeadGemm g{o_latent, static_cast<const char *>(w) + off, out, int64_t(H) * L, L, 1, L,
             int64_t(Dn + Dv) * L, int64_t(H) * Dv, Dv, T, Dv, L};
  return d.dtype == MLA_DTYPE_BF16 ? head_gemm<__nv_bfloat16>(g, H, s) : head_gemm<float>(g, H, s);
}

bool latent_simt_ok(const mla_dims_t &d) { return d.kv_lora_rank + d.qk_rope_dim <= 1024; }

int launch_latent_attn_simt(const mla_dims_t &d, int causal, int R, const int32_t *qsl,
                            const int32_t *seq_lens, int T, const void *q, const void *cache,
                            int num_blocks, const int32_t *block_table, int bt_stride, void *o,
                            float *lse, int32_t *status, cudaStream_t s) {
  LatentArgs a{q, cache, o, lse, qsl, seq_lens, block_table, status, T, R, d.num_heads,
               d.kv_lora_rank, d.qk_rope_dim, d.block_size, num_blocks, bt_stride, causal,
               d.softmax_scale * 1.4426950408889634f};
  launch_begin(s);
  if (d.dtype == MLA_DTYPE_BF16)
    launch_attn_t<__nv_bfloat16>(a, T * d.num_heads, s);
  else
    launch_attn_t<float>(a, T * d.num_heads, s);
  return launch_status(s, "latent_attn_simt");
}

}  // namespace mla
