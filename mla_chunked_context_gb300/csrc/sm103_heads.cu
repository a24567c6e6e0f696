// The decode step's per-head products with the two halves of W_kv_b on the
// 5th-generation tensor cores (sm_103a), DeepSeek-V3 head shape, bf16:
//   absorb: q_latent[t, h, :] = q_nope[t, h, :] W_uk[h]     128 -> 512 columns
//   expand: out[t, h, :]      = W_uv[h] o_latent[t, h, :]   512 -> 128 columns
// Per token and head 131 kFLOP on 1.3 KB: far below the tensor pipe's share,
// so the kernel is there to stream: the weight halves (16.8 MB each at 128
// heads) once for few tokens, the activations once for many.
//
// A CTA computes 128 tokens x NC columns of one head; two (expand) or three to
// four (absorb) CTAs an SM, so that one's loads run beside another's epilogue.
// NC is 128, and 64 where heads and tokens are too few to give every SM two
// CTAs, to spread the weights' loads over more SMs.  A stage has room for the
// tokens there are, so that for few of them all of the contraction is in flight
// at once (with stages for 128: absorb of one token 5.9 us, expand of 16 5.2;
// so 4.5 and 4.8, of which the weights' way takes most).
// Many tokens (500, 128 heads) take 25.9 and 18.9 us, 4.4 and 5.2 TB/s: a CTA's
// loads wait for L2, and absorb's 2048 CTAs, three an SM, are 4.5 waves run as 5.  Absorb with 256 columns a CTA: 27.0, with 64 34.3, as a
// persistent kernel with two accumulators 32.2, with the four CTAs of a token
// tile sharing its loads by multicast 32.9; expand with 64 columns 21.7.
//   warp 0     TMA loads: per 64 columns of the contraction, the tokens' box
//              (only as many rows as there are tokens: what the others' rows of
//              the accumulator hold is never stored) and the weight's: absorb's
//              weight rows run along the output (MN-major), expand's along the
//              contraction (K-major)
//   warp 1     MMAs, M=128, one accumulator in tensor memory
//   warps 2-5  absorb: copy the rope columns meanwhile; then tensor memory ->
//              bf16 -> swizzled shared memory (a stage's, free by then) ->
//              tensor stores, which clip the rows past the last token
#include <algorithm>
#include <atomic>

#include "sm103.cuh"

namespace mla {
namespace sm103 {
namespace {

constexpr int LAT = 512, ROPE = 64, HEAD = 128;   // L, P, Dn = Dv
constexpr int TM = 128;                           // tokens of a tile
constexpr int A_BYTES = TM * 128;                 // 128 tokens x 64 columns
constexpr int MAX_STAGES = 8;
constexpr int THREADS = 192;

template <bool EXPAND>
struct Cfg {
  static constexpr int K = EXPAND ? LAT : HEAD, N = EXPAND ? HEAD : LAT;
  static constexpr int MAX_NC = 128;
  static constexpr int KBLOCKS = K / 64;
  static constexpr int CTAS = EXPAND ? 2 : 4;       // an SM, at most
  static constexpr int MAX_SMEM = (EXPAND ? 112 : 75) * 1024;  // of a CTA: 2 or 3 an SM fit
};

struct HeadArgs {
  const __nv_bfloat16 *q;  // absorb: rope columns to copy, or null
  __nv_bfloat16 *q_latent;
  int T, H, nc, box_rows;
  int stages, stage_bytes, bars;          // bars: offset of the barriers
};

// MT: tiles of tokens of a CTA
template <bool EXPAND, int MT>
__global__ void __launch_bounds__(THREADS, Cfg<EXPAND>::CTAS)
    head_gemm_kernel(const __grid_constant__ CUtensorMap tm_a,
                     const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_o, const HeadArgs g) {
  using C = Cfg<EXPAND>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + g.bars);
  const uint32_t full = smem_u32(bars), empty = full + 8 * MAX_STAGES,
                 acc_full = empty + 8 * MAX_STAGES;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * MAX_STAGES + 1);
  const uint32_t stage0 = smem_u32(smem), a_bytes = uint32_t(MT * g.box_rows) * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * g.nc, t0 = blockIdx.y * TM * MT, h = blockIdx.z;
  const uint32_t cols = uint32_t(MT * g.nc);  // 64, 128 or 256

  if (threadIdx.x == 0) {
    for (int i = 0; i < g.stages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    mbar_init(acc_full, 1);
    fence_mbar_init();
    prefetch_map(&tm_a);
    prefetch_map(&tm_w);
    prefetch_map(&tm_o);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), cols);
    chain_release();  // (not before: a later kernel's CTA could take the columns and wait for us)
  }
  if (warp == 0 && lane == 0) {
    // the weights on their way to L2 while the kernels before this one finish
    for (int k = 0; k < C::K; k += 64) {
      if (EXPAND)
        prefetch_2d(&tm_w, k, h * 2 * HEAD + HEAD + n0);
      else
        for (int j = 0; j < g.nc; j += 64) prefetch_2d(&tm_w, n0 + j, h * 2 * HEAD + k);
    }
  }
  chain_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t bytes = uint32_t((MT * g.box_rows + g.nc) * 128);
      int st = 0;
      uint32_t parity = 1;
      for (int kb = 0; kb < C::KBLOCKS; ++kb) {
        if (!mbar_wait(empty + 8 * st, parity)) break;
        const uint32_t a = stage0 + st * g.stage_bytes, w = a + a_bytes, bar = full + 8 * st;
        mbar_expect_tx(bar, bytes);
        if (EXPAND) {
          tma_load_2d(w, &tm_w, bar, kb * 64, h * 2 * HEAD + HEAD + n0);  // NC rows
        } else {
          for (int j = 0; j < g.nc / 64; ++j)  // 64 rows of the contraction, 64 columns
            tma_load_2d(w + j * 8192, &tm_w, bar, n0 + j * 64, h * 2 * HEAD + kb * 64);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
          tma_load_2d(a + m * A_BYTES, &tm_a, bar,
                      (EXPAND ? h * LAT : h * (HEAD + ROPE)) + kb * 64, t0 + m * TM);
        if (++st == g.stages) {
          st = 0;
          parity ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_f16kind(TM, g.nc, false, !EXPAND, true);
      int st = 0;
      uint32_t parity = 0;
      for (int kb = 0; kb < C::KBLOCKS; ++kb) {
        if (!mbar_wait(full + 8 * st, parity)) break;
        tc_fence_after();
        // (rows of A from box_rows on are whatever follows it)
        const uint32_t a = stage0 + st * g.stage_bytes, w = a + a_bytes;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_bf16(tmem + m * g.nc, desc_kmajor_sw128(a + m * A_BYTES + ks * 32),
                     EXPAND ? desc_kmajor_sw128(w + ks * 32)
                            : desc_mnmajor_sw128(w + ks * 2048, 8192),
                     idesc, (kb | ks) != 0);
        mma_commit(empty + 8 * st);
        if (++st == g.stages) {
          st = 0;
          parity ^= 1;
        }
      }
      mma_commit(acc_full);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;  // tensor-memory lanes 32*quarter .. +31
    if (!EXPAND && g.q && n0 == 0) {
      // rope columns: 8 lanes a row of 128 bytes
      const int tid = (warp - 2) * 32 + lane;
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = t0 + i * 16 + (tid >> 3);
        if (t < g.T)
          v[i] = *reinterpret_cast<const uint4 *>(
              g.q + (int64_t(t) * g.H + h) * (HEAD + ROPE) + HEAD + (tid & 7) * 8);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = t0 + i * 16 + (tid >> 3);
        if (t < g.T)
          *reinterpret_cast<uint4 *>(g.q_latent + (int64_t(t) * g.H + h) * (LAT + ROPE) + LAT +
                                     (tid & 7) * 8) = v[i];
      }
    }
    const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full, 0));
    tc_fence_after();
    for (int m = 0; ok && m < MT; ++m) {
      const int t = t0 + m * TM + quarter * 32;
      if (t >= g.T) break;
      // every load has been consumed: the stages are free.  4 KB a piece of 32
      // rows x 64 columns, a warp's pieces behind each other.
      const uint32_t stg = stage0 + (m * 4 + quarter) * (C::MAX_NC / 64) * 4096;
#pragma unroll 1
      for (int j = 0; j < g.nc / 64; ++j) {
        uint32_t lo[32], hi[32];
        const uint32_t src = tmem + (uint32_t(quarter * 32) << 16) + m * g.nc + j * 64;
        tmem_ld32(src, lo);
        tmem_ld32(src + 32, hi);
        tmem_wait_ld();
        const uint32_t row = stg + j * 4096 + lane * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t *x = c < 4 ? lo + 8 * c : hi + 8 * (c - 4);
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = pack_bf16(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
          st_shared_v4(row + ((c ^ (lane & 7)) << 4), make_uint4(v[0], v[1], v[2], v[3]));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tm_o, stg + j * 4096, (EXPAND ? h * HEAD : h * (LAT + ROPE)) + n0 + j * 64,
                       t);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, cols);
}

template <bool EXPAND, int MT>
int launch_heads(const CUtensorMap &ta, const CUtensorMap &tw, const CUtensorMap &to, HeadArgs g,
                 cudaStream_t s) {
  using C = Cfg<EXPAND>;
  constexpr int MAX_DEV = 64;
  static std::atomic<int> ready[MAX_DEV];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEV) return MLA_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(head_gemm_kernel<EXPAND, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::MAX_SMEM) != cudaSuccess)
      return MLA_ERR_CUDA;
    ready[dev].store(1, std::memory_order_release);
  }
  // As many stages as there are blocks of the contraction, if they fit.  The
  // rows behind a short box of A, which its MMAs read, and the epilogue's 32
  // rows x 64 columns a warp stay within the stages or the room behind them.
  constexpr int BARS = 8 * (2 * MAX_STAGES + 2);
  g.stage_bytes = (MT * g.box_rows + g.nc) * 128;
  g.stages = std::min(C::KBLOCKS, (C::MAX_SMEM - 1024 - BARS) / g.stage_bytes);
  const int warps = MT * std::min(4, (g.box_rows + 31) / 32);  // pieces of the epilogue
  g.bars = std::max({g.stages * g.stage_bytes, (g.stages - 1) * g.stage_bytes + A_BYTES,
                     warps * (C::MAX_NC / 64) * 4096});
  return launch_chained(head_gemm_kernel<EXPAND, MT>, dim3(C::N / g.nc, (g.T + MT * TM - 1) / (MT * TM), g.H),
                        THREADS, 1024 + g.bars + BARS, 1, s,
                        EXPAND ? "expand_kernel" : "absorb_kernel", ta, tw, to, g);
}

// Columns of a CTA.
int pick_nc(int T, int H, int n) {
  const int64_t tiles = int64_t((T + TM - 1) / TM) * H;
  return tiles * (n / 128) < 2 * num_sms() ? 64 : 128;
}

}  // namespace
}  // namespace sm103

int launch_absorb_tc(const mla_dims_t &d, const void *q, int T, const void *w, int rope_columns,
                     void *q_latent, cudaStream_t s) {
  using namespace sm103;
  const int H = d.num_heads, QK = HEAD + ROPE, LP = LAT + ROPE;
  HeadArgs g{rope_columns ? static_cast<const __nv_bfloat16 *>(q) : nullptr,
             static_cast<__nv_bfloat16 *>(q_latent), T, H, pick_nc(T, H, LAT),
             std::min(TM, (T + 7) / 8 * 8)};
  CUtensorMap ta, tw, to;
  if (!make_tmap_2d_16(&ta, false, q, uint64_t(H) * QK, T, uint64_t(H) * QK * 2, 64, g.box_rows,
                       true) ||
      !make_tmap_2d_16(&tw, false, w, LAT, uint64_t(H) * 2 * HEAD, LAT * 2, 64, 64, true) ||
      !make_tmap_2d_16(&to, false, q_latent, uint64_t(H) * LP, T, uint64_t(H) * LP * 2, 64, 32,
                       true))
    return MLA_ERR_CUDA;
  return launch_heads<false, 1>(ta, tw, to, g, s);
}

int launch_expand_tc(const mla_dims_t &d, const void *o_latent, int T, const void *w, void *out,
                     cudaStream_t s) {
  using namespace sm103;
  const int H = d.num_heads;
  // two tiles of tokens a CTA where one each would not fit the GPU at once: the
  // weights come once for both (500 tokens 20.2 -> 18.7 us, 1000 36.0 -> 32.8;
  // absorb, whose contraction is short, gains nothing: 26.4 -> 27.4)
  const int nc = pick_nc(T, H, HEAD);
  const int64_t tiles = int64_t((T + TM - 1) / TM) * H;
  const bool two = nc == 128 && T > TM && tiles > Cfg<true>::CTAS * num_sms();
  HeadArgs g{nullptr, nullptr, T, H, nc, std::min(TM, (T + 7) / 8 * 8)};
  CUtensorMap ta, tw, to;
  if (!make_tmap_2d_16(&ta, false, o_latent, uint64_t(H) * LAT, T, uint64_t(H) * LAT * 2, 64,
                       g.box_rows, true) ||
      !make_tmap_2d_16(&tw, false, w, LAT, uint64_t(H) * 2 * HEAD, LAT * 2, 64, g.nc, true) ||
      !make_tmap_2d_16(&to, false, out, uint64_t(H) * HEAD, T, uint64_t(H) * HEAD * 2, 64, 32,
                       true))
    return MLA_ERR_CUDA;
  return two ? launch_heads<true, 2>(ta, tw, to, g, s) : launch_heads<true, 1>(ta, tw, to, g, s);
}

int heads_take_errors() { return sm103::take_error_flags_here(); }

}  // namespace mla
