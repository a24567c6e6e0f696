// Verification of drafted tokens (mla_verify_tree): which nodes of a sequence's
// tree the target keeps, and the token that follows them.
//
// From the root on, at a node with target row p, its children c in index order:
//   with draft rows   r = p at first; kept when u_c q(x_c) < r(x_c); else
//                     r <- max(r - q, 0) / (its sum).  So r is always
//                     max(p - t q, 0) / S, S the sum of max(p - t q, 0), with t =
//                     0, S = 1 at first, t = 1 after a rejection and t <- t + S
//                     after each further one: a rejection costs one sum over the
//                     row, and nothing is stored or divided.
//   without           kept when u_c S < p(x_c), S = 1 at first and then the sum
//                     of p without the tokens rejected before.
//   greedy            kept when x_c is the row's largest value.
// Then the next token: the first v with r(0) + .. + r(v) > u_next S.
// (Leviathan, Kalman, Matias 2023 for one child; with several the tokens keep
// the target's distribution when each child was drawn from its parent's q.)
//
// The results are whole numbers that have to be the same whatever the order of
// sums, and a vocabulary's cumulated float32 sum is off by more than a token's
// share.  So a value is rounded to units of 2^-45, as two integers (left_units.h:
// what adding 2, and then 1.5 * 2^-22, leaves in a float32's low bits), and sums are
// sums of integers: exact, in any order, and the same at every level of the search
// for the next token.  (Pairs of float32 with 64-bit floating point for the walk,
// which has a 64th of float32's rate here, took 22 us for a chain of 5 over
// 32000 tokens, 149 for 64 trees of 16 over 131072 and 58 for 24 of up to 21 over
// 100003 in bf16; this 5.9, 50 and 12.  With one step less for p - t q, which is then
// off by up to 2^-25 where the grid's step ties, 5.7 and 46.)
//
// Only the rows where a child was rejected and the last node's row are read,
// one row at a time as each depends on the walk: a call of few sequences is
// bound by latency (of 11500 clocks for a chain: 3100 to the gathered values,
// 2500 for the walk, 2700 for the row, 1400 for the cluster's sums, 1500 for the
// next token; much of each is code fetched for the first time), one of many by
// its sequence with the most rejections: 64 trees read 119 rows, 20 us of HBM,
// but one of them 11, each some 9000 clocks once the others are done (2200 for the
// walk, 5500 for the row, 1200 for the sums).  (More bytes on their way, by a ring
// in shared memory or by prefetches, did not shorten that.)  A cluster of 2 to 8 CTAs takes a sequence; each walks the tree
// by itself (the same numbers, the same steps) over values gathered at the start,
// sums its part of a row, and tells the others through distributed shared memory.
// For the next token the sums of CTAs, of warps, then of 32 lanes' 16-byte pieces
// are searched by one warp of one CTA.  Where a warp's part of a row is four
// pieces a lane or less it stays in registers for the sums that follow at the
// same node.
#include <type_traits>

#include "left_units.h"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr int MAX_WARPS = 32;
constexpr int NODES = 1024;  // of a sequence
constexpr int MAX_CLUSTER = 8;
constexpr int U = 4;         // pieces a lane has in flight
constexpr uint64_t NEVER = ~uint64_t(0);
enum Mode { kDraft, kPoint, kGreedy };

struct VerifyArgs {
  const void *p, *q;
  int64_t p_ld, q_ld;
  const int32_t *tokens, *parents, *qsl;
  const float *u, *u_next;
  int32_t *path, *kept, *next, *status;
  int T, V, path_ld, cluster_log2, warps_log2;
};

// A fraction in units of 2^-64, and its part of a sum, rounded down.  (By
// conversions of 32 bits: those of 64 are slow.)
__device__ __forceinline__ uint64_t fraction(float x) {  // 0 <= x < 1, in 2^-64
  const float y = x * 4294967296.f;
  const uint32_t hi = __float2uint_rz(y);
  const uint32_t lo = __float2uint_rz(__fsub_rn(y, truncf(y)) * 4294967296.f);
  return uint64_t(hi) << 32 | lo;
}
__device__ __forceinline__ int64_t part(uint64_t x, int64_t v) {
  return int64_t(__umul64hi(x, uint64_t(v)));
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {  // by 22, 22 and 20 bits
  const uint32_t a = __reduce_add_sync(0xffffffffu, uint32_t(v) & 0x3fffff);
  const uint32_t b = __reduce_add_sync(0xffffffffu, uint32_t(v >> 22) & 0x3fffff);
  const int c = __reduce_add_sync(0xffffffffu, int(v >> 44));
  return int64_t(a) + (int64_t(b) << 22) + (int64_t(c) << 44);
}
__device__ __forceinline__ int64_t warp_scan(int64_t v) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (int(threadIdx.x & 31) >= o) v += y;
  }
  return v;
}

// A row's 16-byte pieces, counted from the aligned address at or before its
// start; `head` elements of the first lie before the row.
template <typename T>
struct Pieces {
  static constexpr int N = 16 / sizeof(T);
  const T *p, *q;
  int V, head, count;
  bool same;  // q's pieces are aligned with p's
  __device__ __forceinline__ Pieces(const T *row, const T *row_q, int v) : p(row), q(row_q), V(v) {
    head = int((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    same = !row_q ||
           ((reinterpret_cast<uintptr_t>(row_q) ^ reinterpret_cast<uintptr_t>(row)) & 15) == 0;
    count = (V + head + N - 1) / N;
  }
  __device__ __forceinline__ int first(int piece) const { return piece * N - head; }
  // elements outside the row are zeros
  __device__ __forceinline__ static uint4 one(const T *row, int at, int V) {
    alignas(16) T e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = at + i >= 0 && at + i < V ? row[at + i] : from_f32<T>(0.f);
    return *reinterpret_cast<const uint4 *>(e);
  }
  // Do steps s0 .. s1 - 1 reach over a row's ends, or does q lie otherwise than p?
  __device__ __forceinline__ bool odd(int s0, int s1) const {
    return first(s0 * 32) < 0 || first(s1 * 32) > V || !same;
  }
  // this lane's piece of step s
  template <bool Q>
  __device__ __forceinline__ void load(int s, bool odd, uint4 &vp, uint4 &vq) const {
    const int e = first(s * 32 + int(threadIdx.x & 31));
    const bool whole = unsigned(e) < unsigned(max(V - N + 1, 0));
    vp = make_uint4(0, 0, 0, 0);
    if (Q) vq = make_uint4(0, 0, 0, 0);
    if (whole) vp = __ldg(reinterpret_cast<const uint4 *>(p + e));
    if (Q && whole && !odd) vq = __ldg(reinterpret_cast<const uint4 *>(q + e));
    if (odd && e < V) {
      if (!whole) vp = one(p, e, V);
      if (Q) vq = one(q, e, V);
    }
  }
  __device__ __forceinline__ static float get(const uint4 &v, int i) {
    return to_f32(reinterpret_cast<const T *>(&v)[i]);
  }
};

struct Shared {
  // of a node: u q (or u) as a fraction; p and q of its token in its parent's rows
  uint64_t uq[NODES];  // (NEVER: 1 or more, which no part of a sum exceeds)
  float p[NODES], q[NODES];
  int token[NODES];
  int16_t parent[NODES], path[NODES];
  int16_t out[NODES];           // nodes whose tokens are taken out of the row
  uint8_t first[NODES];         // whether it is kept as its parent's first child
  int64_t warp[MAX_WARPS];      // sums of warps; greedy: largest value and place
  int64_t cta[2][MAX_CLUSTER];  // the same of the cluster's CTAs
  uint64_t bar[2];              // their arrival
  // what the walk asks of the row, and then of the search
  Two t;
  int cur, kept, finish, gone, minus_q;
  int64_t border;
  int owner;
};

// Stores 8 bytes in a CTA of the cluster and counts them on an mbarrier there.
__device__ __forceinline__ void st_async(uint32_t addr, int64_t v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                   addr),
               "l"(v), "r"(bar)
               : "memory");
}

// A float's order as an unsigned integer's; 0 for NaN and -infinity.
__device__ __forceinline__ uint32_t order_of(float v) {
  if (!(v > neg_inf())) return 0;
  const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <typename T, int MODE>
__global__ void __launch_bounds__(1024, 1) verify_kernel(const VerifyArgs a) {
  using sm103::cluster_arrive;
  using sm103::cluster_wait;
  using sm103::mapa_shared;
  using sm103::mbar_wait;
  using sm103::smem_u32;
  constexpr int N = Pieces<T>::N;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads >> 5;
  const int C = 1 << a.cluster_log2, rank = int(blockIdx.x) & (C - 1);
  const int r = int(blockIdx.x >> a.cluster_log2);
  if (tid == 0) {
    sm103::mbar_init(smem_u32(&sh.bar[0]), 1);
    sm103::mbar_init(smem_u32(&sh.bar[1]), 1);
    sm103::fence_mbar_init();
  }
  cluster_arrive();  // (its wait comes before any write to another CTA)
  chain_release();
  chain_wait();
  const int q0 = min(max(__ldg(a.qsl + r), 0), a.T), q1 = min(__ldg(a.qsl + r + 1), a.T);
  const int n = max(q1 - q0, 0), nodes = min(n, NODES), depth = min(a.path_ld, nodes);
  const T *P = static_cast<const T *>(a.p) + int64_t(q0) * a.p_ld;
  const T *Q = MODE == kDraft ? static_cast<const T *>(a.q) + int64_t(q0) * a.q_ld : nullptr;
  const float u_next = MODE != kGreedy ? __ldg(a.u_next + r) : 0.f;
  bool bad = n > nodes;
  for (int i = tid; i < nodes; i += threads) {
    int up = __ldg(a.parents + q0 + i);
    const int x = __ldg(a.tokens + q0 + i);
    const float u = MODE != kGreedy ? __ldg(a.u + q0 + i) : 0.f;
    if (up < -1 || up >= i) {
      bad = true;
      up = -1;
    }
    if (i > 0 && up >= 0 && (x < 0 || x >= a.V)) {
      bad = true;
      up = -1;  // nobody's child
    }
    sh.parent[i] = int16_t(up);
    sh.token[i] = x;
    if (MODE != kGreedy && i > 0 && up >= 0) {
      const float p = to_f32(P[up * a.p_ld + x]);
      const float q = MODE == kDraft ? to_f32(Q[up * a.q_ld + x]) : 1.f;
      const float y = __fmul_rn(u, q), rest = __fmaf_rn(u, q, -y);
      sh.p[i] = p;
      sh.q[i] = q;
      sh.first[i] = y < p || (y == p && rest < 0.f);  // u q < p, exactly
      sh.uq[i] = y < 1.f || (y == 1.f && rest < 0.f)
                     ? (y < 1.f ? fraction(y) : 0) +
                           uint64_t(__float2ll_rn(rest * 18446744073709551616.f))
                     : NEVER;
    }
  }
  if (bad && rank == 0 && a.status) atomicOr(a.status, MLA_STATUS_BAD_TREE);
  if (tid == 0) sh.path[0] = 0;
  __syncthreads();
  cluster_wait();

  // the first child of cur behind node `after`, or -1 (by a whole warp)
  auto next_child = [&](int cur, int after) {
    for (int i0 = (after + 1) & ~31; i0 < nodes; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t m =
          __ballot_sync(0xffffffffu, i > after && i < nodes && sh.parent[i] == cur);
      if (m) return i0 + __ffs(int(m)) - 1;
    }
    return -1;
  };
  // Warp 0: tells every CTA of the cluster this one's value, and returns CTA
  // `lane`'s (none: for the lanes without one).  Two barriers take turns: a CTA
  // that is a pass ahead writes to the other one, and cannot be two ahead, as it
  // needs this one's value.  (A wait that gave up is the last: what follows
  // is not valid, and short.)
  int pass = 0;
  bool lost = false;
  auto exchange = [&](int64_t v, int64_t none) {
    if (lost) return none;
    const int b = pass & 1;
    const uint32_t bar = smem_u32(&sh.bar[b]);
    if (lane == 0) sm103::mbar_expect_tx(bar, uint32_t(C) * 8);
    __syncwarp();
    if (lane < C)
      st_async(mapa_shared(smem_u32(&sh.cta[b][rank]), lane), v, mapa_shared(bar, lane));
    lost = !__all_sync(0xffffffffu, mbar_wait(bar, (pass >> 1) & 1));
    ++pass;
    return !lost && lane < C ? *const_cast<volatile int64_t *>(&sh.cta[b][lane]) : none;
  };
  // this CTA's and this warp's steps of 32 pieces
  auto steps_of = [&](const Pieces<T> &x, int &s0, int &s1) {
    const int steps = (x.count + 31) / 32, per_cta = (steps + C - 1) >> a.cluster_log2;
    const int c0 = min(rank * per_cta, steps), c1 = min(c0 + per_cta, steps);
    const int per_warp = (c1 - c0 + warps - 1) >> a.warps_log2;
    s0 = min(c0 + warp * per_warp, c1);
    s1 = min(s0 + per_warp, c1);
  };
  auto store_path = [&](int kept) {
    for (int d = tid; d < a.path_ld; d += threads)
      a.path[int64_t(r) * a.path_ld + d] = d < kept ? sh.path[d] : -1;
    if (tid == 0) a.kept[r] = kept;
  };

  if constexpr (MODE == kGreedy) {
    int cur = 0, kept = nodes > 0, best = -1;
    while (kept > 0) {
      const Pieces<T> x(P + cur * a.p_ld, nullptr, a.V);
      int s0, s1;
      steps_of(x, s0, s1);
      uint32_t top = 0;
      int at = 0x7fffffff;
      const bool odd = x.odd(s0, s1);
      for (int s = s0; s < s1; s += U) {
        uint4 v[U], none;
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (s + k < s1) x.template load<false>(s + k, odd, v[k], none);
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (s + k < s1) {
            const int e = x.first((s + k) * 32 + lane);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const uint32_t o = order_of(x.get(v[k], i));
              if (o > top && e + i >= 0 && e + i < a.V) {  // (rising indices: ties stay)
                top = o;
                at = e + i;
              }
            }
          }
      }
      // the largest value and the lowest of its places
      auto join = [&](uint32_t t, int i) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, t);
        const uint32_t f = __reduce_min_sync(0xffffffffu, t == m ? uint32_t(i) : 0x7fffffffu);
        return int64_t(uint64_t(m) << 32 | f);
      };
      int64_t v = join(top, at);
      if (lane == 0) sh.warp[warp] = v;
      __syncthreads();
      if (warp == 0) {
        v = lane < warps ? sh.warp[lane] : 0x7fffffff;
        v = join(uint32_t(uint64_t(v) >> 32), int(v));
        v = exchange(v, 0x7fffffff);
        v = join(uint32_t(uint64_t(v) >> 32), int(v));
        if (lane == 0) sh.border = v;
      }
      __syncthreads();
      v = sh.border;
      best = v >> 32 ? int(v) : 0;  // (a row of nothing but -inf and NaN)
      int child = -1;
      if (kept < depth) {
        child = next_child(cur, cur);
        while (child >= 0 && sh.token[child] != best) child = next_child(cur, child);
      }
      if (child < 0) break;
      if (tid == 0) sh.path[kept] = int16_t(child);
      ++kept;
      cur = child;
    }
    if (rank == 0) {
      __syncthreads();
      store_path(kept);
      if (tid == 0) a.next[r] = best;
    }
    return;
  } else {
    if (nodes == 0) {
      if (rank == 0) {
        store_path(0);
        if (tid == 0) a.next[r] = -1;
      }
      return;
    }
    // Which of a lane's values of steps s .. s + U - 1 are tokens taken out: N
    // bits a step.
    auto taken = [&](const Pieces<T> &x, int s) {
      uint32_t m = 0;
      for (int i = 0; i < sh.gone; ++i) {
        const int e = sh.token[sh.out[i]] + x.head, at = e / (32 * N) - s;
        if (at >= 0 && at < U && (e / N & 31) == lane) m |= 1u << (at * N + e % N);
      }
      return m;
    };
    // the walk's state, the same in all lanes of warp 0
    int cur = 0, after = 0, kept = 1, tried = 0;
    uint64_t t = 0;    // in units; below 2^64 for 1023 sums below 512
    Two t_two{0.f, 0.f};
    int64_t mass = 0;  // of what is left, from the first rejection on
    bool told = true;  // it is of what is left now
    uint4 vp[U], vq[U];
    int held = -1;  // the node whose values vp, vq hold
    for (;;) {
      if (warp == 0) {
        int finish = 0;
        for (;;) {
          const int c = kept < depth ? next_child(cur, after) : -1;
          if (c < 0) {
            finish = 1;
            break;
          }
          if (!told) break;  // the children behind a rejected one need the sum
          bool keep;
          int64_t w = 0;
          if (tried == 0) {  // S = 1, r = p
            keep = sh.first[c];
          } else {
            if (MODE == kDraft) {
              w = left_of<true>(t_two, sh.p[c], sh.q[c]);
            } else {
              const int x = sh.token[c];
              bool again = false;
              for (int i = lane; i < tried; i += 32) again = again || sh.token[sh.out[i]] == x;
              w = __any_sync(0xffffffffu, again) ? 0 : left_of<false>(Two(), sh.p[c], 0.f);
            }
            keep = sh.uq[c] != NEVER && part(sh.uq[c], mass) < w;
          }
          if (keep) {
            if (lane == 0) sh.path[kept] = int16_t(c);
            ++kept;
            cur = after = c;
            tried = 0;
            t = 0;
            t_two = Two{0.f, 0.f};
            continue;
          }
          after = c;
          if (MODE == kDraft) {
            t = tried == 0 ? ONE : t + mass;
            t_two = number(t);
            ++tried;
            told = false;
          } else if (tried == 0 || w > 0) {
            if (lane == 0) sh.out[tried] = int16_t(c);
            if (tried == 0)
              told = false;
            else
              mass -= w;
            ++tried;
            __syncwarp();
          }
        }
        if (lane == 0) {
          sh.cur = cur;
          sh.kept = kept;
          sh.finish = finish;
          sh.gone = MODE == kPoint ? tried : 0;
          sh.minus_q = MODE == kDraft && tried > 0;
          if (MODE == kDraft) sh.t = t_two;
        }
      }
      __syncthreads();
      // ---- the sum of what is left of the row of sh.cur
      const int node = sh.cur, minus_q = sh.minus_q, finish = sh.finish, gone = sh.gone;
      const Two t2 = sh.t;
      const Pieces<T> x(P + node * a.p_ld, MODE == kDraft ? Q + node * a.q_ld : nullptr, a.V);
      int s0, s1;
      steps_of(x, s0, s1);
      const bool fits = s1 - s0 <= U;
      bool out = false;  // a token that was taken out is in this warp's part
      int64_t sum = 0;
      if (MODE == kPoint) {
        const int e0 = x.first(s0 * 32), e1 = x.first(s1 * 32);
        for (int i = 0; i < gone; ++i) {
          const int c = sh.out[i], t = sh.token[c];
          if (t >= e0 && t < e1) {
            if (lane == 0) sum -= left_of<false>(t2, sh.p[c], 0.f);
            out = true;
          }
        }
      }
      auto sum_row = [&](auto with_q) {
        constexpr bool Q = decltype(with_q)::value;
        const bool odd = x.odd(s0, s1);
        for (int s = s0; s < s1; s += U) {
          if (!fits || held != node) {
#pragma unroll
            for (int k = 0; k < U; ++k)
              if (s + k < s1) x.template load<Q>(s + k, odd, vp[k], vq[k]);
          }
          uint32_t hi = 0, lo = 0;  // (at most 32 values of 23 bits)
#pragma unroll
          for (int k = 0; k < U; ++k)
            if (s + k < s1) {
#pragma unroll
              for (int i = 0; i < N; ++i)
                add_left<Q>(t2, x.get(vp[k], i), x.get(vq[k], i), hi, lo);
            }
          sum += units(hi, lo);
        }
      };
      if (MODE == kDraft && minus_q)
        sum_row(std::true_type());
      else
        sum_row(std::false_type());
      held = node;
      sum = warp_sum(sum);
      if (lane == 0) sh.warp[warp] = sum;
      __syncthreads();
      if (warp == 0) {
        const int64_t of_warp = lane < warps ? sh.warp[lane] : 0;
        const int64_t of_cta = exchange(warp_sum(of_warp), 0), total = warp_sum(of_cta);
        if (!finish) {
          mass = total;
          told = true;
          continue;
        }
        if (total <= 0 && minus_q + gone > 0) {
          if (lane == 0) sh.owner = -2;  // nothing left (rounded rows): the row itself
        } else {
          // the border, and whose part it is in: the CTA, then the warp
          const int64_t border =
              total > 0 ? min(part(fraction(u_next), total), total - 1) : 0;
          const int64_t up_to = warp_scan(of_cta);
          const uint32_t over = __ballot_sync(0xffffffffu, up_to > border);
          const int owner = over ? __ffs(int(over)) - 1 : -1;
          int of = -1;
          if (owner == rank) {
            const int64_t before = __shfl_sync(0xffffffffu, up_to - of_cta, rank);
            const int64_t inc = before + warp_scan(of_warp);
            const uint32_t m = __ballot_sync(0xffffffffu, inc > border);
            of = m ? __ffs(int(m)) - 1 : warps - 1;
            const int64_t rest = border - __shfl_sync(0xffffffffu, inc - of_warp, of);
            if (lane == 0) sh.border = rest;
          } else if (owner < 0 && rank == 0 && lane == 0) {
            a.next[r] = a.V - 1;  // a row without mass
          }
          if (lane == 0) sh.owner = of;
        }
      } else if (!finish) {
        continue;
      }
      __syncthreads();
      if (sh.owner == -2) {
        if (warp == 0) {
          tried = 0;  // (no children are left: the walk comes back with the row)
          t_two = Two{0.f, 0.f};
        }
        __syncthreads();
        continue;
      }
      // ---- the next token, by the warp that has it: the step, the lane, the value
      if (warp == sh.owner) {
        int64_t border = sh.border;
        int found = -1;
        // (one step at a time, in little code, which runs once)
#pragma unroll 1
        for (int s = s0; s < s1 && found < 0; ++s) {
          uint4 wp, wq = make_uint4(0, 0, 0, 0);
          if (MODE == kDraft && minus_q)
            x.template load<true>(s, x.odd(s0, s1), wp, wq);
          else
            x.template load<false>(s, x.odd(s0, s1), wp, wq);
          const uint32_t gone_bits = MODE == kPoint && out ? taken(x, s) : 0;
          int64_t v[N], mine = 0;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            v[i] = left_of<MODE == kDraft>(t2, x.get(wp, i), x.get(wq, i));
            if (gone_bits >> i & 1) v[i] = 0;
            mine += v[i];
          }
          const int64_t inc = warp_scan(mine);
          const uint32_t hit = __ballot_sync(0xffffffffu, inc > border);
          if (hit) {
            const int e = x.first(s * 32 + lane);
            int64_t run = inc - mine;
            int here = e + N - 1;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              run += v[i];
              if (run > border) here = min(here, e + i);
            }
            found = __shfl_sync(0xffffffffu, here, __ffs(int(hit)) - 1);
          }
          border -= __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) a.next[r] = found < 0 || found >= a.V ? a.V - 1 : found;
      }
      if (rank == 0) store_path(sh.kept);
      return;
    }
  }
}

}  // namespace

int launch_verify(const void *p, int64_t p_ld, const void *q, int64_t q_ld, int dtype, int V,
                  const int32_t *tokens, const int32_t *parents, int T, int R, const int32_t *qsl,
                  const float *u, const float *u_next, int32_t *path, int path_ld, int32_t *kept,
                  int32_t *next, int32_t *status, cudaStream_t s) {
  VerifyArgs a{p, q, p_ld, q_ld, tokens, parents, qsl, u, u_next, path, kept, next, status,
               T, V, path_ld, 1, 5};
  // Clusters of 8 while four CTAs an SM are no fewer than them all, but of two at
  // least: the kernel's stores to a cluster's shared memory fault in a launch that
  // has no clusters (more than 304 sequences each on a CTA of its own).  1024 threads
  // an SM: a CTA has 32 to 8 warps, or 16 at least where 8 would have more than U
  // pieces a lane each (8 and 16: 64 trees, V 131072 55 and 49.5 us, 109 chains of 9,
  // greedy, 98294 86 and 70; 126 trees of 9, 2066 in bf16 15.7 and 20, 58 single
  // nodes, 57225 in bf16 7.4 and 10.5, 1000 trees of 5, 2066 26 and 45).
  const int sms = num_sms();
  while (2 << a.cluster_log2 <= MAX_CLUSTER && (int64_t(R) * 2 << a.cluster_log2) <= 4 * sms)
    ++a.cluster_log2;
  const int step = 32 * 16 / elem_bytes(dtype), steps = (V + step - 1) / step;
  const int fewest = steps > (8 * U << a.cluster_log2) ? 4 : 3;
  while (a.warps_log2 > fewest &&
         (int64_t(R) << a.cluster_log2) > (int64_t(sms) << (5 - a.warps_log2)))
    --a.warps_log2;
  const int threads = 32 << a.warps_log2;
  auto pick = [&](auto t) {
    using E = decltype(t);
    return !u ? verify_kernel<E, kGreedy> : q ? verify_kernel<E, kDraft> : verify_kernel<E, kPoint>;
  };
  auto *kernel = dtype == MLA_DTYPE_BF16 ? pick(__nv_bfloat16()) : pick(float());
  return launch_chained(kernel, dim3(unsigned(R) << a.cluster_log2), threads, 0,
                        1 << a.cluster_log2, s, "verify_kernel", a);
}

int verify_take_errors() { return sm103::take_error_flags_here(); }

}  // namespace mla
