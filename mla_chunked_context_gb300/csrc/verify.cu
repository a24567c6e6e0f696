// Verification of drafted tokens (mla_verify_tree): which nodes of a sequence's
// tree the target keeps, and the token that follows them.
//
// From the root on, at a node with target row p, its children c in index order:
//   with draft rows   r = p at first; kept when u_c q(x_c) < r(x_c); else
//                     r <- max(r - q, 0) / S, S the sum of max(r - q, 0).  So r
//                     = max(a p - b q, 0) always, with a = b = 1 after the first
//                     rejection and then a <- a / S, b <- b / S + 1: a rejection
//                     costs one sum over the row and nothing is stored.
//   without           kept when u_c S < p(x_c), S = 1 at first and then the sum
//                     of p without the tokens rejected before.
//   greedy            kept when x_c is the row's largest value.
// Then the next token: the first v with r(0) + .. + r(v) > u_next S.
// (Leviathan, Kalman, Matias 2023 for one child; with several the tokens keep
// the target's distribution when each child was drawn from its parent's q.)
//
// The results are whole numbers that have to be the same whatever the order of
// sums, and a vocabulary's cumulated float32 sum is off by more than a token's
// share.  So sums are pairs of float32 (48 bits; Dekker 1971, Knuth's two-sum),
// and the few scalars 64-bit.  (64-bit sums of all values would be bound by
// their rate, a 64th of float32's.)
//
// Only the rows where a child was rejected and the last node's row are read,
// one row at a time as each depends on the walk: a call of few sequences is
// bound by latency, one of many by HBM.  A cluster of up to 8 CTAs takes a
// sequence; each walks the tree by itself (the same numbers, the same steps)
// over values gathered at the start, sums its part of a row, and tells the
// others through distributed shared memory.  For the next token the sums of
// CTAs, of warps, then of 32 lanes' 16-byte pieces are searched; only the last
// warp reads its part of the row again.
#include <type_traits>

#include "sm103.cuh"

namespace mla {
namespace {

constexpr int VT = 512, VW = VT / 32;  // threads, warps
constexpr int NODES = 1024;            // of a sequence
constexpr int MAX_CLUSTER = 8;
enum Mode { kDraft, kPoint, kGreedy };

struct VerifyArgs {
  const void *p, *q;
  int64_t p_ld, q_ld;
  const int32_t *tokens, *parents, *qsl;
  const float *u, *u_next;
  int32_t *path, *kept, *next, *status;
  int T, V, path_ld, cluster;
};

// A sum in two floats, |lo| <= half a step of hi (once renormalised).
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float x_lo) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
    hi = s;
    lo = __fadd_rn(lo, __fadd_rn(e, x_lo));
  }
  __device__ __forceinline__ void renormalise() {
    const float s = __fadd_rn(hi, lo);
    lo = __fsub_rn(lo, __fsub_rn(s, hi));
    hi = s;
  }
};

__device__ __forceinline__ Sum2 warp_sum(Sum2 s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, s.hi, o), l = __shfl_xor_sync(0xffffffffu, s.lo, o);
    s.add(h, l);
    s.renormalise();
  }
  return s;
}

// What is left of a row: max(a p - b q, 0), a and b in two floats each.
struct Left {
  float ah, al, bh, bl;
  int kind;  // 0: p; 1: p - q; 2: any
  __device__ __forceinline__ static Left of(double a, double b) {
    Left l;
    l.ah = float(a);
    l.al = float(a - double(l.ah));
    l.bh = float(b);
    l.bl = float(b - double(l.bh));
    l.kind = b == 0.0 ? 0 : a == 1.0 && b == 1.0 ? 1 : 2;
    return l;
  }
};
template <int KIND>
__device__ __forceinline__ void left_of(const Left &l, float p, float q, float &hi, float &lo) {
  lo = 0.f;
  if (KIND == 0) {
    hi = fmaxf(p, 0.f);  // (0 for a NaN)
    return;
  }
  float x = p, y = q, e = 0.f;
  if (KIND == 2) {
    x = __fmul_rn(l.ah, p);
    y = __fmul_rn(l.bh, q);
    const float ex = __fmaf_rn(l.al, p, __fmaf_rn(l.ah, p, -x));
    const float ey = __fmaf_rn(l.bl, q, __fmaf_rn(l.bh, q, -y));
    e = __fsub_rn(ex, ey);
  }
  const float d = __fsub_rn(x, y), b = __fsub_rn(d, x);
  e = __fadd_rn(e, __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(y, b)));
  const bool some = __fadd_rn(d, e) > 0.f;
  hi = some ? d : 0.f;
  lo = some ? e : 0.f;
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
    same = ((reinterpret_cast<uintptr_t>(row_q) ^ reinterpret_cast<uintptr_t>(row)) & 15) == 0;
    count = (V + head + N - 1) / N;
  }
  __device__ __forceinline__ int first(int piece) const { return piece * N - head; }
  // elements outside the row are zeros
  __device__ __forceinline__ static uint4 one(const T *row, bool vector, int at, int V) {
    if (vector) return __ldg(reinterpret_cast<const uint4 *>(row + at));
    alignas(16) T e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = at + i >= 0 && at + i < V ? row[at + i] : from_f32<T>(0.f);
    return *reinterpret_cast<const uint4 *>(e);
  }
  template <bool Q>
  __device__ __forceinline__ void load(int piece, uint4 &vp, uint4 &vq) const {
    const int at = first(piece);
    const bool whole = piece < count && at >= 0 && at + N <= V;
    vp = one(p, whole, at, V);
    if (Q) vq = one(q, whole && same, at, V);
  }
  __device__ __forceinline__ static float get(const uint4 &v, int i) {
    return to_f32(reinterpret_cast<const T *>(&v)[i]);
  }
};

struct Shared {
  int parent[NODES], token[NODES], path[NODES];
  float p[NODES], q[NODES], u[NODES];  // p and q of a node's token in its parent's rows
  float hi[VW], lo[VW];                // sums of warps
  float all_hi[2][MAX_CLUSTER], all_lo[2][MAX_CLUSTER];  // of the cluster's CTAs
  int all_at[2][MAX_CLUSTER];                            // greedy: where the largest value is
  // what the walk asks of the row
  int cur, kept, finish, gone;  // gone: tokens taken out, in `out`
  double a, b;
  int out[NODES];
  int next;
};

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <typename T, int MODE>
__global__ void __launch_bounds__(VT, 2) verify_kernel(const VerifyArgs a) {
  using sm103::cluster_arrive;
  using sm103::cluster_wait;
  using sm103::mapa_shared;
  using sm103::smem_u32;
  constexpr int N = Pieces<T>::N;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.cluster;
  const int rank = int(blockIdx.x) % C, r = int(blockIdx.x) / C;
  cluster_arrive();  // (nobody writes to a CTA that has not started)
  chain_release();
  chain_wait();
  const int q0 = min(max(__ldg(a.qsl + r), 0), a.T), q1 = min(__ldg(a.qsl + r + 1), a.T);
  const int n = max(q1 - q0, 0), nodes = min(n, NODES), depth = min(a.path_ld, nodes);
  const T *P = static_cast<const T *>(a.p) + int64_t(q0) * a.p_ld;
  const T *Q = MODE == kDraft ? static_cast<const T *>(a.q) + int64_t(q0) * a.q_ld : nullptr;
  bool bad = n > nodes;
  for (int i = tid; i < nodes; i += VT) {
    int up = __ldg(a.parents + q0 + i);
    const int x = __ldg(a.tokens + q0 + i);
    if (up < -1 || up >= i) {
      bad = true;
      up = -1;
    }
    if (i > 0 && up >= 0 && (x < 0 || x >= a.V)) {
      bad = true;
      up = -1;  // nobody's child
    }
    sh.parent[i] = up;
    sh.token[i] = x;
    if (MODE != kGreedy && i > 0 && up >= 0) {
      sh.u[i] = __ldg(a.u + q0 + i);
      sh.p[i] = to_f32(P[up * a.p_ld + x]);
      if (MODE == kDraft) sh.q[i] = to_f32(Q[up * a.q_ld + x]);
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
  int pass = 0;
  // tells every CTA of the cluster this one's sum (and place)
  auto tell = [&](float hi, float lo, int at) {
    if (warp == 0 && lane < C) {
      const int b = pass & 1;
      st_cluster(mapa_shared(smem_u32(&sh.all_hi[b][rank]), lane), __float_as_uint(hi));
      st_cluster(mapa_shared(smem_u32(&sh.all_lo[b][rank]), lane), __float_as_uint(lo));
      if (MODE == kGreedy) st_cluster(mapa_shared(smem_u32(&sh.all_at[b][rank]), lane), at);
    }
    cluster_arrive();
    cluster_wait();
  };
  // this CTA's and this warp's steps of 32 pieces
  auto steps_of = [&](const Pieces<T> &x, int &s0, int &s1) {
    const int steps = (x.count + 31) / 32, per_cta = (steps + C - 1) / C;
    const int c0 = min(rank * per_cta, steps), c1 = min(c0 + per_cta, steps);
    const int per_warp = (c1 - c0 + VW - 1) / VW;
    s0 = min(c0 + warp * per_warp, c1);
    s1 = min(s0 + per_warp, c1);
  };
  // Is token v among those taken out?
  auto taken = [&](int v) {
    for (int i = 0; i < sh.gone; ++i)
      if (sh.out[i] == v) return true;
    return false;
  };

  if constexpr (MODE == kGreedy) {
    int cur = 0, kept = nodes > 0;
    int best = -1;
    while (kept > 0) {
      const Pieces<T> x(P + cur * a.p_ld, nullptr, a.V);
      int s0, s1;
      steps_of(x, s0, s1);
      float top = neg_inf();
      int at = a.V;
      constexpr int U = 4;
      for (int s = s0; s < s1; s += U) {
        uint4 v[U], none;
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (s + k < s1) x.template load<false>((s + k) * 32 + lane, v[k], none);
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (s + k < s1) {
            const int e = x.first((s + k) * 32 + lane);
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (x.get(v[k], i) > top && e + i >= 0 && e + i < a.V) {  // (rising: ties stay)
                top = x.get(v[k], i);
                at = e + i;
              }
          }
      }
      auto better = [&](float t, int i) {
        if (t > top || (t == top && i < at)) {
          top = t;
          at = i;
        }
      };
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        better(__shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, at, o));
      if (lane == 0) {
        sh.hi[warp] = top;
        sh.out[warp] = at;
      }
      __syncthreads();
      if (warp == 0) {
        top = lane < VW ? sh.hi[lane] : neg_inf();
        at = lane < VW ? sh.out[lane] : a.V;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          better(__shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, at, o));
      }
      tell(top, 0.f, at);
      top = neg_inf();
      at = a.V;
      for (int c = 0; c < C; ++c) better(sh.all_hi[pass & 1][c], sh.all_at[pass & 1][c]);
      best = at < a.V ? at : 0;  // (a row of nothing but -inf and NaN)
      ++pass;
      int child = -1;
      if (kept < depth) {
        child = next_child(cur, cur);
        while (child >= 0 && sh.token[child] != best) child = next_child(cur, child);
      }
      if (child < 0) break;
      if (tid == 0) sh.path[kept] = child;
      ++kept;
      cur = child;
    }
    if (rank == 0) {
      __syncthreads();
      for (int d = tid; d < a.path_ld; d += VT)
        a.path[int64_t(r) * a.path_ld + d] = d < kept ? sh.path[d] : -1;
      if (tid == 0) {
        a.kept[r] = kept;
        a.next[r] = best;
      }
    }
    return;
  } else {
    // the walk's state, the same in all lanes of warp 0
    int cur = 0, after = 0, kept = nodes > 0, tried = 0;
    double ca = 1.0, cb = 0.0, mass = 1.0;
    bool summed = false, told = true;  // told: `mass` is of what is left now
    // Sums what is left of the row of sh.cur: this warp's sum goes to sh.hi,
    // sh.lo, the CTAs' to sh.all_hi, sh.all_lo.
    auto row_pass = [&](auto kind, const Left &l, const Pieces<T> &x, int s0, int s1, bool out) {
      constexpr int K = decltype(kind)::value, U = 16 / N;  // (16 elements a thread in flight)
      Sum2 sum;
      for (int s = s0; s < s1; s += U) {
        uint4 vp[U], vq[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          vp[k] = vq[k] = make_uint4(0, 0, 0, 0);
          if (s + k < s1) x.template load<K != 0>((s + k) * 32 + lane, vp[k], vq[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            float hi, lo;
            left_of<K>(l, x.get(vp[k], i), x.get(vq[k], i), hi, lo);
            if (out && taken(x.first((s + k) * 32 + lane) + i)) hi = lo = 0.f;
            sum.add(hi, lo);
          }
        sum.renormalise();
      }
      return sum;
    };
    auto sum_row = [&](const Left &l, const Pieces<T> &x, int s0, int s1) {
      bool out = false;  // a token that was taken out is in this warp's part
      if (MODE == kPoint) {
        const int e0 = x.first(s0 * 32), e1 = x.first(s1 * 32);
        for (int i = 0; i < sh.gone; ++i) out = out || (sh.out[i] >= e0 && sh.out[i] < e1);
      }
      Sum2 s;
      if (MODE == kPoint || l.kind == 0)
        s = row_pass(std::integral_constant<int, 0>(), l, x, s0, s1, out);
      else if (l.kind == 1)
        s = row_pass(std::integral_constant<int, 1>(), l, x, s0, s1, false);
      else
        s = row_pass(std::integral_constant<int, 2>(), l, x, s0, s1, false);
      s = warp_sum(s);
      if (lane == 0) {
        sh.hi[warp] = s.hi;
        sh.lo[warp] = s.lo;
      }
      __syncthreads();
      if (warp == 0) {
        s.hi = lane < VW ? sh.hi[lane] : 0.f;
        s.lo = lane < VW ? sh.lo[lane] : 0.f;
        s = warp_sum(s);
      }
      tell(s.hi, s.lo, 0);
      double total = 0.0;
      if (warp == 0 || sh.finish)
        for (int c = 0; c < C; ++c)
          total += double(sh.all_hi[pass & 1][c]) + double(sh.all_lo[pass & 1][c]);
      ++pass;
      return total;
    };
    if (nodes == 0) {
      if (rank == 0) {
        for (int d = tid; d < a.path_ld; d += VT) a.path[int64_t(r) * a.path_ld + d] = -1;
        if (tid == 0) {
          a.kept[r] = 0;
          a.next[r] = -1;
        }
      }
      return;
    }
    for (;;) {
      if (warp == 0) {
        bool finish = false;
        for (;;) {
          const int c = kept < depth ? next_child(cur, after) : -1;
          if (c < 0) {
            finish = true;
            break;
          }
          if (!told) {  // the children behind a rejected one need the sum
            if (MODE == kDraft || !summed) break;
            told = true;
          }
          const int x = sh.token[c];
          double w = fmax(double(sh.p[c]), 0.0), q = 1.0;
          if (MODE == kDraft) {
            q = double(sh.q[c]);
            if (cb != 0.0) w = fmax(ca * double(sh.p[c]) - cb * q, 0.0);
          } else {
            for (int i = lane; i < tried; i += 32)
              if (sh.out[i] == x) w = -1.0;
            if (__any_sync(0xffffffffu, w < 0.0)) w = 0.0;
          }
          if (double(sh.u[c]) * q * mass < w) {
            if (lane == 0) sh.path[kept] = c;
            ++kept;
            cur = after = c;
            tried = 0;
            ca = mass = 1.0;
            cb = 0.0;
            summed = false;
            told = true;
            continue;
          }
          after = c;
          if (MODE == kDraft) {
            if (mass > 0.0) {
              ca /= mass;
              cb = cb / mass + 1.0;
            }
            told = false;
          } else {
            if (w > 0.0 || tried == 0) {
              if (lane == 0) sh.out[tried] = x;
              ++tried;
              if (summed)
                mass -= w;
              else
                told = false;
            }
            __syncwarp();
          }
        }
        if (lane == 0) {
          sh.cur = cur;
          sh.kept = kept;
          sh.finish = finish;
          sh.gone = MODE == kPoint ? tried : 0;
          sh.a = ca;
          sh.b = cb;
        }
      }
      __syncthreads();
      const int64_t at = sh.cur;
      const Pieces<T> x(P + at * a.p_ld, MODE == kDraft ? Q + at * a.q_ld : nullptr, a.V);
      int s0, s1;
      steps_of(x, s0, s1);
      Left l = Left::of(sh.a, sh.b);
      double total = sum_row(l, x, s0, s1);
      if (!sh.finish) {
        if (warp == 0) {
          mass = total;
          told = summed = true;
        }
        __syncthreads();  // sh.cur .. are read
        continue;
      }
      if (!(total > 0.0)) {  // nothing left (rounded rows): the row itself
        __syncthreads();
        l = Left::of(1.0, 0.0);
        if (tid == 0) sh.gone = 0;
        __syncthreads();
        total = sum_row(l, x, s0, s1);
      }
      // ---- the next token: the CTA, the warp, the lane, the element
      const int last = (pass - 1) & 1;
      const double border = double(__ldg(a.u_next + r)) * total;
      int owner = -1, some = 0;
      double before = 0.0, mine = 0.0;
      for (int c = 0; c < C; ++c) {
        const double v = double(sh.all_hi[last][c]) + double(sh.all_lo[last][c]);
        if (v > 0.0) some = c;
        if (c == rank) mine = before;
        before += v;
        if (owner < 0 && before > border) owner = c;
      }
      if (owner < 0) owner = some;  // the border is the sum: the last token with mass
      if (rank == owner) {
        if (warp == 0) {
          const double v = lane < VW ? double(sh.hi[lane]) + double(sh.lo[lane]) : 0.0;
          double inc = v;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
          }
          const uint32_t over = __ballot_sync(0xffffffffu, lane < VW && mine + inc > border);
          const uint32_t has = __ballot_sync(0xffffffffu, v > 0.0);
          const int w = over ? __ffs(int(over)) - 1 : has ? 31 - __clz(int(has)) : 0;
          const double up_to = __shfl_sync(0xffffffffu, mine + (inc - v), w);
          if (lane == 0) {
            sh.cur = w;
            sh.a = up_to;
          }
        }
        __syncthreads();
        if (warp == sh.cur) {
          double base = sh.a;
          int found = -1, final_some = -1;
          for (int s = s0; s < s1 && found < 0; ++s) {
            uint4 vp, vq = make_uint4(0, 0, 0, 0);
            const int piece = s * 32 + lane, e = x.first(piece);
            double v[N], sum = 0.0;
            if (MODE == kDraft && l.kind != 0)
              x.template load<true>(piece, vp, vq);
            else
              x.template load<false>(piece, vp, vq);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              float hi, lo;
              if (MODE == kPoint || l.kind == 0)
                left_of<0>(l, x.get(vp, i), 0.f, hi, lo);
              else if (l.kind == 1)
                left_of<1>(l, x.get(vp, i), x.get(vq, i), hi, lo);
              else
                left_of<2>(l, x.get(vp, i), x.get(vq, i), hi, lo);
              if (MODE == kPoint && taken(e + i)) hi = lo = 0.f;
              v[i] = double(hi) + double(lo);
              sum += v[i];
            }
            double inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const double y = __shfl_up_sync(0xffffffffu, inc, o);
              if (lane >= o) inc += y;
            }
            double run = base + (inc - sum);
            int here = -1, last_some = -1;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              run += v[i];
              if (v[i] > 0.0) {
                last_some = e + i;
                if (here < 0 && run > border) here = e + i;
              }
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, here >= 0);
            const uint32_t has = __ballot_sync(0xffffffffu, last_some >= 0);
            if (has) final_some = __shfl_sync(0xffffffffu, last_some, 31 - __clz(int(has)));
            if (hit) found = __shfl_sync(0xffffffffu, here, __ffs(int(hit)) - 1);
            base += __shfl_sync(0xffffffffu, inc, 31);
          }
          if (found < 0) found = final_some >= 0 ? final_some : a.V - 1;
          if (lane == 0) a.next[r] = found;
        }
      }
      if (rank == 0) {
        for (int d = tid; d < a.path_ld; d += VT)
          a.path[int64_t(r) * a.path_ld + d] = d < sh.kept ? sh.path[d] : -1;
        if (tid == 0) a.kept[r] = sh.kept;
      }
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
               T, V, path_ld, 1};
  // two CTAs an SM
  while (a.cluster < MAX_CLUSTER && int64_t(R) * a.cluster * 2 <= 2 * num_sms()) a.cluster *= 2;
  auto pick = [&](auto t) {
    using E = decltype(t);
    return !u ? verify_kernel<E, kGreedy> : q ? verify_kernel<E, kDraft> : verify_kernel<E, kPoint>;
  };
  auto *kernel = dtype == MLA_DTYPE_BF16 ? pick(__nv_bfloat16()) : pick(float());
  return launch_chained(kernel, dim3(unsigned(R) * unsigned(a.cluster)), VT, 0, a.cluster, s,
                        "verify_kernel", a);
}

}  // namespace mla
