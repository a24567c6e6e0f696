// Trees of drafted tokens around the attention: what each node sees and where
// it stands (mla_tree_layout), and the cache rows of the nodes that were kept
// moved behind the cached tokens (mla_commit_tree).
//
//   mask[t]      = bit t | mask[parent]            (as an index of its sequence)
//   positions[t] = seq_len - n + depth
//   cache[base + d] = cache[base + path[d]],  base = seq_len - n, d < kept
//
// Layout: a few hundred bytes a sequence, so it is bound by a launch and its
// dependent loads (locations, parents).  A block has a sequence's parents in
// shared memory and each thread walks up from a node of its own; ancestors
// come in falling order, so one word of the mask is held at a time.  A walk is as long
// as its node is deep: nodes from LIMIT on have no parent, which bounds a call
// that is no tree anybody drafts.
//
// Commit: every moved row is read and written once in every layer; all layers
// go in one launch, their addresses in its parameters.  A path's indices are at
// least their places in it (path[d] >= d: a parent comes before its children),
// so rows only move down, and a thread that moves its 16-byte column of all
// rows in the path's order, or reads several ahead, never overwrites what it
// has still to read.
#include "common.cuh"

namespace mla {
namespace {

constexpr int LAYOUT_THREADS = 128, STAGED = 1024;  // parents held in shared memory
constexpr int LIMIT = 16384;

__global__ void __launch_bounds__(LAYOUT_THREADS)
    tree_layout_kernel(const int32_t *parents, const int32_t *qsl, const int32_t *seq_lens, int T,
                       int words, uint64_t *mask, int32_t *positions, int32_t *status) {
  __shared__ int staged[STAGED];
  const int r = blockIdx.x;
  chain_release();
  chain_wait();
  const int q0 = min(max(__ldg(qsl + r), 0), T), q1 = min(__ldg(qsl + r + 1), T);
  const int n = q1 - q0;
  if (n <= 0) return;
  const int len = seq_lens ? max(__ldg(seq_lens + r), 0) : 0;
  bool bad = n > LIMIT || n > 64 * int64_t(words);
  // a parent that is no earlier node of the sequence counts as none
  auto fetch = [&](int i) {
    const int p = __ldg(parents + q0 + i);
    if (p >= -1 && p < i && i < LIMIT) return p;
    bad = true;
    return -1;
  };
  for (int i = threadIdx.x; i < min(n, STAGED); i += LAYOUT_THREADS) staged[i] = fetch(i);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += LAYOUT_THREADS) {
    uint64_t *row = mask + int64_t(q0 + i) * words;
    int depth = -1, w = words;  // words from w on are written
    uint64_t v = 0;
    for (int j = i; j >= 0; j = j < STAGED ? staged[j] : fetch(j)) {
      ++depth;
      const int wj = j >> 6;
      if (wj >= words) continue;
      if (wj != w) {
        if (w < words) row[w] = v;
        for (int k = w - 1; k > wj; --k) row[k] = 0;
        w = wj;
        v = 0;
      }
      v |= uint64_t(1) << (j & 63);
    }
    if (w < words) row[w] = v;
    for (int k = w - 1; k >= 0; --k) row[k] = 0;
    if (positions) positions[q0 + i] = len - n + depth;
  }
  if (bad && status) atomicOr(status, MLA_STATUS_BAD_TREE);
}

// ---- commit -----------------------------------------------------------------
constexpr int COMMIT_THREADS = 256, COMMIT_LAYERS = 256;  // layers of a launch

struct CommitArgs {
  const int32_t *path, *kept, *qsl, *seq_lens, *block_table;
  int32_t *new_lens, *status;
  int T, path_ld, bs, num_blocks, bt_stride, pieces, layers, group;
  uint4 *cache[COMMIT_LAYERS];
};

__global__ void __launch_bounds__(COMMIT_THREADS)
    commit_kernel(const __grid_constant__ CommitArgs a) {
  // rows to move, in the path's order: from, to
  __shared__ int64_t src[COMMIT_THREADS], dst[COMMIT_THREADS];
  __shared__ int moves_of[COMMIT_THREADS / 32];
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  chain_release();
  chain_wait();
  const int q0 = min(max(__ldg(a.qsl + r), 0), a.T), q1 = min(__ldg(a.qsl + r + 1), a.T);
  const int n = max(q1 - q0, 0), asked = __ldg(a.kept + r);
  const int kept = max(0, min(asked, min(n, a.path_ld)));
  const int base = max(__ldg(a.seq_lens + r), 0) - n;
  const bool first = blockIdx.y == 0;
  int bad = asked != kept ? MLA_STATUS_BAD_TREE : 0;
  if (first && tid == 0 && a.new_lens) a.new_lens[r] = max(0, base + kept);
  const int32_t *bt = a.block_table + int64_t(r) * a.bt_stride;
  auto row_of = [&](int j) -> int64_t {
    const int b = j / a.bs, blk = b < a.bt_stride ? __ldg(bt + b) : -1;
    if (blk >= 0 && blk < a.num_blocks) return int64_t(blk) * a.bs + (j - b * a.bs);
    bad |= MLA_STATUS_BAD_BLOCK;
    return -1;
  };
  const int l0 = blockIdx.y * a.group, nl = min(a.group, a.layers - l0);
  for (int d0 = 0; d0 < kept; d0 += COMMIT_THREADS) {
    const int d = d0 + tid;
    int64_t from = -1, to = -1;
    if (d < kept) {
      const int at = __ldg(a.path + int64_t(r) * a.path_ld + d);
      if (at < d || at >= n) {
        bad |= MLA_STATUS_BAD_TREE;
      } else if (at > d && base + d >= 0) {
        from = row_of(base + at);
        to = row_of(base + d);
      }
    }
    const bool move = from >= 0 && to >= 0;
    const uint32_t m = __ballot_sync(0xffffffffu, move);
    if (lane == 0) moves_of[warp] = __popc(m);
    __syncthreads();
    int before = 0, moves = 0;
#pragma unroll
    for (int i = 0; i < COMMIT_THREADS / 32; ++i) {
      if (i < warp) before += moves_of[i];
      moves += moves_of[i];
    }
    if (move) {
      const int k = before + __popc(m & ((1u << lane) - 1));
      src[k] = from;
      dst[k] = to;
    }
    __syncthreads();
    for (int x = tid; x < nl * a.pieces; x += COMMIT_THREADS) {
      const int l = x / a.pieces, c = x - l * a.pieces;
      uint4 *cache = a.cache[l0 + l] + c;
      constexpr int U = 8;
      for (int k = 0; k < moves; k += U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k + u < moves) v[u] = cache[src[k + u] * a.pieces];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k + u < moves) cache[dst[k + u] * a.pieces] = v[u];
      }
    }
    __syncthreads();
  }
  if (bad && first && a.status) atomicOr(a.status, bad);
}

}  // namespace

int launch_tree_layout(const int32_t *parents, const int32_t *qsl, const int32_t *seq_lens, int T,
                       int R, int words, uint64_t *mask, int32_t *positions, int32_t *status,
                       cudaStream_t s) {
  return launch_chained(tree_layout_kernel, R, LAYOUT_THREADS, 0, 1, s, "tree_layout_kernel",
                        parents, qsl, seq_lens, T, words, mask, positions, status);
}

int launch_commit(const mla_dims_t &d, const int32_t *path, int path_ld, const int32_t *kept, int T,
                  int R, const int32_t *qsl, const int32_t *seq_lens, void *const *caches,
                  int layers, int num_blocks, const int32_t *block_table, int bt_stride,
                  int32_t *new_lens, int32_t *status, cudaStream_t s) {
  CommitArgs a{path, kept, qsl, seq_lens, block_table, new_lens, status, T, path_ld, d.block_size,
               num_blocks, bt_stride,
               (d.kv_lora_rank + d.qk_rope_dim) * elem_bytes(d.dtype) / 16, 0, 0, {}};
  for (int l0 = 0; l0 == 0 || l0 < layers; l0 += COMMIT_LAYERS) {  // (lengths without layers too)
    a.layers = layers - l0 < COMMIT_LAYERS ? layers - l0 : COMMIT_LAYERS;
    for (int l = 0; l < a.layers; ++l) a.cache[l] = static_cast<uint4 *>(caches[l0 + l]);
    // Layers of a block: one while the blocks of all sequences and layers fit the
    // SMs at once, then as many as keep them there.
    const int64_t fit = 4 * num_sms();
    a.group = int((int64_t(R) * a.layers + fit - 1) / fit);
    if (a.group > a.layers) a.group = a.layers;
    if (a.group < 1) a.group = 1;
    const dim3 grid(R, a.layers ? (a.layers + a.group - 1) / a.group : 1);
    const int rc = launch_chained(commit_kernel, grid, COMMIT_THREADS, 0, 1, s, "commit_kernel", a);
    if (rc) return rc;
    a.new_lens = nullptr;  // the first launch has written them
  }
  return MLA_OK;
}

}  // namespace mla
