// The latent attention's join of a value over the four threads that share a
// row (host code compiles it too: the order of its accesses can be run there).
#pragma once

#ifdef __CUDACC__
#define MLA_JOIN_FN __device__ __forceinline__
#else
#define MLA_JOIN_FN inline
#endif

namespace mla {

// Threads tid, tid ^ 64, tid ^ 128 and tid ^ 192 of THREADS share a row.  Each
// writes its value, passes one barrier of all THREADS, and reads the others'.
//
// A thread that has left a join's barrier may write the next join's value while
// another has still to read this one's; it can write the one after that only
// behind the next barrier, which the other reaches when it has read.  So one
// barrier a join is enough as long as successive joins, whatever they join,
// take turns between two buffers: this object has all of a thread's joins, and
// counts them.
template <int THREADS>
struct RowJoin {
  float *buffers;  // [2][THREADS]
  int tid, at = 0;
  MLA_JOIN_FN RowJoin(float *b, int t) : buffers(b), tid(t) {}
  template <typename Barrier, typename F>
  MLA_JOIN_FN float operator()(float v, Barrier barrier, F f) {
    float *x = buffers + at;
    at ^= THREADS;
    x[tid] = v;
    barrier();
    return f(f(v, x[tid ^ 64]), f(x[tid ^ 128], x[tid ^ 192]));
  }
};

}  // namespace mla
