// Host helpers shared by the C-ABI entry points (abi.cu, abi_decode.cu):
// argument checks, workspace carving and the choice between the tensor-core
// and the CUDA-core kernels.
#pragma once
#include "common.cuh"

namespace mla {

bool generic_dims_ok(const mla_dims_t &d);
bool tc_available();

inline constexpr size_t kAlign = 256;

struct Carve {
  char *base;
  size_t off = 0;
  explicit Carve(void *b) : base(static_cast<char *>(b)) {}
  void *take(size_t bytes) {
    off = (off + kAlign - 1) / kAlign * kAlign;
    void *p = base ? base + off : nullptr;
    off += bytes;
    return p;
  }
};

inline int check_dims(const mla_dims_t *d) {
  if (!d) return MLA_ERR_INVALID;
  if (d->num_heads < 1 || d->kv_lora_rank < 1 || d->qk_rope_dim < 0 || d->qk_nope_dim < 1 ||
      d->v_dim < 1 || d->block_size < 1 || !valid_dtype(d->dtype))
    return MLA_ERR_INVALID;
  if (!(d->softmax_scale > 0.f)) return MLA_ERR_INVALID;
  const int es = elem_bytes(d->dtype);
  if (((d->kv_lora_rank + d->qk_rope_dim) * es) % 16 != 0) return MLA_ERR_UNSUPPORTED;
  if (d->v_dim % 8 != 0) return MLA_ERR_UNSUPPORTED;
  if (!generic_dims_ok(*d)) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

inline int kv_width(const mla_dims_t &d) { return d.num_heads * (d.qk_nope_dim + d.v_dim); }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// The tensor-core kernels serve bf16 storage with the DeepSeek-V3 head shape
// (latent 512, rope 64, nope 128, v 128); the CUDA-core kernels serve float32
// storage and every other head shape.  A call of the tensor-core shape runs
// on the tensor-core kernels or fails with MLA_ERR_UNSUPPORTED (no tcgen05
// GPU, an operand not 16-byte aligned, a K/V type they do not take): it is
// never handed to the CUDA-core kernels, which are 10-100x slower.
inline bool tc_shape(const mla_dims_t &d) {
  return d.dtype == MLA_DTYPE_BF16 && d.kv_lora_rank == 512 && d.qk_rope_dim == 64 &&
         d.qk_nope_dim == 128 && d.v_dim == 128;
}

}  // namespace mla
