// C entry points of the operators next to the step: every argument is checked here, on the
// host, before anything is launched. Nothing here allocates or throws.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "ops_host.h"

namespace {

using moe::set_error;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Bytes of an activation value, 0 for an unknown type.
int type_bytes(int type) { return type == MOE_F32 ? 4 : type == MOE_F16 || type == MOE_BF16 ? 2 : 0; }

// Rows of `wa` bytes every `sa` bytes (na of them) against the same of b: whether they
// share a byte. Two views of one buffer (equal strides) may interleave.
bool rows_overlap(const void* a, int64_t na, int64_t sa, int64_t wa, const void* b, int64_t nb, int64_t sb,
                  int64_t wb) {
  if (na <= 0 || nb <= 0) return false;
  const char* pa = static_cast<const char*>(a);
  const char* pb = static_cast<const char*>(b);
  if (pa >= pb + (nb - 1) * sb + wb || pb >= pa + (na - 1) * sa + wa) return false;
  if (sa != sb) return true;
  const int64_t off = ((pb - pa) % sa + sa) % sa;  // b's row within a's row pitch
  return off < wa || off + wb > sa;
}

int check_matvec(const moe_matvec_cfg* c) {
  if (!c) return set_error(MOE_ERR_NULL_PTR, "cfg is NULL");
  int unit = 32;
  switch (c->qtype) {
    case MOE_Q4_0:
    case MOE_Q4_1: break;
    case MOE_Q4_K: unit = 256; break;
    case MOE_Q4_PLANES:
      if (c->group != 32 && c->group != 64 && c->group != 128)
        return set_error(MOE_ERR_INVALID_CFG, "group %d: MOE_Q4_PLANES takes 32, 64 or 128", c->group);
      unit = c->group;
      break;
    default:
      return set_error(MOE_ERR_INVALID_CFG, "qtype %d: expected MOE_Q4_0, MOE_Q4_1, MOE_Q4_K or MOE_Q4_PLANES",
                       c->qtype);
  }
  if (c->qtype != MOE_Q4_PLANES && c->group != 0)
    return set_error(MOE_ERR_INVALID_CFG, "group %d: only MOE_Q4_PLANES has a group", c->group);
  if (c->rows < 1) return set_error(MOE_ERR_INVALID_CFG, "rows %d: must be positive", c->rows);
  if (c->cols < 32 || c->cols > 16384 || c->cols % unit)
    return set_error(MOE_ERR_INVALID_CFG, "cols %d: must be a multiple of %d, at most 16384", c->cols, unit);
  if (c->n_vec < 0 || c->n_vec > 65535)
    return set_error(MOE_ERR_INVALID_CFG, "n_vec %d: must be in [0, 65535]", c->n_vec);
  if (!type_bytes(c->x_type) || !type_bytes(c->y_type))
    return set_error(MOE_ERR_INVALID_CFG, "x_type %d, y_type %d: expected MOE_F32, MOE_F16 or MOE_BF16", c->x_type,
                     c->y_type);
  if (c->flags & ~(MOE_ACCUMULATE | MOE_NO_PDL))
    return set_error(MOE_ERR_INVALID_CFG, "unknown flag bits 0x%x", c->flags);
  if (c->x_stride != 0 && (c->x_stride < c->cols || c->x_stride > (int64_t)1 << 28))
    return set_error(MOE_ERR_INVALID_CFG, "x_stride %lld: must be 0 or at least cols", (long long)c->x_stride);
  if (c->y_stride != 0 && (c->y_stride < c->rows || c->y_stride > (int64_t)1 << 28))
    return set_error(MOE_ERR_INVALID_CFG, "y_stride %lld: must be 0 or at least rows", (long long)c->y_stride);
  if (c->x_stride * type_bytes(c->x_type) % 16)
    return set_error(MOE_ERR_ALIGNMENT, "x_stride %lld: vectors must start on 16 bytes", (long long)c->x_stride);
  return MOE_OK;
}

int check_linattn(const moe_linattn_cfg* c) {
  if (!c) return set_error(MOE_ERR_NULL_PTR, "cfg is NULL");
  if (c->n_seq < 0 || c->n_seq > 65535)
    return set_error(MOE_ERR_INVALID_CFG, "n_seq %d: must be in [0, 65535]", c->n_seq);
  if (c->n_tokens < 0) return set_error(MOE_ERR_INVALID_CFG, "n_tokens %d < 0", c->n_tokens);
  if (c->n_heads < 1 || c->n_heads > 1024)
    return set_error(MOE_ERR_INVALID_CFG, "n_heads %d: must be in [1, 1024]", c->n_heads);
  if (c->n_qk_heads < 1 || c->n_heads % c->n_qk_heads)
    return set_error(MOE_ERR_INVALID_CFG, "n_qk_heads %d must divide n_heads %d", c->n_qk_heads, c->n_heads);
  if (c->key_dim < 8 || c->key_dim > 128 || c->key_dim % 8 || c->value_dim < 8 || c->value_dim > 128 ||
      c->value_dim % 8)
    return set_error(MOE_ERR_INVALID_CFG, "key_dim %d, value_dim %d: must be multiples of 8 from 8 to 128",
                     c->key_dim, c->value_dim);
  if (c->n_states < 0) return set_error(MOE_ERR_INVALID_CFG, "n_states %d < 0", c->n_states);
  const int tb = type_bytes(c->type);
  if (!tb) return set_error(MOE_ERR_INVALID_CFG, "type %d: expected MOE_F32, MOE_F16 or MOE_BF16", c->type);
  if (!std::isfinite(c->scale)) return set_error(MOE_ERR_INVALID_CFG, "scale is not finite");
  if (c->flags & ~(MOE_FRESH_STATE | MOE_TOKEN_DECAY | MOE_NO_PDL))
    return set_error(MOE_ERR_INVALID_CFG, "unknown flag bits 0x%x", c->flags);
  const int64_t qk = (int64_t)c->n_qk_heads * c->key_dim, vo = (int64_t)c->n_heads * c->value_dim;
  const int64_t strides[4] = {c->q_stride, c->k_stride, c->v_stride, c->o_stride};
  const int64_t least[4] = {qk, qk, vo, vo};
  for (int i = 0; i < 4; ++i) {
    if (strides[i] != 0 && (strides[i] < least[i] || strides[i] > (int64_t)1 << 28))
      return set_error(MOE_ERR_INVALID_CFG, "%c_stride %lld: must be 0 or at least %lld", "qkvo"[i],
                       (long long)strides[i], (long long)least[i]);
    if (strides[i] * tb % 16)
      return set_error(MOE_ERR_ALIGNMENT, "%c_stride %lld: tokens must start on 16 bytes", "qkvo"[i],
                       (long long)strides[i]);
  }
  return MOE_OK;
}

// The checks of a call's pointers, and its kernel arguments.
int linattn_args(const void* q, const void* k, const void* v, const float* g, const int32_t* offsets,
                 const int32_t* slots, const moe_linattn_cfg* c, float* state, void* o, moe::LinattnArgs* a) {
  const bool tokens = c->n_tokens > 0;
  if (!state || (tokens && (!q || !k || !v || !o)) || (!g && (tokens || !(c->flags & MOE_TOKEN_DECAY))))
    return set_error(MOE_ERR_NULL_PTR, "q, k, v, log_decay, state and o must not be NULL");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(state, 16))
    return set_error(MOE_ERR_ALIGNMENT, "q, k, v, o and state must be 16-byte aligned");
  if (!aligned(g, 4) || !aligned(offsets, 4) || !aligned(slots, 4))
    return set_error(MOE_ERR_ALIGNMENT, "log_decay, offsets and slots must be 4-byte aligned");
  if (!slots && c->n_seq > c->n_states)
    return set_error(MOE_ERR_INVALID_CFG, "%d sequences without slots need as many states (n_states %d)", c->n_seq,
                     c->n_states);
  const int64_t tb = type_bytes(c->type);
  const int64_t qk = (int64_t)c->n_qk_heads * c->key_dim, vo = (int64_t)c->n_heads * c->value_dim;
  a->q = q;
  a->k = k;
  a->v = v;
  a->g = g;
  a->offsets = offsets;
  a->slots = slots;
  a->state = state;
  a->o = o;
  a->qs = c->q_stride ? c->q_stride : qk;
  a->ks = c->k_stride ? c->k_stride : qk;
  a->vs = c->v_stride ? c->v_stride : vo;
  a->os = c->o_stride ? c->o_stride : vo;
  a->B = c->n_seq;
  a->N = c->n_tokens;
  a->seq_len = c->n_tokens / c->n_seq;
  a->H = c->n_heads;
  a->rep = c->n_heads / c->n_qk_heads;
  a->dk = c->key_dim;
  a->dv = c->value_dim;
  a->n_states = c->n_states;
  a->scale = c->scale;
  a->fresh = (c->flags & MOE_FRESH_STATE) != 0;
  a->token_decay = (c->flags & MOE_TOKEN_DECAY) != 0;
  const int64_t n = c->n_tokens;
  if (rows_overlap(o, n, a->os * tb, vo * tb, q, n, a->qs * tb, qk * tb) ||
      rows_overlap(o, n, a->os * tb, vo * tb, k, n, a->ks * tb, qk * tb) ||
      rows_overlap(o, n, a->os * tb, vo * tb, v, n, a->vs * tb, vo * tb))
    return set_error(MOE_ERR_INVALID_CFG, "o overlaps q, k or v");
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_q4_matvec(const void* x, const void* weights, const void* scales, const void* mins, const float* bias,
                  const moe_matvec_cfg* c, void* y, void* stream) {
  moe::clear_error();
  const int rc = check_matvec(c);
  if (rc != MOE_OK) return rc;
  if (c->n_vec == 0) return MOE_OK;
  if (!x || !weights || !y) return set_error(MOE_ERR_NULL_PTR, "x, weights and y must not be NULL");
  const bool planes = c->qtype == MOE_Q4_PLANES;
  if (planes && !scales) return set_error(MOE_ERR_NULL_PTR, "MOE_Q4_PLANES needs scales");
  if (!planes && (scales || mins))
    return set_error(MOE_ERR_INVALID_CFG, "scales and mins are planes of MOE_Q4_PLANES: blocks hold their own");
  const int xb = type_bytes(c->x_type), yb = type_bytes(c->y_type);
  if (!aligned(x, 16) || !aligned(weights, 16) || !aligned(scales, 16) || !aligned(mins, 16))
    return set_error(MOE_ERR_ALIGNMENT, "x, weights, scales and mins must be 16-byte aligned");
  if (!aligned(y, yb) || !aligned(bias, 4))
    return set_error(MOE_ERR_ALIGNMENT, "y and bias must be aligned to their elements");
  moe::MatvecArgs a{};
  a.x = x;
  a.w = static_cast<const uint8_t*>(weights);
  a.scales = static_cast<const uint8_t*>(scales);
  a.mins = static_cast<const uint8_t*>(mins);
  a.bias = bias;
  a.y = y;
  a.xs = c->x_stride ? c->x_stride : c->cols;
  a.ys = c->y_stride ? c->y_stride : c->rows;
  a.rows = c->rows;
  a.cols = c->cols;
  a.T = c->n_vec;
  a.qtype = c->qtype;
  a.group = c->group;
  a.x_type = c->x_type;
  a.y_type = c->y_type;
  a.flags = c->flags;
  if (rows_overlap(x, a.T, a.xs * xb, (int64_t)a.cols * xb, y, a.T, a.ys * yb, (int64_t)a.rows * yb))
    return set_error(MOE_ERR_INVALID_CFG, "x and y overlap");
  const cudaError_t e = moe::matvec_launch(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "matrix-vector kernel launch");
}

size_t moe_linattn_workspace_size(const moe_linattn_cfg* c) {
  moe::clear_error();
  if (check_linattn(c) != MOE_OK) return 0;
  return moe::linattn_workspace(c->n_tokens, c->n_heads, c->key_dim, c->value_dim, c->type);
}

int moe_linattn_prefill(const void* q, const void* k, const void* v, const float* log_decay, const int32_t* offsets,
                        const int32_t* slots, const moe_linattn_cfg* c, float* state, void* o, void* workspace,
                        size_t workspace_bytes, void* stream) {
  moe::clear_error();
  int rc = check_linattn(c);
  if (rc != MOE_OK) return rc;
  if (c->n_seq == 0) return MOE_OK;
  if (!offsets && c->n_tokens % c->n_seq)
    return set_error(MOE_ERR_INVALID_CFG, "n_tokens %d: without offsets it must be a multiple of n_seq %d",
                     c->n_tokens, c->n_seq);
  moe::LinattnArgs a{};
  rc = linattn_args(q, k, v, log_decay, offsets, slots, c, state, o, &a);
  if (rc != MOE_OK) return rc;
  if (!workspace) return set_error(MOE_ERR_NULL_PTR, "workspace is NULL");
  if (!aligned(workspace, 256)) return set_error(MOE_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
  const size_t need = moe_linattn_workspace_size(c);
  if (workspace_bytes < need)
    return set_error(MOE_ERR_WORKSPACE, "workspace of %zu bytes, this call needs %zu", workspace_bytes, need);
  const cudaError_t e = moe::linattn_prefill_launch(a, c->type, workspace, (c->flags & MOE_NO_PDL) == 0,
                                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "linear attention kernel launch");
}

int moe_linattn_step(const void* q, const void* k, const void* v, const float* log_decay, const int32_t* slots,
                     const moe_linattn_cfg* c, float* state, void* o, void* stream) {
  moe::clear_error();
  int rc = check_linattn(c);
  if (rc != MOE_OK) return rc;
  if (c->n_tokens != c->n_seq)
    return set_error(MOE_ERR_INVALID_CFG, "n_tokens %d: a step has one token for each of the %d sequences",
                     c->n_tokens, c->n_seq);
  if (c->n_seq == 0) return MOE_OK;
  moe::LinattnArgs a{};
  rc = linattn_args(q, k, v, log_decay, nullptr, slots, c, state, o, &a);
  if (rc != MOE_OK) return rc;
  const cudaError_t e =
      moe::linattn_step_launch(a, c->type, (c->flags & MOE_NO_PDL) == 0, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::set_cuda_error(e, "linear attention kernel launch");
}

}  // extern "C"
