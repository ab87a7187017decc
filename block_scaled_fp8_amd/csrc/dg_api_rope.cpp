// C ABI of norm and rotation of queries and keys: argument validation and launch.  Validation runs before any HIP call.
#include <cmath>

#include "dg_api_check.h"

namespace {

using dg::aligned;
using dg::api_fail;
using dg::api_ok;
using dg::check_rows;
using dg::kMaxIndex;

int check_shape(int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return api_fail(DG_ERR_UNSUPPORTED, "head_dim = %d: 64, 128 and 256 are supported", head_dim);
  if (num_tokens < 0 || num_tokens > kMaxIndex) return api_fail(DG_ERR_SHAPE, "num_tokens = %d must be in [0, 2^30]", num_tokens);
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads > 65535 || num_kv_heads > 65535)
    return api_fail(DG_ERR_SHAPE, "num_q_heads = %d and num_kv_heads = %d must be in [1, 65535]", num_q_heads, num_kv_heads);
  return DG_OK;
}

// Checks of everything but the rows; `empty`: there are no tokens, so only the weights' gradients may be written.
int check_call(const dg_norm_rope* a) {
  if (!a) return api_fail(DG_ERR_NULL, "the norm's and rotation's arguments must not be NULL");
  if (int s = check_shape(a->num_tokens, a->num_q_heads, a->num_kv_heads, a->head_dim)) return s;
  if (a->dtype != DG_IN_BF16 && a->dtype != DG_IN_F32) return api_fail(DG_ERR_DTYPE, "dtype %d is not DG_IN_BF16 or DG_IN_F32", a->dtype);
  if (a->weight_dtype != DG_IN_BF16 && a->weight_dtype != DG_IN_F32)
    return api_fail(DG_ERR_DTYPE, "weight_dtype %d is not DG_IN_BF16 or DG_IN_F32", a->weight_dtype);
  if (a->rot_dim < 16 || a->rot_dim > a->head_dim || a->rot_dim % 16)
    return api_fail(DG_ERR_SHAPE, "rot_dim = %d must be a multiple of 16 in [16, head_dim = %d]", a->rot_dim, a->head_dim);
  if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return api_fail(DG_ERR_SHAPE, "eps must be finite and not negative");
  if (a->num_positions < 0 || a->num_positions > kMaxIndex) return api_fail(DG_ERR_SHAPE, "num_positions = %lld must be in [0, 2^30]", (long long)a->num_positions);
  if (a->num_positions > 1 && a->cos_sin_stride < a->rot_dim) return api_fail(DG_ERR_LAYOUT, "cos_sin_stride must be at least rot_dim");
  if (a->num_tokens == 0) return DG_OK;
  if (!a->q_weight || !a->k_weight || !a->positions || (!a->cos_sin && a->num_positions))
    return api_fail(DG_ERR_NULL, "q_weight, k_weight, cos_sin and positions must not be NULL");
  if (!aligned(a->q_weight, 16) || !aligned(a->k_weight, 16)) return api_fail(DG_ERR_LAYOUT, "q_weight and k_weight must be 16-byte aligned");
  if (!aligned(a->cos_sin, 16) || (a->num_positions > 1 && a->cos_sin_stride % 4))
    return api_fail(DG_ERR_LAYOUT, "cos_sin must have 16-byte aligned rows");
  if (!aligned(a->positions, 8)) return api_fail(DG_ERR_LAYOUT, "positions must be 8-byte aligned");
  return DG_OK;
}

int element_size(const dg_norm_rope* a) { return a->dtype == DG_IN_BF16 ? 2 : 4; }

int check_operand(const dg_norm_rope* a, const char* name, const dg::Rows& r) {
  return check_rows(name, r.p, r.token_stride, r.head_stride, element_size(a));
}

dg::Rows rows(const void* p, int64_t token_stride, int64_t head_stride) { return {const_cast<void*>(p), token_stride, head_stride}; }

dg::Rows from_token(const dg::Rows& r, int64_t token, int esz) {
  return {static_cast<char*>(r.p) + token * r.token_stride * esz, r.token_stride, r.head_stride};
}

dg::RopeParams kernel_params(const dg_norm_rope* a) {
  dg::RopeParams p{};
  p.q_weight = a->q_weight;
  p.k_weight = a->k_weight;
  p.cos_sin = a->cos_sin;
  p.cos_sin_stride = a->num_positions > 1 ? a->cos_sin_stride : 0;
  p.positions = a->positions;
  p.num_positions = a->num_positions;
  p.rot = a->rot_dim;
  p.num_tokens = a->num_tokens;
  p.q_heads = a->num_q_heads;
  p.kv_heads = a->num_kv_heads;
  p.eps = a->eps;
  p.weights_bf16 = a->weight_dtype == DG_IN_BF16;
  const int heads = dg::rope_heads(a->head_dim);
  p.q_pieces = (a->num_q_heads + heads - 1) / heads;
  p.kv_pieces = (a->num_kv_heads + heads - 1) / heads;
  return p;
}

int forward(const dg_norm_rope* a, dg::Rows q, dg::Rows k, dg::Rows v, dg::Rows q_out, dg::Rows k_out, const dg_fp8_kv_cache* cache,
            const int64_t* slots, hipStream_t stream) {
  const int esz = element_size(a);
  dg::RopeParams p = kernel_params(a);
  const int pieces = p.q_pieces + (cache ? 2 : 1) * p.kv_pieces;
  p.pieces = dg::fast_div(pieces);
  if (cache) p.c = dg::kernel_cache(cache);
  // A grid has less than 2^32 threads (one of more is cut to its low 32 bits without an error): 2^25 waves at a time.
  const int32_t most = (1 << 25) / pieces;
  for (int32_t from = 0; from < a->num_tokens; from += most) {
    p.q = from_token(q, from, esz);
    p.k = from_token(k, from, esz);
    p.q_out = from_token(q_out, from, esz);
    if (cache) {
      p.v = from_token(v, from, esz);
      p.slots = slots + from;
    } else {
      p.k_out = from_token(k_out, from, esz);
    }
    p.positions = a->positions + from;
    p.num_tokens = a->num_tokens - from < most ? a->num_tokens - from : most;
    const hipError_t e = dg::launch_norm_rope(p, a->head_dim, a->dtype == DG_IN_BF16, a->interleaved != 0, cache != nullptr, stream);
    if (e != hipSuccess) return api_fail(DG_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  }
  return api_ok();
}

// Workgroups of the backward kernel: its waves go over (token, heads of a wave) in turn, and each workgroup leaves one set
// of the weights' sums.  Four for a compute unit, as many as it holds: 8192 tokens of 32 + 8 heads of 128, forward and backward, take 78.0 us, with
// five (and registers for them) 80.9; with two and with eight it was 5 and 2.5 us more.
int backward_workgroups(int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int num_sms) {
  const int heads = dg::rope_heads(head_dim);
  const int most = num_q_heads > num_kv_heads ? num_q_heads : num_kv_heads;
  const int64_t waves = int64_t(num_tokens) * ((most + heads - 1) / heads), groups = (waves + 3) / 4, limit = int64_t(num_sms) * 4;
  return int(groups < 1 ? 1 : groups < limit ? groups : limit);
}

int64_t backward_workspace(int workgroups, int32_t head_dim) { return workgroups > 1 ? int64_t(workgroups) * 2 * head_dim * 4 : 0; }

}  // namespace

extern "C" {

int dg_qk_norm_rope(const dg_norm_rope* a, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                    const void* k, int64_t k_token_stride, int64_t k_head_stride,
                    void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                    void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                    hipStream_t stream) {
  const dg::Rows q_rows = rows(q, q_token_stride, q_head_stride);
  const dg::Rows k_rows = rows(k, k_token_stride, k_head_stride);
  const dg::Rows q_out_rows = rows(q_out, q_out_token_stride, q_out_head_stride);
  const dg::Rows k_out_rows = rows(k_out, k_out_token_stride, k_out_head_stride);
  if (int s = check_call(a)) return s;
  if (a->num_tokens == 0) return api_ok();
  if (int s = check_operand(a, "q", q_rows)) return s;
  if (int s = check_operand(a, "k", k_rows)) return s;
  if (int s = check_operand(a, "q_out", q_out_rows)) return s;
  if (int s = check_operand(a, "k_out", k_out_rows)) return s;
  return forward(a, q_rows, k_rows, {}, q_out_rows, k_out_rows, nullptr, nullptr, stream);
}

int dg_qk_norm_rope_fp8_kv_cache_write(const dg_norm_rope* a, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                    const void* k, int64_t k_token_stride, int64_t k_head_stride,
                    const void* v, int64_t v_token_stride, int64_t v_head_stride,
                    void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                    const dg_fp8_kv_cache* cache, const int64_t* slots, hipStream_t stream) {
  const dg::Rows q_rows = rows(q, q_token_stride, q_head_stride);
  const dg::Rows k_rows = rows(k, k_token_stride, k_head_stride);
  const dg::Rows v_rows = rows(v, v_token_stride, v_head_stride);
  const dg::Rows q_out_rows = rows(q_out, q_out_token_stride, q_out_head_stride);
  if (int s = check_call(a)) return s;
  if (int s = dg::check_cache(cache, a->num_tokens == 0)) return s;
  if (cache->num_heads != a->num_kv_heads || cache->head_dim != a->head_dim)
    return api_fail(DG_ERR_SHAPE, "the cache has %d heads of %d, the keys %d of %d", cache->num_heads, cache->head_dim, a->num_kv_heads, a->head_dim);
  if (a->num_tokens == 0) return api_ok();
  if (int s = check_operand(a, "q", q_rows)) return s;
  if (int s = check_operand(a, "k", k_rows)) return s;
  if (int s = check_operand(a, "v", v_rows)) return s;
  if (int s = check_operand(a, "q_out", q_out_rows)) return s;
  if (!slots) return api_fail(DG_ERR_NULL, "slots must not be NULL");
  if (!aligned(slots, 8)) return api_fail(DG_ERR_LAYOUT, "slots must be 8-byte aligned");
  return forward(a, q_rows, k_rows, v_rows, q_out_rows, {}, cache, slots, stream);
}

int64_t dg_qk_norm_rope_backward_workspace(int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (int s = check_shape(num_tokens, num_q_heads, num_kv_heads, head_dim)) return s;
  const int num_sms = dg::api_num_sms();
  if (num_sms <= 0) return api_fail(DG_ERR_HIP, "could not query the device's compute-unit count");
  return backward_workspace(backward_workgroups(num_tokens, num_q_heads, num_kv_heads, head_dim, num_sms), head_dim);
}

int dg_qk_norm_rope_backward(const dg_norm_rope* a, const void* dq_out, int64_t dq_out_token_stride, int64_t dq_out_head_stride,
                    const void* dk_out, int64_t dk_out_token_stride, int64_t dk_out_head_stride,
                    const void* q, int64_t q_token_stride, int64_t q_head_stride,
                    const void* k, int64_t k_token_stride, int64_t k_head_stride,
                    void* dq, int64_t dq_token_stride, int64_t dq_head_stride,
                    void* dk, int64_t dk_token_stride, int64_t dk_head_stride,
                    float* dq_weight, float* dk_weight, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const dg::Rows dq_out_rows = rows(dq_out, dq_out_token_stride, dq_out_head_stride);
  const dg::Rows dk_out_rows = rows(dk_out, dk_out_token_stride, dk_out_head_stride);
  const dg::Rows q_rows = rows(q, q_token_stride, q_head_stride);
  const dg::Rows k_rows = rows(k, k_token_stride, k_head_stride);
  const dg::Rows dq_rows = rows(dq, dq_token_stride, dq_head_stride);
  const dg::Rows dk_rows = rows(dk, dk_token_stride, dk_head_stride);
  if (int s = check_call(a)) return s;
  if (!dq_weight || !dk_weight) return api_fail(DG_ERR_NULL, "dq_weight and dk_weight must not be NULL");
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return api_fail(DG_ERR_LAYOUT, "dq_weight and dk_weight must be 4-byte aligned");
  if (!a->q_weight || !a->k_weight || !aligned(a->q_weight, 16) || !aligned(a->k_weight, 16))
    return api_fail(a->q_weight && a->k_weight ? DG_ERR_LAYOUT : DG_ERR_NULL, "q_weight and k_weight must be given, 16-byte aligned");
  if (a->num_tokens > 0) {
    if (int s = check_operand(a, "dq_out", dq_out_rows)) return s;
    if (int s = check_operand(a, "dk_out", dk_out_rows)) return s;
    if (int s = check_operand(a, "q", q_rows)) return s;
    if (int s = check_operand(a, "k", k_rows)) return s;
    if (int s = check_operand(a, "dq", dq_rows)) return s;
    if (int s = check_operand(a, "dk", dk_rows)) return s;
  }
  const int num_sms = dg::api_num_sms();
  if (num_sms <= 0) return api_fail(DG_ERR_HIP, "could not query the device's compute-unit count");
  dg::RopeParams p = kernel_params(a);
  p.workgroups = backward_workgroups(a->num_tokens, a->num_q_heads, a->num_kv_heads, a->head_dim, num_sms);
  const int64_t need = backward_workspace(p.workgroups, a->head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return api_fail(workspace ? DG_ERR_SHAPE : DG_ERR_NULL, "this call needs a workspace of %lld bytes", (long long)need);
  if (need > 0 && !aligned(workspace, 16)) return api_fail(DG_ERR_LAYOUT, "workspace must be 16-byte aligned");
  p.q = q_rows;
  p.k = k_rows;
  p.dq = dq_out_rows;
  p.dk = dk_out_rows;
  p.q_out = dq_rows;
  p.k_out = dk_rows;
  p.dq_weight = dq_weight;
  p.dk_weight = dk_weight;
  p.parts = static_cast<float*>(workspace);
  const hipError_t e = dg::launch_norm_rope_backward(p, a->head_dim, a->dtype == DG_IN_BF16, a->interleaved != 0, stream);
  if (e != hipSuccess) return api_fail(DG_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return api_ok();
}

}  // extern "C"
