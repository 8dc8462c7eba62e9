// vc_verify_rows.h -- windowed verification of at most 8 query rows per
// (request, KV head) (nq * g <= 8: single-token decoding and short blocks).
#pragma once

#include "../../include/vc.h"

namespace vc {

// The rule has no length in it: at most 8 rows keep all 24 bits of a weight
// (include/vc.h), whatever the context.  It is the faster form too, but for one
// KV head over a very long context (times in vc_verify_rows.cu).
inline bool verify_rows_apply(const vc_attn_shape& sh, int nq) { return nq * (sh.Hq / sh.Hkv) <= 8; }
size_t verify_rows_workspace(const vc_attn_shape& sh, int nq);
// Arguments checked by the caller.
vc_status verify_rows_launch(const vc_attn_shape& sh, const void* q, const void* k, const void* v, int64_t T,
                             const int32_t* lens, int nq, int64_t window, int64_t n_sink, float* out, float* lse,
                             void* ws, void* stream);

}  // namespace vc
