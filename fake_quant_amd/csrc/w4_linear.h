// w4_linear.h -- host entry points of the kernels behind fq_linear.h (arguments
// already checked there).
#pragma once

#include "fq_linear.h"

namespace fqw {

// Up to kFewTokens rows of x, groups that span_of takes.
constexpr int64_t kFewTokens = 64;
int few_matmul(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, const fql_w4& w, void* y,
               hipStream_t stream);
int few_gated(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, int act, const fql_w4& gate,
              const fql_w4& up, void* h, void* g, void* u, hipStream_t stream);

}  // namespace fqw
