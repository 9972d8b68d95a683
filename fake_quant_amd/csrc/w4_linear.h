// w4_linear.h -- host entry points of the kernels behind fq_linear.h (arguments
// already checked there).
#pragma once

#include "fq_linear.h"

namespace fqw {

// Up to kFewTokens rows of x, groups that span_of takes.
constexpr int64_t kFewTokens = 512;
int few_matmul(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, const fql_w4& w, void* y,
               hipStream_t stream);
int few_gated(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, int act, const fql_w4& gate,
              const fql_w4& up, void* h, void* g, void* u, hipStream_t stream);

// Widths under this keep 256 rows of three bfloat16 parts under 2^31 bytes.
constexpr int64_t kTileWidth = (int64_t)1 << 20;

// Any more rows of x.  x 16-byte aligned unless forward_workspace is not 0: the
// workspace holds x in the layout that the tiles read, where x itself has another.
size_t forward_workspace(int dtype, int64_t m, int64_t k);
int forward_matmul(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, const fql_w4& w, void* y,
                   void* workspace, hipStream_t stream);
int forward_gated(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, int act, const fql_w4& gate,
                  const fql_w4& up, void* h, void* g, void* u, void* workspace, hipStream_t stream);

// Gradients.  dy and x (dh, g and u only to 2 bytes) 16-byte aligned where their
// rows are whole 16-byte chunks; the workspace holds the others with padded rows,
// and the gated block's dg and du.
size_t backward_workspace(int64_t m, int64_t n, int64_t k, bool gated);
int matmul_backward(const void* dy, const void* x, int64_t m, int64_t n, int64_t k, int64_t group, const fql_w4* w,
                    void* dx, void* dw, int dw_dtype, void* workspace, hipStream_t stream);
int gated_backward(const void* dh, const void* x, const void* g, const void* u, int64_t m, int64_t n, int64_t k,
                   int64_t group, int act, const fql_w4* gate, const fql_w4* up, void* dx, void* dw_gate, void* dw_up,
                   int dw_dtype, void* workspace, hipStream_t stream);

}  // namespace fqw
