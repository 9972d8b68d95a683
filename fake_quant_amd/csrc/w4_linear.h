// w4_linear.h -- host entry points of the kernels behind fq_linear.h (arguments
// already checked there).
#pragma once

#include "fq_linear.h"

namespace fqw {

constexpr int64_t kUnits = 256;  // compute units

// 128 x 256 or 256 x 256 tiles for `rows` x `cols` outputs: a round of the former over
// the compute units takes about 2/3 of a round of the latter (4096 summation indices,
// groups of 128: 96 us for 256 tiles of 128 rows, 115 .. 140 us for 128 .. 256 of 256).
inline bool big_tiles(int64_t rows, int64_t cols) {
    const int64_t wide = (cols + 255) / 256;
    const int64_t mid = ((rows + 127) / 128 * wide + kUnits - 1) / kUnits;
    const int64_t big = ((rows + 255) / 256 * wide + kUnits - 1) / kUnits;
    return 2 * mid >= 3 * big;
}
// Products that the few-token kernel serves: its time grows with the tokens (4096 x
// 4096, 64-column groups: 100 us for 1024), that of one round of tiles does not (93 us
// up to 128 tiles of 128 rows).  columns: outputs per token, of both weights of a pair.
inline bool few_tokens(int64_t m, int64_t columns) {
    return ((m + 127) / 128) * ((columns + 255) / 256) < 112;
}
int few_matmul(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, const fql_w4& w, void* y,
               hipStream_t stream);
int few_gated(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, int act, const fql_w4& gate,
              const fql_w4& up, void* h, void* g, void* u, hipStream_t stream);

// Widths under this keep 256 rows of three bfloat16 parts under 2^31 bytes.
constexpr int64_t kTileWidth = (int64_t)1 << 20;

// The tile kernel.  x 16-byte aligned unless forward_workspace is not 0: the
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
