// w4_forward.hip -- products of many token rows with 4-bit group-quantized
// weights: y = x W^T and the gated block, for prompts and training steps.
//
// What bounds it: the matrix instructions, 2 m n k operations.  Codes become exact
// bfloat16 integers on their way into LDS, once per tile; each span's sum (64
// columns, or 32 where groups are that fine) is multiplied by its scale as it
// joins the tile's sum, so no weight is rounded.
#include "fq_host.h"
#include "w4_linear.h"
#include "w4_tile.h"

namespace fqw {
namespace {

template <class T>
struct ForwardArgs {
    const uint16_t* x;  // [m] rows of `cols` columns, ld apart: `parts` 64-column pieces per 64 columns of W
    int64_t ld, cols;
    int parts;
    W4Mat w[2];
    T* out[3];  // y, or h, g, u
    int64_t m, n, k;
    uint32_t spans, per_group;  // spans in a row, spans in a group
    uint32_t ni, nj;            // tiles
    int act;
};

// The weights' side of a tile: a thread holds 32 codes of one of the tile's rows.
template <int BN, int SPAN, bool ZP, int W>
struct CodeRows {
    const uint8_t* p;
    const float* scale;
    const int32_t* zp;
    int64_t left;  // bytes of the matrix from p on
    uint32_t spans, per_group;
    int row, half;
    u32x4 c;
    float s, z;
    template <class Args>
    __device__ __forceinline__ CodeRows(const Args& a, int64_t col0, int t)
        : spans(a.spans), per_group(a.per_group), row(t / 2), half(t % 2) {
        // a wave's 64 rows hold 32 of the gate matrix and then the same 32 of the up matrix
        const W4Mat& w = a.w[W == 1 ? 0 : row / 32 % 2];
        int64_t r = col0 + (W == 1 ? row : row / 64 * 32 + row % 32);
        r = r < a.n ? r : a.n - 1;
        p = w.codes + r * w.row_bytes + half * 16;
        left = (a.n - r) * w.row_bytes - half * 16;
        scale = w.scale + r * w.ng;
        zp = w.zp ? w.zp + r * w.ng : nullptr;
    }
    __device__ __forceinline__ void load(uint32_t step) {
        const int64_t b = (int64_t)step * 32;
        // past its row's end a thread reads codes of the next row, which meet zeros of x
        c = load16_part(p + b, left - b);
        uint32_t i = SPAN == 64 ? step : 2 * step + half;
        i = i < spans ? i : spans - 1;
        if (per_group > 1) i /= per_group;
        s = scale[i];
        if constexpr (ZP) z = zp ? (float)zp[i] : 0.0f;
    }
    __device__ __forceinline__ void store(uint16_t* tile, float* scales) const {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<bf16x8*>(tile + by_rows(row, half * 4 + j)) = codes_bf16<ZP>(c[j], ZP ? z * 0.0625f : 0.0f);
        if (SPAN == 32 || half == 0) scales[(SPAN == 32 ? half * BN : 0) + row] = s * 16.0f;
    }
};

template <class S, int SPAN, bool ZP, int W, class T>
__global__ __launch_bounds__(S::kThreads, 2) void k_forward(ForwardArgs<T> a) {
    constexpr int BM = S::BM, BN = S::BN, kSums = kDeep / SPAN;
    __shared__ __attribute__((aligned(1024))) uint16_t xa[2][BM * kDeep];
    __shared__ __attribute__((aligned(1024))) uint16_t wb[2][BN * kDeep];
    __shared__ float sc[2][kSums * BN];
    const int t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
    uint32_t ti, tj;
    tile_at(blockIdx.x, a.ni, a.nj, ti, tj);
    const int64_t i0 = (int64_t)ti * BM, j0 = (int64_t)tj * (BN / W);
    const DenseRows<BM, S::kThreads> xs(a.x, i0, a.m, a.ld, a.cols, wave, lane);
    CodeRows<BN, SPAN, ZP, W> ws(a, j0, t);
    const uint32_t steps = (uint32_t)((a.cols + kDeep - 1) / kDeep), parts = a.parts;
    const int wi = wave / S::WN * (S::MS * 32), wj = wave % S::WN * (S::NS * 32);

    f32x16 acc[S::MS][S::NS] = {};
    ws.load(0);
    xs.fill(xa[0], 0);
    ws.store(wb[0], sc[0]);
    uint32_t kt = 0, part = 0;  // step of W, part of x, of the codes in registers
    auto advance = [&] {
        if (++part == parts) part = 0, ++kt;
    };
    advance();
    if (1 < steps) ws.load(kt);
    wait_dma();
    __syncthreads();
    for (uint32_t st = 0; st < steps; ++st) {
        const int cur = st & 1;
        if (st + 1 < steps) {
            ws.store(wb[cur ^ 1], sc[cur ^ 1]);  // before new loads, which its wait would include
            xs.fill(xa[cur ^ 1], (int64_t)(st + 1) * kDeep);
            advance();
            if (st + 2 < steps) ws.load(kt);
        }
        bf16x8 b[S::NS][4];
        float s[kSums][S::NS];
#pragma unroll
        for (int j = 0; j < S::NS; ++j) {
#pragma unroll
            for (int d = 0; d < 4; ++d) b[j][d] = frag_rows(wb[cur], wj + 32 * j, d, lane);
#pragma unroll
            for (int g = 0; g < kSums; ++g) s[g][j] = sc[cur][g * BN + wj + 32 * j + lane % 32];
        }
#pragma unroll
        for (int i = 0; i < S::MS; ++i) {
            bf16x8 f[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) f[d] = frag_rows(xa[cur], wi + 32 * i, d, lane);
#pragma unroll
            for (int g = 0; g < kSums; ++g)
#pragma unroll
                for (int j = 0; j < S::NS; ++j) {
                    f32x16 p = {};
#pragma unroll
                    for (int d = g * (4 / kSums); d < (g + 1) * (4 / kSums); ++d)
                        p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[d], b[j][d], p, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(p[e], s[g][j], acc[i][j][e]);
                }
        }
        wait_dma();
        __syncthreads();
    }

#pragma unroll
    for (int i = 0; i < S::MS; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int64_t r = i0 + wi + 32 * i + 8 * (e / 4) + 4 * (lane / 32) + e % 4;
            if (r >= a.m) continue;
            if constexpr (W == 1) {
#pragma unroll
                for (int j = 0; j < S::NS; ++j) {
                    const int64_t c = j0 + wj + 32 * j + lane % 32;
                    if (c < a.n) store_f(a.out[0] + r * a.n + c, acc[i][j][e]);
                }
            } else {
                const int64_t c = j0 + wj / 2 + lane % 32, at = r * a.n + c;
                if (c >= a.n) continue;
                store_f(a.out[0] + at, act_value(a.act, acc[i][0][e]) * acc[i][1][e]);
                if (a.out[1]) {
                    store_f(a.out[1] + at, acc[i][0][e]);
                    store_f(a.out[2] + at, acc[i][1][e]);
                }
            }
        }
}

// x as the kernel reads it: [m][pieces of 64 columns][PARTS][64] bfloat16, zeros
// past the row's end.  float32 in three parts, bfloat16 as it is.
template <class T>
__global__ __launch_bounds__(256) void k_pieces(const T* x, int64_t m, int64_t k, int64_t kp, uint16_t* out) {
    constexpr int P = Tokens<T>::kParts;
    const int64_t chunks = kp / 8;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < m * chunks; i += gridDim.x * 256ll) {
        const int64_t r = i / chunks, c = i % chunks * 8;
        Tokens<T> f;
        f.load_part(x + r * k + c, k - c);
        bf16x8 v[P];
        f.parts(v);
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<bf16x8*>(out + r * kp * P + (c / 64 * P + p) * 64 + c % 64) = v[p];
    }
}

template <class S, int SPAN, int W, class T>
int launch(ForwardArgs<T> a, bool zp, hipStream_t stream) {
    const int64_t ni = (a.m + S::BM - 1) / S::BM, nj = (a.n + S::BN / W - 1) / (S::BN / W);
    if (ni * nj > 0x7FFFFFFF) return FQ_E_UNSUPPORTED;
    a.ni = (uint32_t)ni;
    a.nj = (uint32_t)nj;
    const dim3 g((unsigned)(ni * nj)), b(S::kThreads);
    if (zp) k_forward<S, SPAN, true, W, T><<<g, b, 0, stream>>>(a);
    else k_forward<S, SPAN, false, W, T><<<g, b, 0, stream>>>(a);
    return fqh::launched();
}

template <int W, class T>
int forward(ForwardArgs<T> a, const T* x, int64_t group, void* workspace, hipStream_t stream) {
    constexpr int P = Tokens<T>::kParts;
    if (forward_workspace(P == 3 ? FQ_F32 : FQ_BF16, a.m, a.k)) {
        const int64_t kp = (a.k + 63) / 64 * 64;
        k_pieces<T><<<fqh::grid_all(a.m * kp / 8, 256), 256, 0, stream>>>(x, a.m, a.k, kp, (uint16_t*)workspace);
        a.x = (const uint16_t*)workspace;
        a.ld = a.cols = kp * P;
    } else {
        a.x = (const uint16_t*)x;
        a.ld = a.cols = a.k;
    }
    a.parts = P;
    const bool fine = !(group >= a.k || group % 64 == 0), zp = a.w[0].zp || a.w[W - 1].zp;
    const int span = fine ? 32 : 64;
    a.spans = (uint32_t)((a.k + span - 1) / span);
    a.per_group = spans_per_group(group, a.k, span);
    using Big = Shape<256, 256, 2, 4>;
    using Small = Shape<128, 128, 2, 2>;
    const int64_t big = ((a.m + 255) / 256) * ((a.n * W + 255) / 256);
    if (big >= fqh::num_cus() / 2) {
        return fine ? launch<Big, 32, W, T>(a, zp, stream) : launch<Big, 64, W, T>(a, zp, stream);
    }
    return fine ? launch<Small, 32, W, T>(a, zp, stream) : launch<Small, 64, W, T>(a, zp, stream);
}

}  // namespace

size_t forward_workspace(int dtype, int64_t m, int64_t k) {
    const int64_t kp = (k + 63) / 64 * 64;
    if (dtype == FQ_F32) return (size_t)(m * kp * 6);
    return k % 8 ? (size_t)(m * kp * 2) : 0;
}

int forward_matmul(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, const fql_w4& w, void* y,
                   void* workspace, hipStream_t stream) {
    const W4Mat wm = w4_mat(w, k, group);
    if (dtype == FQ_F32) {
        ForwardArgs<float> a{nullptr, 0, 0, 0, {wm, wm}, {(float*)y}, m, n, k};
        return forward<1, float>(a, (const float*)x, group, workspace, stream);
    }
    ForwardArgs<uint16_t> a{nullptr, 0, 0, 0, {wm, wm}, {(uint16_t*)y}, m, n, k};
    return forward<1, uint16_t>(a, (const uint16_t*)x, group, workspace, stream);
}

int forward_gated(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, int act, const fql_w4& gate,
                  const fql_w4& up, void* h, void* g, void* u, void* workspace, hipStream_t stream) {
    const W4Mat wg = w4_mat(gate, k, group), wu = w4_mat(up, k, group);
    if (dtype == FQ_F32) {
        ForwardArgs<float> a{nullptr, 0, 0, 0, {wg, wu}, {(float*)h, (float*)g, (float*)u}, m, n, k, 0, 0, 0, 0, act};
        return forward<2, float>(a, (const float*)x, group, workspace, stream);
    }
    ForwardArgs<uint16_t> a{nullptr, 0, 0, 0, {wg, wu}, {(uint16_t*)h, (uint16_t*)g, (uint16_t*)u}, m, n, k, 0, 0, 0, 0, act};
    return forward<2, uint16_t>(a, (const uint16_t*)x, group, workspace, stream);
}

}  // namespace fqw
