// w4_backward.hip -- gradients of the products with 4-bit group-quantized weights:
// dx = dy W and dw = dy^T x; the gated block first forms dg and du beside each
// other, so that one pair of products serves both matrices.
//
// What bounds it: the matrix instructions.  dx sums over the rows of W, whose
// scales differ, so W enters as bfloat16 rounded to nearest (2^-8 of a value at
// most, as bfloat16 gradients themselves); dw holds no weight and its products are
// exact.  dg and du are rounded to bfloat16 for the same instructions.
#include "fq_host.h"
#include "w4_linear.h"
#include "w4_tile.h"

namespace fqw {
namespace {

struct DxArgs {
    const uint16_t* dy;  // [m] rows, ld apart, of `cols` columns: n, or two runs of `run` >= n for a pair of weights
    int64_t ld, cols, run;
    W4Mat w[2];
    uint16_t* dx;
    int64_t m, n, k;
    uint32_t ni, nj;
};
template <class T>
struct DwArgs {
    const uint16_t* dy;  // as above
    const uint16_t* x;   // [m] rows of k columns, ldx apart
    int64_t ld, cols, run, ldx;
    T* dw[2];
    int64_t m, n, k;
    uint32_t ni, nj;
};

// The weights' side of a tile, 64 rows by BN columns: a thread holds 32 codes of a row.
template <int BN, bool ZP>
struct CodeSteps {
    static constexpr int kParts = BN / 32;
    const DxArgs& a;
    int64_t byte, gi;
    int line, part;
    u32x4 c;
    float s, z;
    __device__ __forceinline__ CodeSteps(const DxArgs& a_, int64_t col0, int t) : a(a_), line(t / kParts), part(t % kParts) {
        const int64_t col = col0 + 32 * part;
        byte = col / 2;
        gi = (col < a.k ? col : a.k - 1) / a.w[0].group;
    }
    __device__ __forceinline__ void load(int64_t l0) {
        const int which = l0 >= a.run;  // a step lies in one of the matrices
        const W4Mat& w = a.w[which];
        const int64_t r = l0 - (which ? a.run : 0) + line, at = r < a.n ? r : a.n - 1;
        c = load16_part(w.codes + at * w.row_bytes + byte, (a.n - at) * w.row_bytes - byte);
        s = r < a.n ? w.scale[at * w.ng + gi] * 16.0f : 0.0f;
        if constexpr (ZP) z = w.zp ? (float)w.zp[at * w.ng + gi] * 0.0625f : 0.0f;
        else z = 0.0f;
    }
    __device__ __forceinline__ void store(uint16_t* tile) const {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<bf16x8*>(tile + line * BN + by_steps(4 * part + j, line) * 8) = weights_bf16<ZP>(c[j], z, s);
    }
};

// A tile's sums to rows i0 .. of a matrix of k columns.  Lanes hold one row each and
// runs of four columns: they meet in LDS, so that memory sees whole rows.
template <class S, class T, class Row>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[S::MS][S::NS], T* lds, int64_t j0, int64_t k, Row row) {
    constexpr int kPasses = sizeof(T) / 2, kRows = S::BM / kPasses, kPitch = S::BN + 16 / sizeof(T);
    constexpr int kVec = 16 / sizeof(T), kWide = S::BN / kVec;
    static_assert(kPasses == 1 || kPasses == S::WM, "a pass takes whole waves");
    const int t = threadIdx.x, lane = t % 64, wave = t / 64;
    const int wi = wave / S::WN * (S::MS * 32), wj = wave % S::WN * (S::NS * 32);
    const bool whole = k % kVec == 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        if (p) __syncthreads();
        if (kPasses == 1 || wave / S::WN == p)
#pragma unroll
            for (int i = 0; i < S::MS; ++i)
#pragma unroll
                for (int j = 0; j < S::NS; ++j)
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        T* d = lds + (wi - p * kRows + 32 * i + lane % 32) * kPitch + wj + 32 * j + 2 * e + 4 * (lane / 32);
#pragma unroll
                        for (int f = 0; f < 4; ++f) store_f(d + f, acc[i][j][e + f]);
                    }
        __syncthreads();
        for (int v = t; v < kRows * kWide; v += S::kThreads) {
            const int r = v / kWide, c = v % kWide * kVec;
            T* out = row(p * kRows + r);
            if (!out || j0 + c >= k) continue;
            const T* s = lds + r * kPitch + c;
            if (whole) *reinterpret_cast<u32x4*>(out + j0 + c) = *reinterpret_cast<const u32x4*>(s);
            else
                for (int f = 0; f < kVec; ++f)
                    if (j0 + c + f < k) out[j0 + c + f] = s[f];
        }
    }
}

template <class S, class T>
struct TileLds {
    union {
        struct {
            __attribute__((aligned(1024))) uint16_t a[2][S::BM * kDeep], b[2][S::BN * kDeep];
        };
        T out[S::BM * 2 / sizeof(T) * (S::BN + 16 / sizeof(T))];
    };
};

template <class S, bool ZP>
__global__ __launch_bounds__(S::kThreads, 2) void k_dx(DxArgs a) {
    __shared__ TileLds<S, uint16_t> lds;
    const int t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
    uint32_t ti, tj;
    tile_at(blockIdx.x, a.ni, a.nj, ti, tj);
    const int64_t i0 = (int64_t)ti * S::BM, j0 = (int64_t)tj * S::BN;
    const DenseRows<S::BM, S::kThreads> ys(a.dy, i0, a.m, a.ld, a.cols, wave, lane);
    CodeSteps<S::BN, ZP> ws(a, j0, t);
    const int wi = wave / S::WN * (S::MS * 32), wj = wave % S::WN * (S::NS * 32);
    const uint32_t steps = (uint32_t)((a.cols + kDeep - 1) / kDeep);

    f32x16 acc[S::MS][S::NS] = {};
    ws.load(0);
    ws.store(lds.b[0]);
    ys.fill(lds.a[0], 0);
    if (1 < steps) ws.load(kDeep);
    wait_dma();
    __syncthreads();
    for (uint32_t st = 0; st < steps; ++st) {
        const int cur = st & 1;
        if (st + 1 < steps) {
            ws.store(lds.b[cur ^ 1]);
            ys.fill(lds.a[cur ^ 1], (int64_t)(st + 1) * kDeep);
            if (st + 2 < steps) ws.load((int64_t)(st + 2) * kDeep);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            bf16x8 f[S::MS], b[S::NS];
#pragma unroll
            for (int j = 0; j < S::NS; ++j) b[j] = frag_steps<S::BN>(lds.b[cur], wj + 32 * j, d, lane);
#pragma unroll
            for (int i = 0; i < S::MS; ++i) f[i] = frag_rows(lds.a[cur], wi + 32 * i, d, lane);
#pragma unroll
            for (int i = 0; i < S::MS; ++i)
#pragma unroll
                for (int j = 0; j < S::NS; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], f[i], acc[i][j], 0, 0, 0);
        }
        wait_dma();
        __syncthreads();
    }
    store_tile<S>(acc, lds.out, j0, a.k, [&](int r) { return i0 + r < a.m ? a.dx + (i0 + r) * a.k : nullptr; });
}

template <class S, class T>
__global__ __launch_bounds__(S::kThreads, 2) void k_dw(DwArgs<T> a) {
    __shared__ TileLds<S, T> lds;
    const int t = threadIdx.x, lane = t % 64, wave = __builtin_amdgcn_readfirstlane(t / 64);
    uint32_t ti, tj;
    tile_at(blockIdx.x, a.ni, a.nj, ti, tj);
    const int64_t i0 = (int64_t)ti * S::BM, j0 = (int64_t)tj * S::BN;
    const DenseSteps<S::BM, S::kThreads> ys(a.dy, i0, a.cols, a.m, a.ld, wave, lane);
    const DenseSteps<S::BN, S::kThreads> xs(a.x, j0, a.ldx, a.m, a.ldx, wave, lane);
    const int wi = wave / S::WN * (S::MS * 32), wj = wave % S::WN * (S::NS * 32);
    const uint32_t steps = (uint32_t)((a.m + kDeep - 1) / kDeep);

    f32x16 acc[S::MS][S::NS] = {};
    ys.fill(lds.a[0], 0);
    xs.fill(lds.b[0], 0);
    wait_dma();
    __syncthreads();
    for (uint32_t st = 0; st < steps; ++st) {
        const int cur = st & 1;
        if (st + 1 < steps) {
            ys.fill(lds.a[cur ^ 1], (int64_t)(st + 1) * kDeep);
            xs.fill(lds.b[cur ^ 1], (int64_t)(st + 1) * kDeep);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            bf16x8 f[S::MS], b[S::NS];
#pragma unroll
            for (int j = 0; j < S::NS; ++j) b[j] = frag_steps<S::BN>(lds.b[cur], wj + 32 * j, d, lane);
#pragma unroll
            for (int i = 0; i < S::MS; ++i) f[i] = frag_steps<S::BM>(lds.a[cur], wi + 32 * i, d, lane);
#pragma unroll
            for (int i = 0; i < S::MS; ++i)
#pragma unroll
                for (int j = 0; j < S::NS; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], f[i], acc[i][j], 0, 0, 0);
        }
        wait_dma();
        __syncthreads();
    }
    store_tile<S>(acc, lds.out, j0, a.k, [&](int r) -> T* {
        const int64_t i = i0 + r, f = i < a.run ? i : i - a.run;
        return i < a.cols && f < a.n ? a.dw[i < a.run ? 0 : 1] + f * a.k : nullptr;
    });
}

// dg and du beside each other: out [m][2 run], zeros in columns n .. run - 1 of each half.
__global__ __launch_bounds__(256) void k_gate_grad(const uint16_t* dh, const uint16_t* g, const uint16_t* u, int act,
                                                   int64_t m, int64_t n, int64_t run, uint16_t* out) {
    const int64_t chunks = run / 8;
    for (int64_t v = blockIdx.x * 256ll + threadIdx.x; v < m * chunks; v += gridDim.x * 256ll) {
        const int64_t r = v / chunks, c = v % chunks * 8, at = r * n + c;
        Tokens<uint16_t> td, tg, tu;
        td.load_part(dh + at, n - c), tg.load_part(g + at, n - c), tu.load_part(u + at, n - c);
        bf16x8 d[1], gg[1], uu[1], dg, du;
        td.parts(d), tg.parts(gg), tu.parts(uu);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float value, slope;
            const float di = (float)d[0][i];
            act_both(act, (float)gg[0][i], value, slope);
            dg[i] = (__bf16)(di * (float)uu[0][i] * slope);
            du[i] = (__bf16)(di * value);
        }
        *reinterpret_cast<bf16x8*>(out + r * 2 * run + c) = dg;
        *reinterpret_cast<bf16x8*>(out + r * 2 * run + run + c) = du;
    }
}

// Rows of `cols` elements to rows of ld (a multiple of 8), zeros after.
__global__ __launch_bounds__(256) void k_pad_rows(const uint16_t* in, int64_t rows, int64_t cols, int64_t ld,
                                                  uint16_t* out) {
    const int64_t chunks = ld / 8;
    for (int64_t v = blockIdx.x * 256ll + threadIdx.x; v < rows * chunks; v += gridDim.x * 256ll) {
        const int64_t r = v / chunks, c = v % chunks * 8;
        Tokens<uint16_t> f;
        f.load_part(in + r * cols + c, cols - c);
        *reinterpret_cast<u32x4*>(out + r * ld + c) = f.v;
    }
}

int64_t padded(int64_t c, int64_t to) { return (c + to - 1) / to * to; }

// The matrix itself, or a copy at `at` with rows of whole 16-byte chunks (`at` moves past it).
const uint16_t* chunk_rows(const void* p, int64_t rows, int64_t cols, char*& at, hipStream_t stream) {
    if (cols % 8 == 0) return (const uint16_t*)p;
    const int64_t ld = padded(cols, 8);
    uint16_t* out = (uint16_t*)at;
    k_pad_rows<<<fqh::grid_all(rows * ld / 8, 256), 256, 0, stream>>>((const uint16_t*)p, rows, cols, ld, out);
    at += rows * ld * 2;
    return out;
}

template <class S>
int launch_dx(DxArgs a, bool zp, hipStream_t stream) {
    const int64_t ni = (a.m + S::BM - 1) / S::BM, nj = (a.k + S::BN - 1) / S::BN;
    if (ni * nj > 0x7FFFFFFF) return FQ_E_UNSUPPORTED;
    a.ni = (uint32_t)ni, a.nj = (uint32_t)nj;
    const dim3 g((unsigned)(ni * nj)), b(S::kThreads);
    if (zp) k_dx<S, true><<<g, b, 0, stream>>>(a);
    else k_dx<S, false><<<g, b, 0, stream>>>(a);
    return fqh::launched();
}
template <class S, class T>
int launch_dw(DwArgs<T> a, hipStream_t stream) {
    const int64_t ni = (a.cols + S::BM - 1) / S::BM, nj = (a.k + S::BN - 1) / S::BN;
    if (ni * nj > 0x7FFFFFFF) return FQ_E_UNSUPPORTED;
    a.ni = (uint32_t)ni, a.nj = (uint32_t)nj;
    k_dw<S, T><<<dim3((unsigned)(ni * nj)), dim3(S::kThreads), 0, stream>>>(a);
    return fqh::launched();
}

using Big = Shape<256, 256, 2, 4>;
using Small = Shape<128, 128, 2, 2>;
bool big_tiles(int64_t rows, int64_t cols) { return ((rows + 255) / 256) * ((cols + 255) / 256) >= fqh::num_cus() / 2; }

int products(const DxArgs& dx, const uint16_t* x, int64_t ldx, void* dw, void* dw2, int dw_dtype, hipStream_t stream) {
    if (dx.dx) {
        const bool zp = dx.w[0].zp || dx.w[1].zp;
        const int st = big_tiles(dx.m, dx.k) ? launch_dx<Big>(dx, zp, stream) : launch_dx<Small>(dx, zp, stream);
        if (st != FQ_OK || !dw) return st;
    }
    const bool big = big_tiles(dx.cols, dx.k);
    if (dw_dtype == FQ_F32) {
        const DwArgs<float> a{dx.dy, x, dx.ld, dx.cols, dx.run, ldx, {(float*)dw, (float*)dw2}, dx.m, dx.n, dx.k};
        return big ? launch_dw<Big>(a, stream) : launch_dw<Small>(a, stream);
    }
    const DwArgs<uint16_t> a{dx.dy, x, dx.ld, dx.cols, dx.run, ldx, {(uint16_t*)dw, (uint16_t*)dw2}, dx.m, dx.n, dx.k};
    return big ? launch_dw<Big>(a, stream) : launch_dw<Small>(a, stream);
}

}  // namespace

size_t backward_workspace(int64_t m, int64_t n, int64_t k, bool gated) {
    const int64_t a = gated ? 2 * padded(n, kDeep) : n % 8 ? padded(n, 8) : 0, b = k % 8 ? padded(k, 8) : 0;
    return (size_t)(m * (a + b) * 2);
}

int matmul_backward(const void* dy, const void* x, int64_t m, int64_t n, int64_t k, int64_t group, const fql_w4* w,
                    void* dx, void* dw, int dw_dtype, void* workspace, hipStream_t stream) {
    char* at = (char*)workspace;
    const uint16_t* y = chunk_rows(dy, m, n, at, stream);
    const W4Mat wm = dx ? w4_mat(*w, k, group) : W4Mat{};
    const int64_t ld = padded(n, 8);
    return products({y, ld, ld, padded(n, kDeep), {wm, wm}, (uint16_t*)dx, m, n, k},
                    dw ? chunk_rows(x, m, k, at, stream) : nullptr, padded(k, 8), dw, nullptr, dw_dtype, stream);
}

int gated_backward(const void* dh, const void* x, const void* g, const void* u, int64_t m, int64_t n, int64_t k,
                   int64_t group, int act, const fql_w4* gate, const fql_w4* up, void* dx, void* dw_gate, void* dw_up,
                   int dw_dtype, void* workspace, hipStream_t stream) {
    const int64_t run = padded(n, kDeep);
    uint16_t* both = (uint16_t*)workspace;
    char* at = (char*)(both + m * 2 * run);
    k_gate_grad<<<fqh::grid_all(m * run / 8, 256), 256, 0, stream>>>((const uint16_t*)dh, (const uint16_t*)g,
                                                                     (const uint16_t*)u, act, m, n, run, both);
    DxArgs a{both, 2 * run, 2 * run, run, {}, (uint16_t*)dx, m, n, k};
    if (dx) a.w[0] = w4_mat(*gate, k, group), a.w[1] = w4_mat(*up, k, group);
    return products(a, dw_gate ? chunk_rows(x, m, k, at, stream) : nullptr, padded(k, 8), dw_gate, dw_up, dw_dtype,
                    stream);
}

}  // namespace fqw
