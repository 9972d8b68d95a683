// w4_few.hip -- products of few token rows (up to 64) with 4-bit group-quantized
// weights: y = x W^T and the gated block, for single-token serving and small batches.
//
// What bounds it: the codes, k / 2 bytes per row of W, read once; at 64 tokens
// still only 256 products per byte.  A workgroup owns 16 NT rows of W (of both
// weights for the gated block) and its waves deal the row's 128-column steps
// among them, so a 4096 x 4096 weight spreads over all 256 compute units with
// every load in flight at once; the waves' partial sums meet in LDS in wave order.
#include "fq_host.h"
#include "w4_mfma.h"
#include "w4_linear.h"

namespace fqw {
namespace {

constexpr int kFewWaves = 8;
constexpr int kAhead = 4;  // steps whose codes a wave loads before it uses the first

template <class T>
struct FewArgs {
    const T* x;
    W4Mat w[2];
    T *out[3];  // y, or h, g, u
    int64_t m, n, k;
    uint32_t spans, per_group;  // spans in a row, spans in a group
    int act;
};

template <class T, int MT, int NT, int SPAN, bool ZP, int W>
struct FewWave {
    static constexpr int kTiles = NT * W, kSums = kStep / SPAN;
    const FewArgs<T>& a;
    int64_t n0;
    int lane, row, q;
    f32x4 acc[MT][kTiles];

    struct Codes {
        u32x4 c[kTiles];
        float s[kTiles][kSums], z[kTiles][kSums];
    };

    __device__ __forceinline__ int64_t wrow(int t) const {
        const int64_t r = n0 + 16 * (t % NT) + row;
        return r < a.n ? r : a.n - 1;
    }
    // group of span number s of a row (a span past the row's end belongs to its last group)
    __device__ __forceinline__ uint32_t group_of(uint32_t s) const {
        s = s < a.spans ? s : a.spans - 1;
        return a.per_group == 1 ? s : s / a.per_group;
    }
    __device__ __forceinline__ void fetch(Codes& d, int64_t step, bool whole) const {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const W4Mat& w = a.w[t / NT];
            const int64_t r = wrow(t), b = step * (kStep / 2) + q * 16;
            const uint8_t* p = w.codes + r * w.row_bytes + b;
            d.c[t] = whole ? load16(p) : load16_part(p, (a.n - r) * w.row_bytes - b);  // codes past the row's end meet zeros
#pragma unroll
            for (int i = 0; i < kSums; ++i) {
                const int64_t g = r * w.ng + group_of((uint32_t)step * kSums + i);
                d.s[t][i] = w.scale[g] * 16.0f;
                if constexpr (ZP) d.z[t][i] = w.zp ? (float)w.zp[g] * 0.0625f : 0.0f;
                else d.z[t][i] = 0.0f;
            }
        }
    }
    __device__ __forceinline__ void tokens(TokenFrag<T>& f, int mt, int j, int64_t step, bool whole) const {
        const int64_t r = 16 * mt + row;
        const T* p = a.x + (r < a.m ? r : a.m - 1) * a.k;
        const int64_t c = step * kStep + (SPAN == 128 ? 32 * q + 8 * j : 32 * j + 8 * q);
        if (whole) f.load(p + c);
        else f.load_part(p + c, (int)(a.k - c < 8 ? a.k - c : 8));
    }
    __device__ __forceinline__ void use(const Codes& d, int64_t step, bool whole) {
        u32x4 c[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) c[t] = SPAN == 128 ? d.c[t] : transpose_quarters(d.c[t]);
#pragma unroll
        for (int i = 0; i < kSums; ++i) {
            f32x4 part[MT][kTiles];
#pragma unroll
            for (int j = 0; j < SPAN / 32; ++j) {
                bf16x8 b[kTiles];
#pragma unroll
                for (int t = 0; t < kTiles; ++t) b[t] = codes_bf16<ZP>(c[t][i * (SPAN / 32) + j], d.z[t][i]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    TokenFrag<T> f;
                    tokens(f, mt, i * (SPAN / 32) + j, step, whole);
#pragma unroll
                    for (int p = 0; p < TokenFrag<T>::kParts; ++p)
#pragma unroll
                        for (int t = 0; t < kTiles; ++t)
                            part[mt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                f.p[p], b[t], j || p ? part[mt][t] : f32x4{0, 0, 0, 0}, 0, 0, 0);
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[mt][t][e] = fmaf(part[mt][t][e], d.s[t][i], acc[mt][t][e]);
        }
    }
};

// W = 1: y = x W^T.  W = 2: w[0] is the gate, w[1] the up matrix.
template <class T, int MT, int NT, int SPAN, bool ZP, int W>
__global__ __launch_bounds__(64 * kFewWaves) void k_few(FewArgs<T> a) {
    using Wave = FewWave<T, MT, NT, SPAN, ZP, W>;
    constexpr int kTiles = Wave::kTiles;
    __shared__ f32x4 sums[kFewWaves][MT * kTiles][64];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    Wave v{a, (int64_t)blockIdx.x * 16 * NT, lane, lane % 16, lane / 16, {}};
    const int64_t full = a.k / kStep;
    for (int64_t s = wave; s < full; s += kFewWaves * kAhead) {
        typename Wave::Codes d[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (s + i * kFewWaves < full) v.fetch(d[i], s + i * kFewWaves, true);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (s + i * kFewWaves < full) v.use(d[i], s + i * kFewWaves, true);
    }
    if (full * kStep < a.k && full % kFewWaves == wave) {  // the row's last, short step
        typename Wave::Codes d;
        v.fetch(d, full, false);
        v.use(d, full, false);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) sums[wave][mt * kTiles + t][lane] = v.acc[mt][t];
    __syncthreads();
    for (int o = wave; o < MT * NT; o += kFewWaves) {
        const int mt = o / NT, nt = o % NT;
        const int64_t c = v.n0 + 16 * nt + v.row;
        f32x4 r[W];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            r[w] = sums[0][mt * kTiles + w * NT + nt][lane];
            for (int i = 1; i < kFewWaves; ++i) r[w] += sums[i][mt * kTiles + w * NT + nt][lane];
        }
        if (c >= a.n) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t i = 16 * mt + 4 * v.q + e;
            if (i >= a.m) continue;
            const int64_t at = i * a.n + c;
            if constexpr (W == 1) {
                store_f(a.out[0] + at, r[0][e]);
            } else {
                store_f(a.out[0] + at, act_value(a.act, r[0][e]) * r[W - 1][e]);
                if (a.out[1]) {
                    store_f(a.out[1] + at, r[0][e]);
                    store_f(a.out[2] + at, r[W - 1][e]);
                }
            }
        }
    }
}

template <class T, int MT, int NT, int W>
int launch(const FewArgs<T>& a, int span, hipStream_t stream) {
    const int64_t blocks = (a.n + 16 * NT - 1) / (16 * NT);
    if (blocks > 0x7FFFFFFF) return FQ_E_UNSUPPORTED;
    const bool zp = a.w[0].zp || (W == 2 && a.w[1].zp);
    const dim3 g((unsigned)blocks), b(64 * kFewWaves);
    if (span == 128) zp ? k_few<T, MT, NT, 128, true, W><<<g, b, 0, stream>>>(a) : k_few<T, MT, NT, 128, false, W><<<g, b, 0, stream>>>(a);
    else if (span == 64) zp ? k_few<T, MT, NT, 64, true, W><<<g, b, 0, stream>>>(a) : k_few<T, MT, NT, 64, false, W><<<g, b, 0, stream>>>(a);
    else zp ? k_few<T, MT, NT, 32, true, W><<<g, b, 0, stream>>>(a) : k_few<T, MT, NT, 32, false, W><<<g, b, 0, stream>>>(a);
    return fqh::launched();
}

template <class T, int W>
int few(const FewArgs<T>& a, int span, hipStream_t stream) {
    if (a.m <= 16) return launch<T, 1, 1, W>(a, span, stream);
    if (a.m <= 32) return launch<T, 2, 1, W>(a, span, stream);
    return launch<T, 4, 1, W>(a, span, stream);
}

}  // namespace

int few_matmul(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, const fql_w4& w, void* y,
               hipStream_t stream) {
    const int span = span_of(group, k);
    const uint32_t spans = (uint32_t)((k + span - 1) / span), per = spans_per_group(group, k, span);
    const W4Mat wm = w4_mat(w, k, group);
    if (dtype == FQ_F32) return few<float, 1>({(const float*)x, {wm, wm}, {(float*)y}, m, n, k, spans, per, 0}, span, stream);
    return few<uint16_t, 1>({(const uint16_t*)x, {wm, wm}, {(uint16_t*)y}, m, n, k, spans, per, 0}, span, stream);
}

int few_gated(const void* x, int dtype, int64_t m, int64_t n, int64_t k, int64_t group, int act, const fql_w4& gate,
              const fql_w4& up, void* h, void* g, void* u, hipStream_t stream) {
    const int span = span_of(group, k);
    const uint32_t spans = (uint32_t)((k + span - 1) / span), per = spans_per_group(group, k, span);
    const W4Mat wg = w4_mat(gate, k, group), wu = w4_mat(up, k, group);
    if (dtype == FQ_F32)
        return few<float, 2>({(const float*)x, {wg, wu}, {(float*)h, (float*)g, (float*)u}, m, n, k, spans, per, act}, span, stream);
    return few<uint16_t, 2>({(const uint16_t*)x, {wg, wu}, {(uint16_t*)h, (uint16_t*)g, (uint16_t*)u}, m, n, k, spans, per, act}, span,
                            stream);
}

}  // namespace fqw
