// The paged private caches held in 4 bits: what their kernels share.
//
// A head-vector x of D channels is held as D / 8 words of eight codes u and a
// float32 scale t, and stands for t H (u - 7.5), H the Walsh-Hadamard matrix in
// Sylvester's order. Word w holds channels 8 w ... 8 w + 7 of y = H x: channel
// 8 w + 2 k in bits 4 k ... 4 k + 3, channel 8 w + 2 k + 1 sixteen bits above,
// so that one mask leaves two neighbouring channels as the halves of a register.
#pragma once

#include <cuda_fp16.h>

#include "pages.cuh"

namespace kvp {

// The best step of a uniform quantiser of 16 levels for N(0, 1) (J. Max, Quantizing for minimum distortion, IRE
// Transactions on Information Theory 6, 1960, table II): mean square error 0.01154.
constexpr float kStep4 = 0.3352f;

// Position rotation of the new tokens (kvpool_rotary_t).
struct Rotary {
    const float* cos;  // [positions][half]; null: none
    const float* sin;
    const int32_t* at;
    int positions, half, interleaved, offset;
};

struct AppendArgs {
    PagedSeqs s;
    Rotary r;
    const uint16_t* K;
    const uint16_t* V;
    const uint16_t* Q;  // null: none
    uint16_t* Q_out;
    long long k_stride, v_stride, q_stride, q_out_stride;
    int Hq;
    // the layer's pages: bf16 values, or codes and scales
    uint16_t* Kp;
    uint16_t* Vp;
    uint32_t* Kc;
    uint32_t* Vc;
    float* Kt;
    float* Vt;
};

// Attention over codes: PagedAttend's K and V are the layer's code words.
struct PagedAttend4 {
    PagedAttend a;
    const float* Kt;
    const float* Vt;
};

cudaError_t launch_append(const AppendArgs& a, int head_dim, bool four, cudaStream_t st);
cudaError_t launch_pages4_read(const PagedSeqs& s, int head_dim, const uint32_t* Kc, const uint32_t* Vc, const float* Kt,
                               const float* Vt, uint16_t* K, uint16_t* V, cudaStream_t st);
// The two kinds of attention, as of the bf16 pages (pages4_rows.cu, pages4_chunk.cu).
cudaError_t launch_pages4_rows(const PagedAttend4& a, int head_dim, int max_q, int max_kv, int sm_count,
                               cudaStream_t st);
// (ws: memory for tiles made of codes once per call, or null; sequences that it has no room for go without)
long long pages4_chunk_ws_bytes(const PagedSeqs& s, int head_dim, int max_kv);
cudaError_t launch_pages4_chunk(const PagedAttend4& a, int head_dim, int max_q, int max_kv, void* ws, size_t ws_bytes,
                                cudaStream_t st);

// Checks that the entries of the bf16 pages and of the 4-bit pages share.
int check_pages_args(const kvpool_pages_t* pg, int layer);
int check_seqs_args(const kvpool_seqs_t* s);
int check_sm103(int& sms);
int check_copy_args(const kvpool_pages_t* pg, const int32_t* src, const int32_t* dst, int n);
int append_args(const kvpool_pages_t* pg, const kvpool_seqs_t* seqs, const kvpool_rotary_t* rotary, const void* K,
                long long k_stride, const void* V, long long v_stride, const void* Q, long long q_stride, int q_heads,
                void* Q_out, long long q_out_stride, AppendArgs& a);
int pages_status(int32_t* status, void* stream);
// Pages of `pieces` 16-byte pieces, of K and of V, in every layer.
cudaError_t copy_pages(void* K, void* V, int layers, int pages, int pieces, const int32_t* src, const int32_t* dst, int n,
                       cudaStream_t st);
PagedSeqs paged_seqs_view(const kvpool_pages_t* pg, const kvpool_seqs_t* s);

namespace pages {

// Butterflies of the transform over a row that lies in 4 consecutive channels
// per lane, D / 4 lanes.
template <int D>
__device__ __forceinline__ void transform4(float4& a) {
    const float s = a.x + a.y, d = a.x - a.y, u = a.z + a.w, v = a.z - a.w;
    a = make_float4(s + u, d + v, s - u, d - v);
#pragma unroll
    for (int o = 1; o < D / 4; o <<= 1) {
        const float g = threadIdx.x & o ? -1.0f : 1.0f;
        a.x = fmaf(g, a.x, __shfl_xor_sync(0xffffffffu, a.x, o));
        a.y = fmaf(g, a.y, __shfl_xor_sync(0xffffffffu, a.y, o));
        a.z = fmaf(g, a.z, __shfl_xor_sync(0xffffffffu, a.z, o));
        a.w = fmaf(g, a.w, __shfl_xor_sync(0xffffffffu, a.w, o));
    }
}
// The same with a whole warp to a row, D / 32 consecutive channels per lane.
template <int D>
__device__ __forceinline__ void transform_row(float (&a)[D / 32]) {
    constexpr int E = D / 32;
#pragma unroll
    for (int h = 1; h < E; h <<= 1)
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (!(i & h)) {
                const float x = a[i], y = a[i + h];
                a[i] = x + y, a[i + h] = x - y;
            }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float g = threadIdx.x & o ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] = fmaf(g, a[i], __shfl_xor_sync(0xffffffffu, a[i], o));
    }
}

// careful_row over codes: one row over the keys it sees in the units [u0, u1) of
// 2^sh keys, counted without the gap, every us-th one. acc: the sum of p t (u -
// 7.5), not yet transformed.
template <int D, bool SCORED>
__device__ __noinline__ void careful_row4(const PagedAttend4& p4, int seq, int tok, int head, int pos, const Seen& see,
                                          const Gap gap, int sh, int u0, int u1, int us, float& m, float& l,
                                          float (&acc)[D / 32]) {
    constexpr int E = D / 32;  // channels per lane: of a word, E / 2 of its four places in both halves
    const PagedAttend& a = p4.a;
    const int lane = threadIdx.x & 31;
    const PagedSeqs& s = a.s;
    const int g = head / a.G;
    const float slope2 = SCORED && a.slopes ? a.slopes[head] * 1.4426950408889634f : 0.0f;
    float q[E];
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = bf2f(a.Q[(long long)tok * a.q_stride + (long long)head * D + lane * E + e]);
    // a power of two brings the row's largest value into [1/2, 1), so that neither H q nor its products overflow
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(fabsf(q[e])));
    const int e2 = min(max((int)(__reduce_max_sync(0xffffffffu, top) >> 23) - 126, -126), 126);
    const float down = __uint_as_float((uint32_t)(127 - e2) << 23), up = __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] *= down;
    transform_row<D>(q);
    m = -CUDART_INF_F;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    auto level = [&](uint32_t w, int e) {  // of channel lane * E + e
        const int c = (lane * E + e) & 7;
        return (float)(w >> (4 * (c >> 1) + 16 * (c & 1)) & 15) - 7.5f;
    };
    // (a sum that is NaN stays NaN, and with it the row)
    for (int k = 0; l == l && (u0 + (k >> sh) * us) < u1; ++k) {
        const int j = (gap.number(u0 + (k >> sh) * us) << sh) + (k & ((1 << sh) - 1));
        if (!see.has(j)) continue;
        const int page = __ldg(s.table + (long long)seq * s.tstride + (j >> s.pshift));
        const bool ok = page >= 0 && page < s.pages;
        const long long vec = (((long long)(ok ? page : 0) * s.Hk + g) << s.pshift) + (j & ((1 << s.pshift) - 1));
        const long long at = vec * (D / 8) + lane * E / 8;
        const uint32_t kw = __ldg(reinterpret_cast<const uint32_t*>(a.K) + at);
        const uint32_t vw = __ldg(reinterpret_cast<const uint32_t*>(a.V) + at);
        const float tk = ok ? __ldg(p4.Kt + vec) : 0.0f, tv = ok ? __ldg(p4.Vt + vec) : 0.0f;
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) dot = fmaf(q[e], level(kw, e), dot);
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float x = score<SCORED>(a, dot * (tk * up), slope2, pos, j);
        const float mn = fmaxf(m, x), ref = mn == -CUDART_INF_F ? 0.0f : mn;
        const float c = l == 0.0f ? 0.0f : ptx::ex2(m - ref), w = ptx::ex2(x - ref);
        l = l == 0.0f ? w : fmaf(l, c, w);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w * tv, level(vw, e), acc[e] * c);
        m = mn;
    }
    if (m == -CUDART_INF_F && l != 0.0f) m = 0.0f;  // NaN scores alone: keep them
    if (l == 0.0f) m = -CUDART_INF_F;
}

}  // namespace pages
}  // namespace kvp
