// What the kernels over paged private caches share: the arguments of a call,
// which sequence a row belongs to, which keys it sees, and what its scores go
// through.
#pragma once

#include <cuda_bf16.h>
#include <limits.h>
#include <math_constants.h>

#include "kvpool_internal.cuh"
#include "tc_ptx.cuh"

namespace kvp {

constexpr int kPagedDevices = 64;  // devices of a process that the paged calls may run on

// Bits of kvpool_pages_t.status.
enum : int { kPgBadPage = 1, kPgTimeout = 2 };

// The pages of one layer and the sequences of one call.
struct PagedSeqs {
    int pages, Hk, pshift;  // page_tokens = 1 << pshift
    int seqs, tstride, tokens;
    const int32_t* table;
    const int32_t* kv_len;
    const int32_t* q_start;
    int* status;
};

struct PagedAttend {
    PagedSeqs s;
    const uint16_t* K;  // bf16 [pages][Hk][page_tokens][D] of the layer
    const uint16_t* V;
    const uint16_t* Q;  // bf16, q_stride elements per token
    long long q_stride;
    int Hq, G;
    uint32_t g_magic;      // 2^32 / G, rounded up (see div_group)
    float scale_log2;      // softmax scale * log2(e)
    float cap2, cap_in;    // cap * log2(e); 2 * log2(e) * softmax scale / cap
    float cap_z, cap_near; // softmax scale / cap; the products up to which tanh is a polynomial
    float cap_q[5];        // its coefficients times scale_log2
    const float* slopes;
    int window;
    const int32_t* first;
    const int32_t* prefix;
    uint16_t* out;         // bf16 [tokens][Hq][D]
    float* lse;            // [tokens][Hq] or null
    // instead of out and lse, the rows' states for a merge with the shared
    // pool: unnormalised accumulators f32 [tokens][Hq][D] and (m, l), m in log2
    // units, in slices of st_tokens tokens (the last one shorter), each
    // [Hk][slice tokens * G][2]
    float* st_acc;
    float* st_ml;
    int st_tokens;
};

// tanh(z) = z (1 + z^2 q(z^2)) for |z| <= 0.7 within 2.3e-8 relative: q's coefficients.
constexpr float kTanh[5] = {-0.333331913f, 0.13329111f, -0.05355886f, 0.0200919714f, -0.00513866264f};

// Does any score modifier apply (else the causal mask alone, which the plain
// instances of the kernels handle).
inline bool paged_scored(const PagedAttend& a) {
    return a.cap2 > 0.0f || a.slopes || a.window > 0 || a.first || a.prefix;
}

cudaError_t launch_pages_append(const PagedSeqs& s, int head_dim, uint16_t* Kp, uint16_t* Vp, const void* K,
                                long long k_stride, const void* V, long long v_stride, cudaStream_t st);
// The two kinds of attention (pages_rows.cu: few rows per sequence;
// pages_chunk.cu: many); max_q, max_kv as in kvpool_seqs_t, but never 0.
cudaError_t launch_pages_rows(const PagedAttend& a, int head_dim, int max_q, int max_kv, int sm_count,
                              cudaStream_t st);
// What both entry points that attend over pages check and hand on: `a` without
// its outputs; hints of 0 replaced.
int paged_attend_args(const kvpool_pages_t* pg, int layer, const kvpool_seqs_t* seqs, const void* Q,
                      long long q_stride, int q_heads, const kvpool_score_t* score, float softmax_scale, PagedAttend& a,
                      int& max_q, int& max_kv);
// Chooses the kernel; sm_count of the current (sm_103) device.
cudaError_t launch_pages_attend(const PagedAttend& a, int head_dim, int max_q, int max_kv, int sm_count,
                                cudaStream_t st);
cudaError_t launch_pages_chunk(const PagedAttend& a, int head_dim, int max_q, int max_kv, cudaStream_t st);

namespace pages {

__device__ __forceinline__ float bf2f(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }

__device__ __forceinline__ void flag(int* status, int bit) {
    if (status) atomicOr(status, bit);
}

// First row of sequence i: entry i of q_start, held inside [0, tokens].
__device__ __forceinline__ int row_begin(const PagedSeqs& s, int i) { return min(max(__ldg(s.q_start + i), 0), s.tokens); }

// Tokens that sequence i holds by its length, and those that its table has room for.
__device__ __forceinline__ int length_of(const PagedSeqs& s, int i) { return max(__ldg(s.kv_len + i), 0); }
__device__ __forceinline__ int held_tokens(const PagedSeqs& s, int length) {
    return (int)min((long long)length, (long long)s.tstride << s.pshift);
}

// The rows of all sequences cut into blocks of RB rows (a row: a new token and
// one of the G query heads of a KV head; a block holds rows of one sequence).
// Block z: its sequence, its number there, the sequence's first token row q0,
// new tokens n, the first one's position p0 (the others follow) and held tokens
// T: a sequence longer than its table has room for holds the tokens that fit,
// and is recorded. False past the last block. Whole warps call it; 32 sequences
// at a time, their loads independent of one another.
struct RowBlock {
    int seq, blk, q0, n, p0, T;
};
__device__ __forceinline__ bool find_block(const PagedSeqs& s, int G, int RB, int z, RowBlock& b) {
    const int lane = threadIdx.x & 31;
    int before = 0;  // blocks of the sequences before these 32
    for (int base = 0; base < s.seqs; base += 32) {
        const int i = base + lane;
        int q0 = 0, n = 0, len = 0;
        if (i < s.seqs) {
            q0 = row_begin(s, i);
            n = max(row_begin(s, i + 1) - q0, 0);
            len = length_of(s, i);
        }
        const int nb = (int)(((long long)n * G + RB - 1) / RB);
        int sum = nb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + sum > z);
        if (past) {
            const int l = __ffs(past) - 1;
            b.seq = base + l;
            b.q0 = __shfl_sync(0xffffffffu, q0, l);
            b.n = __shfl_sync(0xffffffffu, n, l);
            len = __shfl_sync(0xffffffffu, len, l);
            b.p0 = len - b.n;
            b.T = held_tokens(s, len);
            if (len > b.T && lane == 0) flag(s.status, kPgBadPage);
            b.blk = z - before - __shfl_sync(0xffffffffu, sum - nb, l);
            return true;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return false;
}

// x / G for x G < 2^32: the product's excess over x / G is below x G / 2^32 of a G-th.
__device__ __forceinline__ int div_group(const PagedAttend& a, int x) {
    return a.G == 1 ? x : (int)__umulhi((uint32_t)x, a.g_magic);
}

// The keys a row sees: [a1, b1) and [a2, b2) (overlapping or empty as may be).
struct Seen {
    int a1, b1, a2, b2;
    __device__ __forceinline__ bool has(int j) const { return (j >= a1 && j < b1) || (j >= a2 && j < b2); }
    // every key of [u0, u1)
    __device__ __forceinline__ bool all(int u0, int u1) const {
        return (a1 <= u0 && b1 >= u1) || (a2 <= u0 && b2 >= u1);
    }
    // any key of [u0, u1)
    __device__ __forceinline__ bool some(int u0, int u1) const {
        return max(a1, u0) < min(b1, u1) || max(a2, u0) < min(b2, u1);
    }
    __device__ __forceinline__ int lo() const { return min(b1 > a1 ? a1 : INT_MAX, b2 > a2 ? a2 : INT_MAX); }
    __device__ __forceinline__ int prefix_end() const { return b2 > a2 ? b2 : 0; }
    __device__ __forceinline__ int window_lo() const { return b1 > a1 ? a1 : INT_MAX; }
    __device__ __forceinline__ int hi() const { return max(b1 > a1 ? b1 : 0, b2 > a2 ? b2 : 0); }
};
// Row `tok` (of the call) at position pos of sequence seq, which holds T tokens.
template <bool SCORED>
__device__ __forceinline__ Seen row_seen(const PagedAttend& a, int seq, int tok, int pos, int T) {
    Seen r;
    r.a1 = 0;
    r.b1 = min(pos + 1, T);
    r.a2 = r.b2 = 0;
    if constexpr (SCORED) {
        const int first = a.first ? max(__ldg(a.first + tok), 0) : 0;
        r.a1 = a.window > 0 ? (int)max((long long)pos - a.window + 1, (long long)first) : first;
        if (a.prefix) {
            r.a2 = first;
            r.b2 = min(__ldg(a.prefix + seq), T);
        }
    }
    return r;
}

// Units (or tiles) of keys, counted without those between a prefix and the
// windows behind it, which no row of a block sees: unit u of the count is
// number u + len of the sequence from `at` on.
struct Gap {
    int at, len;
    // prefix_end: the last end of a part [a2, b2) of the block's rows, 0 for none;
    // window_lo: the first begin of a part [a1, b1), INT_MAX for none
    __device__ __forceinline__ Gap(int prefix_end, int window_lo, int unit) {
        at = (prefix_end + unit - 1) / unit;
        len = prefix_end > 0 && window_lo < INT_MAX ? max(window_lo / unit - at, 0) : 0;
    }
    __device__ __forceinline__ Gap() : at(0), len(0) {}
    __device__ __forceinline__ int number(int u) const { return u >= at ? u + len : u; }
    __device__ __forceinline__ int count(int n) const { return n > at ? max(n - len, at) : n; }  // of numbers below n
};

// Where the state (m, l) of token row t and query head hd goes.
__device__ __forceinline__ float2* state_ml(const PagedAttend& a, int t, int hd) {
    const int sl = t / a.st_tokens, tl = t - sl * a.st_tokens, g = hd / a.G;
    const int in = min(a.st_tokens, a.s.tokens - sl * a.st_tokens);  // tokens of the slice
    return reinterpret_cast<float2*>(a.st_ml) + (long long)sl * a.st_tokens * a.G * a.s.Hk +
           ((long long)g * in + tl) * a.G + (hd - g * a.G);
}

// <q, k> -> the score in log2 units, of one key and of 32. The cap's tanh(z):
// up to |z| = 0.7 a polynomial, z + z^3 q(z^2), q fitted to tanh's least largest
// relative error (2.2e-8), so that scores far below the cap keep float32's
// relative precision; beyond, 1 - 2 / (e^(2z) + 1), off by a few units of 2^-24,
// which the cap turns into cap * 2^-22 of a score that is at least 0.6 cap (the
// reciprocal of an overflowed e^(2z) is 0, as it should be). 32 keys take the
// polynomial where all of a warp's are near (no exponential and no reciprocal
// per key), else the other form, whose error is the same part of the cap: 2^-16
// nats at most for caps up to 64. With wider ones (WIDE) each key takes its own.
constexpr float kWideCap2 = 64.0f * 1.4426950408889634f;
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float capped(const PagedAttend& a, float s) {
    const float z = s * a.cap_z, u = z * z;
    float q = fmaf(u, a.cap_q[4], a.cap_q[3]);
    q = fmaf(u, q, a.cap_q[2]), q = fmaf(u, q, a.cap_q[1]), q = fmaf(u, q, a.cap_q[0]);
    const float far = fmaf(-2.0f * a.cap2, rcp(ptx::ex2(s * a.cap_in) + 1.0f), a.cap2);
    return fabsf(s) <= a.cap_near ? s * fmaf(u, q, a.scale_log2) : far;
}
template <bool SCORED>
__device__ __forceinline__ float score(const PagedAttend& a, float s, float slope2, int pos, int j) {
    s = !SCORED || !(a.cap2 > 0.0f) ? s * a.scale_log2 : capped(a, s);
    if (SCORED && a.slopes) s = fmaf(-slope2, fabsf((float)(pos - j)), s);
    return s;
}
// The scores of 32 keys. behind: no key lies behind the row's position, so the
// distance to key j0 joins the constant and each key costs one more step. live:
// the row is one (which form a warp's tanh takes is for its rows to say).
template <bool WIDE>
__device__ __forceinline__ void scores32(const PagedAttend& a, float (&x)[32], float slope2, int pos, int j0,
                                         bool behind, bool live) {
    const float far = (float)(pos - j0), base = a.slopes && behind ? -slope2 * far : 0.0f;
    auto near = [&] {  // (a NaN is passed over, and stays one in either form)
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < 32; k += 2) most = ptx::max3(most, fabsf(x[k]), fabsf(x[k + 1]));
        return __all_sync(0xffffffffu, !live || most <= a.cap_near);
    };
    if (!(a.cap2 > 0.0f)) {
        const float2 f = make_float2(a.scale_log2, a.scale_log2), c = make_float2(base, base);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const float2 y = __ffma2_rn(make_float2(x[k], x[k + 1]), f, c);
            x[k] = y.x, x[k + 1] = y.y;
        }
    } else if (near()) {
        auto both = [](float v) { return make_float2(v, v); };
        const float2 cz = both(a.cap_z), f = both(a.scale_log2), c = both(base);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const float2 s = make_float2(x[k], x[k + 1]), z = __fmul2_rn(s, cz), u = __fmul2_rn(z, z);
            float2 q = __ffma2_rn(u, both(a.cap_q[4]), both(a.cap_q[3]));
            q = __ffma2_rn(u, q, both(a.cap_q[2]));
            q = __ffma2_rn(u, q, both(a.cap_q[1]));
            q = __ffma2_rn(u, q, both(a.cap_q[0]));
            const float2 y = __ffma2_rn(s, __ffma2_rn(u, q, f), c);
            x[k] = y.x, x[k + 1] = y.y;
        }
    } else if constexpr (WIDE) {
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = capped(a, x[k]) + base;
    } else {
        const float2 in = make_float2(a.cap_in, a.cap_in), one = make_float2(1.0f, 1.0f);
        const float2 f = make_float2(-2.0f * a.cap2, -2.0f * a.cap2), c = make_float2(a.cap2 + base, a.cap2 + base);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            float2 y = __fmul2_rn(make_float2(x[k], x[k + 1]), in);
            y = __fadd2_rn(make_float2(ptx::ex2(y.x), ptx::ex2(y.y)), one);
            y = __ffma2_rn(make_float2(rcp(y.x), rcp(y.y)), f, c);
            x[k] = y.x, x[k + 1] = y.y;
        }
    }
    if (!a.slopes) return;
    if (behind) {
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = fmaf(slope2, (float)k, x[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = fmaf(-slope2, fabsf(far - (float)k), x[k]);
    }
}

// One row over the keys it sees in the units [u0, u1) of 2^sh keys, counted
// without the gap, every us-th one, with nothing that it does not see
// touching the result: the slow path of rows whose sums came out infinite or NaN, which a matrix product
// gives for 0 * NaN where a masked key's V is not finite. One warp; lane holds
// D / 32 consecutive channels of acc.
template <int D, bool SCORED>
__device__ __noinline__ void careful_row(const PagedAttend& a, int seq, int tok, int head, int pos, const Seen& see,
                                         const Gap gap, int sh, int u0, int u1, int us, float& m, float& l,
                                         float (&acc)[D / 32]) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const PagedSeqs& s = a.s;
    const int g = head / a.G;
    const float slope2 = SCORED && a.slopes ? a.slopes[head] * 1.4426950408889634f : 0.0f;
    float q[E];
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = bf2f(a.Q[(long long)tok * a.q_stride + (long long)head * D + lane * E + e]);
    m = -CUDART_INF_F;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    // (a sum that is NaN stays NaN, and with it the row)
    for (int k = 0; l == l && (u0 + (k >> sh) * us) < u1; ++k) {
        const int j = (gap.number(u0 + (k >> sh) * us) << sh) + (k & ((1 << sh) - 1));
        if (!see.has(j)) continue;
        const int page = __ldg(s.table + (long long)seq * s.tstride + (j >> s.pshift));
        const bool ok = page >= 0 && page < s.pages;
        const long long at =
            ((((long long)(ok ? page : 0) * s.Hk + g) << s.pshift) + (j & ((1 << s.pshift) - 1))) * D + lane * E;
        float dot = 0.0f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            dot = fmaf(q[e], ok ? bf2f(a.K[at + e]) : 0.0f, dot);
            v[e] = ok ? bf2f(a.V[at + e]) : 0.0f;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float x = score<SCORED>(a, dot, slope2, pos, j);
        const float mn = fmaxf(m, x), ref = mn == -CUDART_INF_F ? 0.0f : mn;
        const float c = l == 0.0f ? 0.0f : ptx::ex2(m - ref), w = ptx::ex2(x - ref);
        l = l == 0.0f ? w : fmaf(l, c, w);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[e], acc[e] * c);
        m = mn;
    }
    if (m == -CUDART_INF_F && l != 0.0f) m = 0.0f;  // NaN scores alone: keep them
    if (l == 0.0f) m = -CUDART_INF_F;
}

}  // namespace pages
}  // namespace kvp
