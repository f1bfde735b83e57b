// New tokens on their way into the pages: K and Q turned by their positions,
// and K and V written as bf16 or in 4 bits; and the way back, tokens of the
// 4-bit pages as bf16.
//
// Mathematics. Rotation: a pair (a, b) of channels becomes (a c - b s, b c + a s),
// two float32 products and their sum, each rounded once (no FMA: the same
// numbers whoever adds them up), then one rounding to bf16 or none before the
// codes. Codes: y = H x, step = 0.3352 |x|, u = clamp(floor(y / step) + 8, 0, 15),
// t = step / D; x is first scaled by a power of two that brings its largest
// value into [1/2, 1), so that neither squares nor sums overflow.
//
// Bound: memory, each byte once. A block takes one token; D / 16 lanes take a
// head-vector, each lane two pieces of 8 channels that lie D / 2 apart: the
// pairs (i, i + D / 2) are then in one lane, a lane's angles serve all heads, and
// of the transform's log2 D stages four stay in registers.
// Measured: 17 thousand tokens of 32 query heads on 8 of 128, half of the channels
// turned, 576 MB in 99 us (5.8 TB/s); into 4 bits with 64 query heads, 620 MB in
// 115 us; 15 tokens in 3 us of a captured graph. Blocks of 256 threads leave a
// token's tail of heads idle (124 us), of 64 take 97 but 3.8 us for the 15 tokens.
#include "pages4.cuh"

namespace kvp {
namespace {

constexpr int kAppThreads = 128;

// How a call's rotation meets a lane's channels: none; pairs (i, i + D / 2), both
// in the lane; pairs elsewhere or fewer channels.
enum { kNoTurn, kWhole, kPart };

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    auto two = [](float lo, float hi) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    };
    return make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
}
// a c - b s and b c + a s
__device__ __forceinline__ float turn_a(float a, float b, float c, float s) {
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) {
    return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// The angles of one piece of 8 channels, p-th of its head: eight for pairs of
// which the piece has one end (the other `reach` pieces on, or back), four for
// neighbouring pairs.
struct Angles {
    float c[8], s[8];
    int reach;  // 0: the piece does not turn, or pairs are neighbours
    bool turns;
    __device__ __forceinline__ void load(const Rotary& r, int at, int p) {
        turns = 8 * p < 2 * r.half;
        reach = 0;
        if (!turns) return;
        const long long row = (long long)at * r.half;
        int i = 4 * p;
        if (!r.interleaved) {
            const int n = r.half / 8;
            reach = p < n ? n : -n;
            i = 8 * (p < n ? p : p - n);
        }
        const float4 *c4 = reinterpret_cast<const float4*>(r.cos + row + i), *s4 = reinterpret_cast<const float4*>(r.sin + row + i);
        *reinterpret_cast<float4*>(c) = __ldg(c4);
        *reinterpret_cast<float4*>(s) = __ldg(s4);
        if (!r.interleaved) {
            *reinterpret_cast<float4*>(c + 4) = __ldg(c4 + 1);
            *reinterpret_cast<float4*>(s + 4) = __ldg(s4 + 1);
        }
    }
    // src: the piece in memory
    __device__ __forceinline__ void turn(float (&x)[8], const uint4* src) const {
        if (!turns) return;
        if (reach == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = turn_a(a, b, c[i], s[i]);
                x[2 * i + 1] = turn_b(a, b, c[i], s[i]);
            }
        } else {
            float y[8];
            unpack8(src[reach], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = reach > 0 ? turn_a(x[i], y[i], c[i], s[i]) : turn_b(y[i], x[i], c[i], s[i]);
        }
    }
};

// Codes of a head-vector spread over its L lanes, which all come here with all
// lanes of the warp: words j and j + L, and the scale.
template <int L>
__device__ __forceinline__ void encode(float (&x0)[8], float (&x1)[8], uint32_t& w0, uint32_t& w1, float& t) {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, max(__float_as_uint(fabsf(x0[i])), __float_as_uint(fabsf(x1[i]))));
#pragma unroll
    for (int o = 1; o < L; o <<= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
    const int e = min(max((int)(top >> 23) - 126, -126), 126);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    float q0[8], q1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x0[i] = __fmul_rn(x0[i], down), x1[i] = __fmul_rn(x1[i], down);
        q0[i] = __fmul_rn(x0[i], x0[i]), q1[i] = __fmul_rn(x1[i], x1[i]);
    }
    // squares in neighbouring pairs: within the pieces, over the lanes, over the halves
#pragma unroll
    for (int n = 4; n; n >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) q0[i] = __fadd_rn(q0[2 * i], q0[2 * i + 1]), q1[i] = __fadd_rn(q1[2 * i], q1[2 * i + 1]);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        q0[0] = __fadd_rn(q0[0], __shfl_xor_sync(kAll, q0[0], o));
        q1[0] = __fadd_rn(q1[0], __shfl_xor_sync(kAll, q1[0], o));
    }
    const float step = __fmul_rn(kStep4, __fsqrt_rn(__fadd_rn(q0[0], q1[0])));
    // the transform: stages 1, 2, 4 in the pieces, then over the lanes, then over the halves
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & h)) {
                float a = x0[i], b = x0[i + h];
                x0[i] = __fadd_rn(a, b), x0[i + h] = __fsub_rn(a, b);
                a = x1[i], b = x1[i + h];
                x1[i] = __fadd_rn(a, b), x1[i + h] = __fsub_rn(a, b);
            }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = __shfl_xor_sync(kAll, x0[i], o), b = __shfl_xor_sync(kAll, x1[i], o);
            x0[i] = upper ? __fsub_rn(a, x0[i]) : __fadd_rn(a, x0[i]);
            x1[i] = upper ? __fsub_rn(b, x1[i]) : __fadd_rn(b, x1[i]);
        }
    }
    const float inv = __fdiv_rn(1.0f, step);
    w0 = w1 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = __fadd_rn(x0[i], x1[i]), b = __fsub_rn(x0[i], x1[i]);
        const int u0 = min(max(__float2int_rd(__fmul_rn(a, inv)), -8), 7) + 8;
        const int u1 = min(max(__float2int_rd(__fmul_rn(b, inv)), -8), 7) + 8;
        w0 |= (uint32_t)u0 << (2 * (i & 6) + 16 * (i & 1));
        w1 |= (uint32_t)u1 << (2 * (i & 6) + 16 * (i & 1));
    }
    if (!(step > 0.0f)) w0 = w1 = 0x88888888u;
    // a vector that holds an infinity or NaN stands for NaN
    t = top >= 0x7F800000u ? CUDART_NAN_F
                           : __fmul_rn(__fmul_rn(step, 1.0f / (16 * L)), __uint_as_float((uint32_t)(127 + e) << 23));
}

// The token row `tok`: its sequence, position and, where the table has a page
// for it, the index of its first head's vector in the layer (-1 where not).
// False: a row behind the last sequence, or a position before 0.
__device__ __forceinline__ bool place_of(const PagedSeqs& s, int tok, int& pos, long long& vec) {
    pages::RowBlock b;
    if (!pages::find_block(s, 1, 1, tok, b)) return false;
    // blocks of one row each are numbered over the sequences' rows alone; rows that belong to
    // nobody lie behind them, so the block's row is the token (q_start ascending from 0, as documented)
    pos = b.p0 + b.blk;
    if (pos < 0 || b.q0 + b.blk != tok) return false;
    vec = -1;
    if (pos >= b.T) return true;  // no room in the table (recorded by find_block)
    const int page = __ldg(s.table + (long long)b.seq * s.tstride + (pos >> s.pshift));
    if (page < 0 || page >= s.pages) {
        if ((threadIdx.x & 31) == 0) pages::flag(s.status, kPgBadPage);
        return true;
    }
    vec = (((long long)page * s.Hk) << s.pshift) + (pos & ((1 << s.pshift) - 1));
    return true;
}

template <int D, bool FOUR, int TURN>
__global__ void __launch_bounds__(kAppThreads)
append_kernel(const AppendArgs a) {
    constexpr int L = D / 16, kSlots = kAppThreads / L;
    const PagedSeqs& s = a.s;
    const int tok = blockIdx.x, slot = threadIdx.x / L, j = threadIdx.x % L;
    // head-vector v of the token: K's heads, then V's
    auto kv = [&](int v) {
        const bool k = v < s.Hk;
        return reinterpret_cast<const uint4*>((k ? a.K + tok * a.k_stride + (long long)v * D
                                                 : a.V + tok * a.v_stride + (long long)(v - s.Hk) * D)) + j;
    };
    auto qh = [&](int h) { return reinterpret_cast<const uint4*>(a.Q + tok * a.q_stride + (long long)h * D) + j; };
    // the first vectors are asked for before the lookups that say where they go have come back
    uint4 p0 = {}, p1 = {}, r0 = {}, r1 = {};
    if (slot < 2 * s.Hk) p0 = kv(slot)[0], p1 = kv(slot)[L];
    const int hq = TURN != kNoTurn && a.Q ? a.Hq : 0;
    if (slot < hq) r0 = qh(slot)[0], r1 = qh(slot)[L];
    int pos;
    long long vec;
    if (!place_of(s, tok, pos, vec)) return;
    Angles a0, a1;
    if constexpr (TURN != kNoTurn) {
        const long long at = a.r.at ? __ldg(a.r.at + tok) : (long long)a.r.offset + pos;
        if (at < 0 || at >= a.r.positions) {  // nothing is written for it
            if (threadIdx.x == 0) pages::flag(s.status, kPgBadPosition);
            return;
        }
        a0.load(a.r, (int)at, j);
        if constexpr (TURN == kPart) a1.load(a.r, (int)at, j + L);
    }
    auto turned = [&](float (&x0)[8], float (&x1)[8], const uint4* src) {
        if constexpr (TURN == kWhole) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = x0[i], q = x1[i];
                x0[i] = turn_a(p, q, a0.c[i], a0.s[i]);
                x1[i] = turn_b(p, q, a0.c[i], a0.s[i]);
            }
        } else if constexpr (TURN == kPart) {
            a0.turn(x0, src);
            a1.turn(x1, src + L);
        }
    };
    // (the loops' bounds are the same for all lanes: encode takes whole warps)
    if (vec >= 0) {
        for (int v0 = 0; v0 < 2 * s.Hk; v0 += kSlots) {
            const int v = v0 + slot;
            const bool mine = v < 2 * s.Hk;
            if (v0 > 0 && mine) p0 = kv(v)[0], p1 = kv(v)[L];
            const bool k = v < s.Hk;
            const long long at = vec + ((long long)(k ? v : v - s.Hk) << s.pshift);
            if constexpr (FOUR) {
                float x0[8], x1[8];
                unpack8(p0, x0);
                unpack8(p1, x1);
                if (mine && k) turned(x0, x1, kv(v));
                uint32_t w0, w1;
                float t;
                encode<L>(x0, x1, w0, w1, t);
                if (mine) {
                    uint32_t* to = (k ? a.Kc : a.Vc) + at * (D / 8) + j;
                    to[0] = w0, to[L] = w1;
                    if (j == 0) (k ? a.Kt : a.Vt)[at] = t;
                }
            } else if (mine) {
                if (k) {
                    float x0[8], x1[8];
                    unpack8(p0, x0);
                    unpack8(p1, x1);
                    turned(x0, x1, kv(v));
                    p0 = pack8(x0), p1 = pack8(x1);
                }
                uint4* to = reinterpret_cast<uint4*>((k ? a.Kp : a.Vp) + at * D) + j;
                to[0] = p0, to[L] = p1;
            }
        }
    }
    if constexpr (TURN != kNoTurn) {
        for (int h0 = 0; h0 < hq; h0 += kSlots) {
            const int h = h0 + slot;
            const bool mine = h < hq;
            if (h0 > 0 && mine) r0 = qh(h)[0], r1 = qh(h)[L];
            float x0[8], x1[8];
            unpack8(r0, x0);
            unpack8(r1, x1);
            if (mine) turned(x0, x1, qh(h));
            if constexpr (TURN == kPart) __syncwarp();  // Q_out may be Q: its pieces are read before any is written
            if (mine) {
                uint4* to = reinterpret_cast<uint4*>(a.Q_out + tok * a.q_out_stride + (long long)h * D) + j;
                to[0] = pack8(x0), to[L] = pack8(x1);
            }
        }
    }
}

// Tokens of the 4-bit pages as bf16 rows: t H (u - 7.5) = t (H (u - 8) + (D / 2)
// e_0). The sums are whole numbers up to 8 D + D / 2, exact in fp16 in any order,
// two to a register; one rounding to float32 with t, one to bf16. A warp takes a
// token, its D / 16 lanes a head-vector, several of them asked for at once.
// Bound: the instructions beside memory: 42,600 tokens of 8 KV heads, 316 MB in 63 us
// (5.0 TB/s) with 86 % of the issue slots taken (butterflies in packed halves 55 % of
// their pipe, masks and packing 59 % of theirs). A block per token, sums in float32: 111.
constexpr int kReadWarps = 4, kReadAhead = 4;

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
// the eight u - 8 of a word, neighbouring channels in a register
__device__ __forceinline__ void levels(uint32_t w, __half2 (&x)[4]) {
    const __half2 even = as_half2(0xE408E408u), odd = as_half2(0xD480D480u), part = as_half2(0x2C002C00u);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t v = k ? w >> 8 : w;
        x[2 * k] = __hadd2(as_half2((v & 0x000F000Fu) | 0x64006400u), even);             // 1024 + u - 1032
        x[2 * k + 1] = __hfma2(as_half2((v & 0x00F000F0u) | 0x64006400u), part, odd);  // (1024 + 16 u) / 16 - 72
    }
}

template <int D>
__global__ void __launch_bounds__(kReadWarps * 32)
read_kernel(const PagedSeqs s, const uint32_t* __restrict__ Kc, const uint32_t* __restrict__ Vc,
            const float* __restrict__ Kt, const float* __restrict__ Vt, uint16_t* __restrict__ K,
            uint16_t* __restrict__ V) {
    constexpr int L = D / 16, kVectors = 32 / L;  // lanes of a vector, vectors of a warp at a time
    const int tok = blockIdx.x * kReadWarps + threadIdx.x / 32, lane = threadIdx.x & 31, j = lane % L;
    if (tok >= s.tokens) return;
    int pos;
    long long vec;
    if (!place_of(s, tok, pos, vec)) return;
    const __half2 first = j == 0 ? __floats2half2_rn(D / 2, 0.0f) : __floats2half2_rn(0.0f, 0.0f);
    const __half2 turn = __floats2half2_rn(1.0f, -1.0f);
    for (int v0 = lane / L; v0 - lane / L < 2 * s.Hk; v0 += kVectors * kReadAhead) {
        uint32_t w0[kReadAhead], w1[kReadAhead];
        float t[kReadAhead];
#pragma unroll
        for (int u = 0; u < kReadAhead; ++u) {
            const int v = v0 + kVectors * u;
            w0[u] = w1[u] = 0x88888888u;  // (tokens without a page: zeros)
            t[u] = 0.0f;
            if (v < 2 * s.Hk && vec >= 0) {
                const bool k = v < s.Hk;
                const long long at = vec + ((long long)(k ? v : v - s.Hk) << s.pshift);
                const uint32_t* from = (k ? Kc : Vc) + at * (D / 8) + j;
                w0[u] = __ldg(from), w1[u] = __ldg(from + L), t[u] = __ldg((k ? Kt : Vt) + at);
            }
        }
#pragma unroll
        for (int u = 0; u < kReadAhead; ++u) {
            const int v = v0 + kVectors * u;
            if (v - lane / L >= 2 * s.Hk) break;  // (the whole warp's)
            __half2 x[8], a[4], c[4];  // channels 8 j ..., and D / 2 further on
            levels(w0[u], a);
            levels(w1[u], c);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __hadd2(a[i], c[i]), x[4 + i] = __hsub2(a[i], c[i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __hfma2(x[i], turn, __lowhigh2highlow(x[i]));  // neighbours
#pragma unroll
            for (int h = 1; h < 4; h <<= 1)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (!(i & h)) {
                        const __half2 p = x[i], q = x[i + h];
                        x[i] = __hadd2(p, q), x[i + h] = __hsub2(p, q);
                    }
#pragma unroll
            for (int o = 1; o < L; o <<= 1) {
                const __half2 sign = lane & o ? __floats2half2_rn(-1.0f, -1.0f) : __floats2half2_rn(1.0f, 1.0f);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = __hfma2(x[i], sign, as_half2(__shfl_xor_sync(0xffffffffu, as_bits(x[i]), o)));
            }
            x[0] = __hadd2(x[0], first);
            if (v < 2 * s.Hk) {
                const bool k = v < s.Hk;
                uint4* to = reinterpret_cast<uint4*>((k ? K : V) + ((long long)tok * s.Hk + (k ? v : v - s.Hk)) * D) + j;
                float y[8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 z = __half22float2(x[4 * i + e]);
                        // (a page that is not there reads as zeros whatever the sum)
                        y[2 * e] = z.x * t[u], y[2 * e + 1] = z.y * t[u];
                    }
                    to[i * L] = pack8(y);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int head_dim, bool four, cudaStream_t st) {
    const int turn = !a.r.cos ? kNoTurn : !a.r.interleaved && 2 * a.r.half == head_dim ? kWhole : kPart;
#define KVP_APPEND(DD, FF, TT) append_kernel<DD, FF, TT><<<a.s.tokens, kAppThreads, 0, st>>>(a)
#define KVP_APPEND_D(FF, TT) (head_dim == 64 ? KVP_APPEND(64, FF, TT) : KVP_APPEND(128, FF, TT))
    if (four) {
        if (turn == kNoTurn) KVP_APPEND_D(true, kNoTurn);
        else if (turn == kWhole) KVP_APPEND_D(true, kWhole);
        else KVP_APPEND_D(true, kPart);
    } else {
        if (turn == kWhole) KVP_APPEND_D(false, kWhole);
        else KVP_APPEND_D(false, kPart);
    }
#undef KVP_APPEND_D
#undef KVP_APPEND
    return cudaGetLastError();
}

cudaError_t launch_pages4_read(const PagedSeqs& s, int head_dim, const uint32_t* Kc, const uint32_t* Vc, const float* Kt,
                               const float* Vt, uint16_t* K, uint16_t* V, cudaStream_t st) {
    const int grid = (s.tokens + kReadWarps - 1) / kReadWarps;
    if (head_dim == 64) read_kernel<64><<<grid, kReadWarps * 32, 0, st>>>(s, Kc, Vc, Kt, Vt, K, V);
    else read_kernel<128><<<grid, kReadWarps * 32, 0, st>>>(s, Kc, Vc, Kt, Vt, K, V);
    return cudaGetLastError();
}

}  // namespace kvp
