// Attention of few query rows per sequence over its pages in 4 bits: decode
// steps, draft tokens.
//
// Mathematics: a key stands for t H c with c = u - 7.5 of its codes, so that
// <q, k> = t <H q, c>, and a row's sum of weighted values is H (sum p t' c'): the
// rows are transformed once at the start, the sums once at the end, and between
// them the matrix products see codes alone. One pass over the keys with a
// running reference m per row, p = 2^(x - m), O and l rescaled when a score
// passes m by more than 2^8. The weights p t' are rounded to bf16 (off by at
// most 2^-8 of each, as the output's own rounding is of it), H q to two fp16
// parts (a power of two has brought the row's largest value into [1/2, 1)). One
// part alone, off by 2^-11, leaves the log of the sum 1e-6 off (relative) where
// 16K keys weigh alike, but 1e-4 where a window, a document or a peaked row leaves
// few keys that count, at any length; the second costs 32 sequences of 32K keys
// 8 % (250 us against 230). With both the log of the sum is within 3e-7 of its size
// in all of these. Codes enter the products exactly: of Q K^T as fp16 u - 8 or 16
// (u - 8) (one mask and one addition; the sixteenth is in that channel's H q, the
// other half of a step is the product's first summand), of P V as bf16 u - 7.5.
//
// Bound: memory, as a step reads D + 8 bytes per key and KV head, and before it the
// instructions that make operands of codes, so the layout serves these. The keys
// are the matrix product's 16 rows and the query rows its 8 columns: each code is
// taken apart once for up to 8 NR query rows, a lane's 16 bytes of a key are its
// operands of all steps over the channels (they are summed, so any order does),
// and the weights turn into the second product's operand by a transpose of 8 x 8
// registers. A CTA has up to 8 NR rows (new tokens x heads of a group) of one
// sequence and KV head; its 4 warps take units of 32 keys in turn, each through a
// ring of its own in shared memory, filled by 16-byte asynchronous copies that
// nothing but the warp itself waits for. The warps' states meet in shared memory at
// the end, those of a cluster's CTAs, which split the keys, in distributed shared
// memory: no workspace, no second launch.
//
// Measured: 32 sequences of 32K keys, 64 query heads on 8 of 128: 250 us, 4.4 TB/s
// of 6.8 (the bf16 pages, 3.8 times the bytes, take 570); without its loads the
// kernel takes 40 us less, without what takes V's codes apart 51, without the
// matrix instructions of Q K^T 75, with one fp16 part of H q 19: a mixture of the
// half-rate integer pipe, the matrix instructions' chains and the issue slots. 5
// tokens of one sequence of 20,011 keys, 28 heads on 4: 26 us, of which a start of
// 1.6 us and a cluster's merge of 3.5 are fixed. Not kept (each against the version
// of its time): 5 or 6 CTAs per SM with two units in a ring (315, 376 us against
// 294), 3 with four (325), blocks of 32 rows (spills; 43 us against 25 on those 5
// tokens), CTAs of 8 warps, shifts by multiplication (326 against 301).
#include <algorithm>
#include <mutex>

#include "pages4.cuh"

namespace kvp {
namespace {

using pages::Seen;

constexpr int kWarps = 4;
constexpr int kUnit = 32;   // keys per unit
constexpr int kStages = 3;  // units in a warp's ring
constexpr float kLazyMax = 8.0f;
constexpr int kMaxSplit = 16;
constexpr int kWave = 100;  // what a wave of CTAs costs beside its units, in units of an SM
// CTAs per SM, by their registers: 8 and 16 rows
constexpr int ctas_per_sm(int NR) { return NR == 1 ? 4 : 3; }

template <int D, int NR>
struct Lay {
    static constexpr int codes = kUnit * D / 2;              // bytes of a unit's K or V
    static constexpr int stage = 2 * codes + 2 * kUnit * 4;  // K, V, their scales
    static constexpr int ring = kWarps * kStages * stage;
    static constexpr int rs = D + 4;                         // floats of a merge row: O, m, l
    static constexpr int rows = 8 * NR;
    // the merge reuses the rings: per warp `rows` rows, then the CTA's merged ones
    static constexpr int merge = (kWarps + 1) * rows * rs * 4;
    // H q as the lanes' operands of every step, 16 bytes each: high and low parts; then 2 floats per row
    static constexpr int q = ring > merge ? ring : merge, steps = D / 16;
    static constexpr int info = q + NR * steps * 512;
    static constexpr int total = info + rows * 8;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// c += A (16 keys x 16 channels) B (16 channels x 8 rows)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the 8 x 8 matrix of 16-bit values that the warp's registers hold, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// (x & mask) | bits in one instruction
__device__ __forceinline__ uint32_t mask_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
    return y;
}
// codes in bits 1-4 of both halves -> bf16 u - 7.5, exactly
__device__ __forceinline__ uint32_t centred(uint32_t x) {
    const uint32_t y = mask_or(x, 0x001E001Eu, 0x42804280u);  // 64 + u
    uint32_t z;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(y), "r"(0xC28FC28Fu));  // - 71.5
    return z;
}

// codes under the mask -> fp16 1024 + u (or 1024 + 16 u) less 1032 (1152), exactly
__device__ __forceinline__ uint32_t half_centred(uint32_t x, uint32_t mask, uint32_t less) {
    const uint32_t y = mask_or(x, mask, 0x64006400u);
    uint32_t z;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(z) : "r"(y), "r"(less));
    return z;
}

// NR: blocks of 8 query rows. SCORED: score modifiers apply. DIRECT: every
// sequence has one block (no search; if it has more, the CTA takes them in
// turn). Grid: blocks x the CTAs of a cluster, KV heads.
template <int D, int NR, bool SCORED, bool DIRECT>
__global__ void __launch_bounds__(kWarps * 32, ctas_per_sm(NR))
pages4_rows_kernel(const PagedAttend4 p4) {
    using L = Lay<D, NR>;
    constexpr int kRows = L::rows;
    constexpr int KS = D / 16;   // steps of Q K^T over the channels
    constexpr int MB = D / 16;   // blocks of 16 channels of P V
    constexpr int W = D / 32;    // words of a key per lane in Q K^T
    constexpr int RS = L::rs;
    const PagedAttend& p = p4.a;
    extern __shared__ __align__(128) unsigned char sm[];
    const PagedSeqs& s = p.s;
    const int S = (int)ptx::cluster_size(), rank = (int)ptx::cluster_rank();
    const int g = blockIdx.y;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const int quad = lane >> 2, qi = lane & 3;

    pages::RowBlock b;
    if constexpr (DIRECT) {
        b.seq = blockIdx.x / S;
        b.blk = 0;
        b.q0 = pages::row_begin(s, b.seq);
        b.n = max(pages::row_begin(s, b.seq + 1) - b.q0, 0);
        const int len = pages::length_of(s, b.seq);
        b.p0 = len - b.n;
        b.T = pages::held_tokens(s, len);
        if (b.n == 0) return;  // the whole cluster's
        if (len > b.T && tid == 0) pages::flag(s.status, kPgBadPage);
    } else {
        if (!pages::find_block(s, p.G, kRows, blockIdx.x / S, b)) return;
    }
    const int T = b.T;
    const int32_t* table = s.table + (long long)b.seq * s.tstride;

    for (;; ++b.blk) {
        const int r_begin = b.blk * kRows;
        const int nr = min(kRows, b.n * p.G - r_begin);
        auto token_of = [&](int r) { return (r_begin + r) / p.G; };
        auto head_of = [&](int r) { return g * p.G + (r_begin + r) % p.G; };

        // H q of the block's rows in two fp16 parts (rows past it repeat its last), half a step's share and the power of two
        for (int r = warp; r < kRows; r += kWarps) {
            const int rr = min(r, nr - 1);
            const uint16_t* src = p.Q + (long long)(b.q0 + token_of(rr)) * p.q_stride + (long long)head_of(rr) * D;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (lane < D / 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + lane);
                x = make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                                __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
            }
            uint32_t top = max(max(__float_as_uint(fabsf(x.x)), __float_as_uint(fabsf(x.y))),
                               max(__float_as_uint(fabsf(x.z)), __float_as_uint(fabsf(x.w))));
            top = __reduce_max_sync(0xffffffffu, top);
            const int e = min(max((int)(top >> 23) - 126, -126), 126);
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
            x.x *= down, x.y *= down, x.z *= down, x.w *= down;
            pages::transform4<D>(x);
            float sum = (x.x + x.y) + (x.z + x.w);
            // channels 4 l + 2 and + 3 meet 16 (u - 8)
            x.z *= 0.0625f, x.w *= 0.0625f;
            const __half2 h0 = __floats2half2_rn(x.x, x.y), h1 = __floats2half2_rn(x.z, x.w);
            const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
            const __half2 l0 = __floats2half2_rn(x.x - f0.x, x.y - f0.y), l1 = __floats2half2_rn(x.z - f1.x, x.w - f1.y);
#pragma unroll
            for (int o = D / 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            auto bits = [](const __half2& h) { return *reinterpret_cast<const uint32_t*>(&h); };
            if (lane < D / 4)  // step lane % KS of the quarter-row lane / KS
                *reinterpret_cast<uint4*>(sm + L::q + (((r >> 3) * KS + lane % KS) * 32 + (r & 7) * 4 + lane / KS) * 16) =
                    make_uint4(bits(h0), bits(h1), bits(l0), bits(l1));
            if (lane == 0)
                *reinterpret_cast<float2*>(sm + L::info + r * 8) =
                    make_float2(0.5f * sum, __uint_as_float((uint32_t)(127 + e) << 23));
        }
        __syncthreads();
        float off[NR][2], mul[NR][2];  // of this lane's rows 8 n + 2 qi + h
        Seen see[NR][2];
        int pos[NR][2];
        float slope2[NR][2];
        int lo = INT_MAX, hi = 0, pre_end = 0, win_lo = INT_MAX;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 8 * n + 2 * qi + h, rr = min(r, nr - 1);
                const float2 c = *reinterpret_cast<const float2*>(sm + L::info + r * 8);
                off[n][h] = c.x;
                mul[n][h] = c.y * (SCORED ? 1.0f : p.scale_log2);
                const int i = token_of(rr);
                pos[n][h] = b.p0 + i;
                see[n][h] = pages::row_seen<SCORED>(p, b.seq, b.q0 + i, pos[n][h], T);
                slope2[n][h] = SCORED && p.slopes ? __ldg(p.slopes + head_of(rr)) * 1.4426950408889634f : 0.0f;
                lo = min(lo, see[n][h].lo());
                hi = max(hi, see[n][h].hi());
                pre_end = max(pre_end, see[n][h].prefix_end());
                win_lo = min(win_lo, see[n][h].window_lo());
            }
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        pages::Gap gap;
        if (SCORED && p.prefix && p.window > 0)
            gap = pages::Gap(__reduce_max_sync(0xffffffffu, pre_end), __reduce_min_sync(0xffffffffu, win_lo), kUnit);

        // keys that any row of the block sees, in units; the cluster's CTAs take
        // consecutive shares of them, the warps of a CTA every fourth unit
        const int u_lo = hi > 0 ? lo / kUnit : 0, u_hi = gap.count((hi + kUnit - 1) / kUnit);
        const int per = (u_hi - u_lo + S - 1) / S;
        const int ua = u_lo + rank * per, ub = min(u_hi, ua + per);
        const int nu = ub - ua > warp ? (ub - ua - warp + kWarps - 1) / kWarps : 0;  // this warp's units

        const uint4* qs = reinterpret_cast<const uint4*>(sm + L::q) + lane;
        const uint32_t ring = ptx::smem_u32(sm) + warp * (kStages * L::stage);
        // the pages of this warp's next 16 units, one per lane for 16 keys each
        auto pages_at = [&](int k) {
            const int i = k + (lane >> 1), t = gap.number(ua + warp + i * kWarps) * kUnit + 16 * (lane & 1);
            return i < nu && t < T ? __ldg(table + (t >> s.pshift)) : 0;
        };
        int pg_now = pages_at(0), pg_next = 0;
        // Where this lane's 16-byte pieces go: within a 128-byte line, pieces are
        // exchanged by the line's number, so that neither product's reads collide
        // (the exchange repeats after 512 bytes, or 256 with D = 64: further rows of
        // the lane lie at fixed distances).
        constexpr int kLineRows = 256 / D;  // keys per line
        auto swizzled = [](int line) { return D == 128 ? 2 * (line & 3) : 2 * (line & 1); };
        auto place = [&](int row, int piece) {  // of the row
            const int line = row / kLineRows;
            return line * 128 + ((((row % kLineRows) * (D / 32) + piece) ^ swizzled(line)) << 4);
        };
        constexpr int kHalf = 16 * D / 2;  // bytes of 16 keys
        const uint32_t to_codes = place(lane / (D / 32), lane % (D / 32));
        const uint32_t to_scales = 2 * L::codes + ((lane >> 2) & 1) * (kUnit * 4) + (lane & 3) * 16;
        const unsigned char* kc = reinterpret_cast<const unsigned char*>(p.K) + lane * 16;
        const unsigned char* vc = reinterpret_cast<const unsigned char*>(p.V) + lane * 16;
        const float* scales = (lane & 4 ? p4.Vt : p4.Kt) + 4 * (lane & 3);
        uint32_t fill = ring;  // the stage that is filled next
        auto load_unit = [&](int k) {
            if ((k & 15) == 0) {
                if (k > 0) pg_now = pg_next;
                pg_next = pages_at(k + 16);
            }
            if (k < nu) {
                const int t0 = gap.number(ua + warp + k * kWarps) * kUnit;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int page = __shfl_sync(0xffffffffu, pg_now, (k & 15) * 2 + h), t = t0 + 16 * h;
                    const bool ok = page >= 0 && page < s.pages;
                    const long long vec =
                        ((((long long)(ok ? page : 0) * s.Hk + g) << s.pshift) + (t & ((1 << s.pshift) - 1)));
                    const uint32_t to = fill + to_codes + h * kHalf;
                    if (ok && t + 16 <= T) {
#pragma unroll
                        for (int it = 0; it < D / 64; ++it) {
                            cp_async16(to + it * 512, kc + vec * (D / 2) + it * 512, 16);
                            cp_async16(to + L::codes + it * 512, vc + vec * (D / 2) + it * 512, 16);
                        }
                        if (lane < 8) cp_async16(fill + to_scales + h * 64, scales + vec, 16);
                    } else {
                        if (!ok && lane == 0) pages::flag(s.status, kPgBadPage);
#pragma unroll
                        for (int it = 0; it < D / 64; ++it) {
                            const int real = ok && t + (it * 32 + lane) / (D / 32) < T ? 16 : 0;
                            cp_async16(to + it * 512, kc + vec * (D / 2) + it * 512, real);
                            cp_async16(to + L::codes + it * 512, vc + vec * (D / 2) + it * 512, real);
                        }
                        // (scales: four keys to a piece)
                        if (lane < 8)
                            cp_async16(fill + to_scales + h * 64, scales + vec,
                                       ok ? min(max(T - t - 4 * (lane & 3), 0), 4) * 4 : 0);
                    }
                }
            }
            cp_commit();  // an empty group past the last unit keeps the count
            fill = fill == ring + (kStages - 1) * L::stage ? ring : fill + L::stage;
        };
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) load_unit(k);

        float O[NR][MB][4];
        float m[NR][2], l[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int k = 0; k < MB; ++k) O[n][k][e] = 0.0f;
            m[n][0] = m[n][1] = -CUDART_INF_F;
            l[n][0] = l[n][1] = 0.0f;
        }

        // this lane's reads: K of key quad (its piece, or half of one), V of keys 2 qi and 2 qi + 1
        const int k_at = D == 128 ? place(quad, qi) : place(quad, qi >> 1) + (qi & 1) * 8;
        const int v_in = D == 128 ? (quad & 1) * 8 : (quad & 3) * 4;
        const int v_at[2] = {place(2 * qi, D == 128 ? quad >> 1 : quad >> 2) + v_in,
                             place(2 * qi + 1, D == 128 ? quad >> 1 : quad >> 2) + v_in};
        constexpr int kEight = 8 * D / 2;  // bytes of 8 keys
        int sees_all = INT_MAX;  // with the causal mask alone: the keys that every row sees
        if constexpr (!SCORED) {
#pragma unroll
            for (int n = 0; n < NR; ++n) sees_all = min(sees_all, min(see[n][0].b1, see[n][1].b1));
            sees_all = __reduce_min_sync(0xffffffffu, sees_all);
        }
        const unsigned char* st = sm + warp * (kStages * L::stage);
        for (int k = 0; k < nu; ++k) {
            load_unit(k + kStages - 1);
            cp_wait<kStages - 1>();
            __syncwarp();
            const int t0 = gap.number(ua + warp + k * kWarps) * kUnit;
            const float* kt = reinterpret_cast<const float*>(st + 2 * L::codes);
            const float* vt = kt + kUnit;
            // ---- scores: c[n][i][e]: key t0 + 16 i + quad (+ 8 for e >= 2), row 8 n + 2 qi + (e & 1)
            float c[NR][2][4];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[n][i][e] = off[n][e & 1];
            uint32_t w[4][W];  // keys quad + 8 y
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const unsigned char* at = st + k_at + y * kEight;
                if constexpr (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4*>(at);
                    w[y][0] = v.x, w[y][1] = v.y, w[y][2] = v.z, w[y][3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(at);
                    w[y][0] = v.x, w[y][1] = v.y;
                }
            }
#pragma unroll
            for (int j = 0; j < 2 * W; ++j) {  // a step: four channels of each lane, half a word
                uint32_t a[4], a16[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    if (j & 1) w[y][j / 2] >>= 8;
                    a[y] = half_centred(w[y][j / 2], 0x000F000Fu, 0xE408E408u);    // u - 8
                    a16[y] = half_centred(w[y][j / 2], 0x00F000F0u, 0xE480E480u);  // 16 (u - 8)
                }
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    const uint4 q = qs[(n * KS + j) * 32];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma_f16(c[n][i], a[2 * i], a[2 * i + 1], a16[2 * i], a16[2 * i + 1], q.x, q.y);
                        mma_f16(c[n][i], a[2 * i], a[2 * i + 1], a16[2 * i], a16[2 * i + 1], q.z, q.w);
                    }
                }
            }
            // ---- weights
            float tk[4], tv[4];  // keys t0 + quad + 8 i
#pragma unroll
            for (int i = 0; i < 4; ++i) tk[i] = kt[quad + 8 * i], tv[i] = vt[quad + 8 * i];
            bool whole = t0 + kUnit <= sees_all;
            if constexpr (SCORED) {
                bool all = true;
#pragma unroll
                for (int n = 0; n < NR; ++n) all = all && see[n][0].all(t0, t0 + kUnit) && see[n][1].all(t0, t0 + kUnit);
                whole = __all_sync(0xffffffffu, all);
            }
            bool move = false;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float t = tk[2 * i + (e >> 1)];
                        // (the row's power of two meets the key's scale first: products overflow only where scores do)
                        const float2 f = __fmul2_rn(make_float2(mul[n][0], mul[n][1]), make_float2(t, t));
                        const float2 x = __fmul2_rn(make_float2(c[n][i][e], c[n][i][e + 1]), f);
                        c[n][i][e] = x.x, c[n][i][e + 1] = x.y;
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int h = e & 1, kk = 2 * i + (e >> 1), j = t0 + quad + 8 * kk;
                        float x = c[n][i][e];
                        if constexpr (SCORED) x = pages::score<SCORED>(p, x, slope2[n][h], pos[n][h], j);
                        if (!whole && !see[n][h].has(j)) x = -CUDART_INF_F;
                        c[n][i][e] = x;
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mx = fmaxf(ptx::max3(c[n][0][h], c[n][0][2 + h], c[n][1][h]), c[n][1][2 + h]);
                    move = move || mx > m[n][h] + kLazyMax;  // (any score above a reference of -inf)
                }
            }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float mx = fmaxf(fmaxf(fmaxf(c[n][0][h], c[n][0][2 + h]), fmaxf(c[n][1][h], c[n][1][2 + h])), m[n][h]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        // (nothing summed yet: sums of 0, or NaN, which stays)
                        const float al = m[n][h] == -CUDART_INF_F ? 1.0f : ptx::ex2(m[n][h] - mx);
                        l[n][h] *= al;
#pragma unroll
                        for (int q = 0; q < MB; ++q) O[n][q][h] *= al, O[n][q][2 + h] *= al;
                        m[n][h] = mx;
                    }
            }
            uint32_t pb[NR][2][2];  // operands of P V: keys of 16 i, in two eights
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const float2 nref = make_float2(m[n][0] == -CUDART_INF_F ? 0.0f : -m[n][0], m[n][1] == -CUDART_INF_F ? 0.0f : -m[n][1]);
                float2 sum = make_float2(l[n][0], l[n][1]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float t = tv[2 * i + (e >> 1)];
                        const float2 d = __fadd2_rn(make_float2(c[n][i][e], c[n][i][e + 1]), nref);
                        const float2 w = make_float2(ptx::ex2(d.x), ptx::ex2(d.y));
                        sum = __fadd2_rn(sum, w);
                        float2 v = __fmul2_rn(w, make_float2(t, t));
                        if (!whole) {  // what a masked place's scale holds has no say (a seen one's does, at any weight)
                            v.x = c[n][i][e] == -CUDART_INF_F ? 0.0f : v.x;
                            v.y = c[n][i][e + 1] == -CUDART_INF_F ? 0.0f : v.y;
                        }
                        pb[n][i][e >> 1] = transposed(pack_bf2(v.x, v.y));
                    }
                l[n][0] = sum.x, l[n][1] = sum.y;
            }
            // ---- O += P V; lane: channels of the D / 8 from quad on, keys 2 qi, 2 qi + 1 of each eight
            const unsigned char* sv = st + L::codes;
            constexpr int VW = D / 64;  // words of a key per lane
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t w[4][VW];  // keys 2 qi, 2 qi + 1, 8 more, one more
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const unsigned char* at = sv + v_at[y & 1] + (2 * i + (y >> 1)) * kEight;
                    if constexpr (D == 128) {
                        const uint2 v = *reinterpret_cast<const uint2*>(at);
                        w[y][0] = v.x, w[y][1] = v.y;
                    } else {
                        w[y][0] = *reinterpret_cast<const uint32_t*>(at);
                    }
                }
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    // even channels of both keys, odd ones; of the first eight keys, of the second
                    const uint32_t ev0 = ptx::prmt(w[0][j], w[1][j], 0x5410), od0 = ptx::prmt(w[0][j], w[1][j], 0x7632);
                    const uint32_t ev1 = ptx::prmt(w[2][j], w[3][j], 0x5410), od1 = ptx::prmt(w[2][j], w[3][j], 0x7632);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        auto nibble = [&](uint32_t x) { return centred(q ? x >> (4 * q - 1) : x << 1); };
                        const uint32_t a0 = nibble(ev0), a1 = nibble(od0), a2 = nibble(ev1), a3 = nibble(od1);
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma_bf16(O[n][4 * j + q], a0, a1, a2, a3, pb[n][i][0], pb[n][i][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read the stage
            st = st == sm + warp * (kStages * L::stage) + (kStages - 1) * L::stage ? sm + warp * (kStages * L::stage) : st + L::stage;
        }
        cp_wait<0>();
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], o);
        __syncthreads();  // every warp is done with its ring

        // the warps' rows: O, then (m, l) with m = -inf where nothing was summed
        float* rows = reinterpret_cast<float*>(sm) + warp * (kRows * RS);
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* dst = rows + (8 * n + 2 * qi + h) * RS;
#pragma unroll
                for (int q = 0; q < MB; ++q)
                    *reinterpret_cast<float2*>(dst + quad * (D / 8) + 2 * q) = make_float2(O[n][q][h], O[n][q][2 + h]);
                if (quad == 0) {
                    dst[D] = l[n][h] == 0.0f ? -CUDART_INF_F : (m[n][h] == -CUDART_INF_F ? 0.0f : m[n][h]);
                    dst[D + 1] = l[n][h];
                }
            }
        __syncthreads();

        // merge: 4 channels per item, whole warps (the transform crosses lanes)
        constexpr int C4 = D / 4;
        auto finish = [&](bool live, int r, int c4, float M, float Lt, float4 a) {
            pages::transform4<D>(a);
            if (!live) return;
            const long long row = (long long)(b.q0 + token_of(r)) * p.Hq + head_of(r);
            const float inv = Lt == 0.0f ? 0.0f : 1.0f / Lt;
            *reinterpret_cast<uint2*>(p.out + row * D + c4 * 4) =
                Lt == 0.0f ? make_uint2(0u, 0u)
                           : make_uint2(pack_bf2(a.x * inv, a.y * inv), pack_bf2(a.z * inv, a.w * inv));
            if (c4 == 0 && p.lse) p.lse[row] = Lt == 0.0f ? -CUDART_INF_F : (M + log2f(Lt)) * 0.6931471805599453f;
        };
        float* merged = reinterpret_cast<float*>(sm) + kWarps * (kRows * RS);
        for (int it0 = 0; it0 < nr * C4; it0 += kWarps * 32) {
            const int it = it0 + tid, r = min(it / C4, nr - 1), c4 = it % C4;
            const bool live = it < nr * C4;
            const float* src = reinterpret_cast<const float*>(sm) + r * RS;
            float M = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, src[w * (kRows * RS) + D]);
            float Lt = 0.0f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* x = src + w * (kRows * RS);
                const float lw = x[D + 1];
                const float f = lw == 0.0f ? 0.0f : ptx::ex2(x[D] - M);
                const float4 v = *reinterpret_cast<const float4*>(x + c4 * 4);
                Lt = fmaf(f, lw, Lt);
                a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
            }
            if (S == 1) {
                finish(live, r, c4, M, Lt, a);
            } else if (live) {
                *reinterpret_cast<float4*>(merged + r * RS + c4 * 4) = a;
                if (c4 == 0) merged[r * RS + D] = M, merged[r * RS + D + 1] = Lt;
            }
        }
        if (S > 1) {
            ptx::cluster_arrive();
            ptx::cluster_wait();
            for (int it0 = rank * (kWarps * 32); it0 < nr * C4; it0 += S * kWarps * 32) {
                const int it = it0 + tid, r = min(it / C4, nr - 1), c4 = it % C4;
                float M = -CUDART_INF_F;
                for (int k = 0; k < S; ++k) M = fmaxf(M, ptx::ld_dsmem(ptx::dsmem_addr(merged + r * RS + D, k)));
                float Lt = 0.0f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < S; ++k) {
                    const float2 ml = ptx::ld_dsmem2(ptx::dsmem_addr(merged + r * RS + D, k));
                    const float4 v = ptx::ld_dsmem4(ptx::dsmem_addr(merged + r * RS + c4 * 4, k));
                    const float f = ml.y == 0.0f ? 0.0f : ptx::ex2(ml.x - M);
                    Lt = fmaf(f, ml.y, Lt);
                    a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
                }
                finish(it < nr * C4, r, c4, M, Lt, a);
            }
            // no CTA goes on (or away) while another reads its rows
            ptx::cluster_arrive();
            ptx::cluster_wait();
        }
        if (!DIRECT || (b.blk + 1) * kRows >= b.n * p.G) break;
        __syncthreads();
    }
}

template <int D, int NR, bool SCORED, bool DIRECT>
cudaError_t launch(const PagedAttend4& a, int split, long long blocks, cudaStream_t st) {
    auto kern = pages4_rows_kernel<D, NR, SCORED, DIRECT>;
    constexpr int smem = Lay<D, NR>::total;
    // opted in once per instance and device
    static std::once_flag once[kPagedDevices];
    static cudaError_t opt[kPagedDevices];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device >= kPagedDevices) return cudaErrorInvalidDevice;
    std::call_once(once[device], [&] {
        opt[device] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (opt[device] == cudaSuccess)
            opt[device] = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (opt[device] != cudaSuccess) return opt[device];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split * blocks), a.a.s.Hk, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, int NR>
cudaError_t launch_rows(const PagedAttend4& p, int max_q, int max_kv, int sm_count, cudaStream_t st) {
    const PagedAttend& a = p.a;
    constexpr int kRows = 8 * NR;
    const bool direct = (long long)max_q * a.G <= kRows;
    const long long blocks = direct ? a.s.seqs : (long long)a.s.tokens * a.G / kRows + a.s.seqs;
    // Keys split over a cluster, every warp with two units at least, so that the
    // fullest SM has least to do: its CTAs' units, and for every wave of CTAs a start
    // and an end that take about as long as kWave units of an SM (32 sequences of 32K
    // keys, 8 KV heads: 292 us in 2, one wave of 512 CTAs on 152 SMs, 256 in 4; 15 of
    // 4,096 keys: 28 us in 5, 33 in 10, though 24 in 4, which this does not tell apart).
    const long long jobs = std::max(1LL, std::min(blocks, a.s.seqs * (((long long)max_q * a.G + kRows - 1) / kRows)) * a.s.Hk);
    const long long units = std::max(1, (max_kv + kUnit - 1) / kUnit), most = std::min(kMaxSplit, max_kv / (2 * kWarps * kUnit));
    long long split = 1, best = LLONG_MAX;
    for (long long k = 1; k <= std::max(1LL, most); ++k) {
        const long long ctas = jobs * k, slots = (long long)ctas_per_sm(NR) * sm_count;
        const long long per_sm = (ctas + sm_count - 1) / sm_count;  // (a CTA alone takes half as long again)
        const long long cost = (2 * per_sm + 1) * ((units + k - 1) / k) + (ctas + slots - 1) / slots * 2 * kWave;
        if (cost < best) best = cost, split = k;
    }
    if (split * blocks > INT_MAX) return cudaErrorInvalidValue;
    if (paged_scored(a))
        return direct ? launch<D, NR, true, true>(p, (int)split, blocks, st)
                      : launch<D, NR, true, false>(p, (int)split, blocks, st);
    return direct ? launch<D, NR, false, true>(p, (int)split, blocks, st)
                  : launch<D, NR, false, false>(p, (int)split, blocks, st);
}

}  // namespace

cudaError_t launch_pages4_rows(const PagedAttend4& a, int head_dim, int max_q, int max_kv, int sm_count,
                               cudaStream_t st) {
    // Blocks of 8 rows fill the GPU sooner and take less time to start; blocks of 16
    // take the codes apart half as often, which pays where there are many units of
    // keys (32 sequences of 16K keys, 16 rows: 206 us against 251, of 4,096 66 against
    // 77; 8 of 4,096: 32 against 25).
    const long long rows = (long long)max_q * a.a.G;
    const bool two = rows > 8 && (double)a.a.s.seqs * ((rows + 15) / 16) * a.a.s.Hk * max_kv >= (double)(1 << 20);
#define KVP_PG4_ROWS(DD) \
    (two ? launch_rows<DD, 2>(a, max_q, max_kv, sm_count, st) : launch_rows<DD, 1>(a, max_q, max_kv, sm_count, st))
    return head_dim == 64 ? KVP_PG4_ROWS(64) : KVP_PG4_ROWS(128);
#undef KVP_PG4_ROWS
}

}  // namespace kvp
