// Attention of few query rows per sequence over its pages: decode steps, draft
// tokens.
//
// Mathematics: softmax over the keys a row sees in one pass, with a running
// reference maximum m per row, p = 2^(x - m), l = sum p and O = sum p v, O and
// l rescaled when the maximum passes m by more than 2^8 (the weights then stay
// below 2^8, which bf16 and fp32 hold as well as numbers below 1).
//
// Bound: memory. A step reads every seen K and V row once; the products are
// 4 * rows FLOP per byte pair, far below what even padded tensor-core tiles
// give. So the layout serves the loads. A CTA has the up to 16 rows (new
// tokens x heads of a group) of one sequence and KV head, which fill an m16
// matrix operand that stays in registers; its 4 warps take units of 16 keys in
// turn, each through a ring of its own in shared memory, filled by 16-byte
// asynchronous copies that nothing but the warp itself waits for (no barrier
// in the loop; a copy of a key behind the sequence's end is told to write
// zeros, so that whatever the page holds there never meets a weight of 0).
// The warps' states meet in shared memory at the end, those of the CTAs of a
// cluster, which split the keys, in distributed shared memory: no workspace
// and no second launch. Two CTAs per SM (their registers) beat three with
// fewer registers, which leave the loads of a unit less overlap (32 sequences
// of 32K keys, 64 query heads on 8 of 128: 588 us against 727); a third unit
// per ring gains nothing (596 us against 624), and a cluster split that runs
// in one wave beats finer ones (16 sequences of 4,096 keys: 59 us at 2, 64 at
// 4, 82 at 9).
//
// Measured: those 32 sequences, 4.1 GB of keys and values, in 577 us, 7.1 TB/s;
// 3 sequences of up to 129 keys in 3.8 us of a captured graph.
#include <algorithm>
#include <mutex>

#include "pages.cuh"

namespace kvp {
namespace {

using pages::Seen;

constexpr int kWarps = 4;
constexpr int kUnit = 16;   // keys per unit (the smallest page)
constexpr int kRows = 16;   // rows of a block (the MMA's m)
constexpr int kStages = 2;  // units in a warp's ring
constexpr float kLazyMax = 8.0f;
constexpr int kMaxSplit = 16;

template <int D>
constexpr int ring_bytes() { return kWarps * kStages * 2 * kUnit * D * 2; }
// the merge reuses the rings: per warp 16 rows of D + 4 floats, then the CTA's
// merged rows; (m, l) in the last two floats of each row
template <int D>
constexpr int merge_bytes() { return (kWarps + 1) * kRows * (D + 4) * 4; }
template <int D>
constexpr int smem_bytes() { return ring_bytes<D>() > merge_bytes<D>() ? ring_bytes<D>() : merge_bytes<D>(); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < CUDART_INF_F; }

// SCORED: score modifiers apply. STATE: the rows' states for a merge instead
// of the output; the weights then go through the matrix product as bf16 hi and
// lo (16 bits), as the merged output is fp32. Otherwise they are rounded to
// bf16 once (off by at most 2^-8 of each, as the output's own rounding is of it).
// DIRECT: every sequence has one block (no search; if it has more, the CTA
// takes them in turn). Grid: blocks x the CTAs of a cluster, KV heads.
template <int D, bool SCORED, bool STATE, bool DIRECT>
__global__ void __launch_bounds__(kWarps * 32)
pages_rows_kernel(const PagedAttend p) {
    constexpr int KS = D / 16;   // k steps of Q K^T
    constexpr int NB = D / 8;    // n blocks of P V
    constexpr int CH = D / 8;    // 16-byte pieces of a row
    constexpr int RS = D + 4;    // floats of a merge row
    constexpr int UB = kUnit * D * 2;
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
        // this thread's two rows
        Seen see[2];
        int tok[2], head[2], pos[2];
        float slope2[2];
        bool live[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = min(quad + 8 * h, nr - 1);  // rows past the block repeat its last one, and are dropped
            live[h] = quad + 8 * h < nr;
            const int i = (r_begin + r) / p.G;
            tok[h] = b.q0 + i;
            head[h] = g * p.G + (r_begin + r) - i * p.G;
            pos[h] = b.p0 + i;
            see[h] = pages::row_seen<SCORED>(p, b.seq, tok[h], pos[h], T);
            slope2[h] = SCORED && p.slopes ? __ldg(p.slopes + head[h]) * 1.4426950408889634f : 0.0f;
        }
        uint32_t qf[KS][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(p.Q + (long long)tok[h] * p.q_stride +
                                                                    (long long)head[h] * D) + qi;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][h] = __ldg(src + k * 8);
                qf[k][2 + h] = __ldg(src + k * 8 + 4);
            }
        }
        // keys that any row of the block sees, in units; the cluster's CTAs take
        // consecutive shares of them, the warps of a CTA every fourth unit
        int lo = min(see[0].lo(), see[1].lo()), hi = max(see[0].hi(), see[1].hi());
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        pages::Gap gap;
        if (SCORED && p.prefix && p.window > 0)
            gap = pages::Gap(__reduce_max_sync(0xffffffffu, max(see[0].prefix_end(), see[1].prefix_end())),
                             __reduce_min_sync(0xffffffffu, min(see[0].window_lo(), see[1].window_lo())), kUnit);
        const int u_lo = hi > 0 ? lo / kUnit : 0, u_hi = gap.count((hi + kUnit - 1) / kUnit);
        const int per = (u_hi - u_lo + S - 1) / S;
        const int ua = u_lo + rank * per, ub = min(u_hi, ua + per);
        const int nu = ub - ua > warp ? (ub - ua - warp + kWarps - 1) / kWarps : 0;  // this warp's units

        const uint32_t ring = ptx::smem_u32(sm) + warp * (kStages * 2 * UB);
        // the pages of this warp's next 32 units, one per lane
        auto pages_at = [&](int k) {
            const int u = gap.number(ua + warp + (k + lane) * kWarps);
            return k + lane < nu ? __ldg(table + ((u * kUnit) >> s.pshift)) : 0;
        };
        int pg_now = pages_at(0), pg_next = 0;
        auto load_unit = [&](int k) {
            if ((k & 31) == 0) {
                if (k > 0) pg_now = pg_next;
                pg_next = pages_at(k + 32);
            }
            if (k < nu) {
                const int page = __shfl_sync(0xffffffffu, pg_now, k & 31);
                const int t0 = gap.number(ua + warp + k * kWarps) * kUnit;
                const bool ok = page >= 0 && page < s.pages;
                if (!ok && lane == 0) pages::flag(s.status, kPgBadPage);
                const long long at =
                    ((((long long)(ok ? page : 0) * s.Hk + g) << s.pshift) + (t0 & ((1 << s.pshift) - 1))) * D;
                const uint32_t dst = ring + (k % kStages) * (2 * UB);
#pragma unroll
                for (int it = 0; it < kUnit * CH / 32; ++it) {
                    const int i = it * 32 + lane, row = i / CH, c = i % CH;
                    const bool real = ok && t0 + row < T;
                    const uint32_t to = dst + row * (D * 2) + ((c ^ (row & 7)) << 4);
                    cp_async16(to, p.K + at + i * 8, real);
                    cp_async16(to + UB, p.V + at + i * 8, real);
                }
            }
            cp_commit();  // an empty group past the last unit keeps the count
        };
#pragma unroll
        for (int k = 0; k < kStages; ++k) load_unit(k);

        float O[NB][4], m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[n][e] = 0.0f;

        for (int k = 0; k < nu; ++k) {
            cp_wait<kStages - 1>();
            __syncwarp();
            const uint32_t sk = ring + (k % kStages) * (2 * UB), sv = sk + UB;
            const int t0 = gap.number(ua + warp + k * kWarps) * kUnit;
            float c[2][4] = {};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t kf[4];
                const int row = ((lane >> 4) << 3) + (lane & 7), ch = ks * 2 + ((lane >> 3) & 1);
                ldsm4(sk + row * (D * 2) + ((ch ^ (row & 7)) << 4), kf);
                mma16816(c[0], qf[ks], kf[0], kf[1]);
                mma16816(c[1], qf[ks], kf[2], kf[3]);
            }
            // scores in log2 units: row h of this thread, keys t0 + 8 nb + 2 qi + e
            const bool whole = __all_sync(0xffffffffu, see[0].all(t0, t0 + kUnit) && see[1].all(t0, t0 + kUnit));
            float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int h = e >> 1, j = t0 + nb * 8 + qi * 2 + (e & 1);
                    float x = pages::score<SCORED>(p, c[nb][e], slope2[h], pos[h], j);
                    if (!whole && !see[h].has(j)) x = -CUDART_INF_F;
                    c[nb][e] = x;
                    mx[h] = fmaxf(mx[h], x);
                }
            bool move = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                move = move || mx[h] > m[h] + kLazyMax || (m[h] == -CUDART_INF_F && mx[h] > m[h]);
            }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mn = fmaxf(m[h], mx[h]);
                    const float al = m[h] == -CUDART_INF_F ? 0.0f : ptx::ex2(m[h] - mn);
                    // rows with nothing seen yet have sums of 0 (or NaN, which stays)
                    l[h] = m[h] == -CUDART_INF_F ? l[h] : l[h] * al;
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        O[n][2 * h] = m[h] == -CUDART_INF_F ? O[n][2 * h] : O[n][2 * h] * al;
                        O[n][2 * h + 1] = m[h] == -CUDART_INF_F ? O[n][2 * h + 1] : O[n][2 * h + 1] * al;
                    }
                    m[h] = mn;
                }
            }
            const float ref[2] = {m[0] == -CUDART_INF_F ? 0.0f : m[0], m[1] == -CUDART_INF_F ? 0.0f : m[1]};
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    c[nb][e] = ptx::ex2(c[nb][e] - ref[e >> 1]);
                    l[e >> 1] += c[nb][e];
                }
            uint32_t pf[4] = {pack_bf2(c[0][0], c[0][1]), pack_bf2(c[0][2], c[0][3]), pack_bf2(c[1][0], c[1][1]),
                              pack_bf2(c[1][2], c[1][3])};
            uint32_t pl[4];
            if constexpr (STATE) {
                auto rest = [](float x, float y, uint32_t hi) {
                    return pack_bf2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
                };
                pl[0] = rest(c[0][0], c[0][1], pf[0]);
                pl[1] = rest(c[0][2], c[0][3], pf[1]);
                pl[2] = rest(c[1][0], c[1][1], pf[2]);
                pl[3] = rest(c[1][2], c[1][3], pf[3]);
            }
#pragma unroll
            for (int n = 0; n < NB; n += 2) {
                uint32_t vf[4];
                const int row = (((lane >> 3) & 1) << 3) + (lane & 7), ch = n + (lane >> 4);
                ldsm4t(sv + row * (D * 2) + ((ch ^ (row & 7)) << 4), vf);
                mma16816(O[n], pf, vf[0], vf[1]);
                mma16816(O[n + 1], pf, vf[2], vf[3]);
                if constexpr (STATE) {
                    mma16816(O[n], pl, vf[0], vf[1]);
                    mma16816(O[n + 1], pl, vf[2], vf[3]);
                }
            }
            __syncwarp();  // every lane has read the stage
            load_unit(k + kStages);
        }
        cp_wait<0>();
        bool odd = false;  // sums that a masked key may have spoilt
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (live[h] && !finite(l[h])) odd = true;
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (live[e >> 1] && !finite(O[n][e])) odd = true;
        __syncthreads();  // every warp is done with its ring

        // the warps' rows: O, then (m, l) with m = -inf where nothing was summed
        float* rows = reinterpret_cast<float*>(sm) + warp * (kRows * RS);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float* dst = rows + (quad + 8 * h) * RS;
#pragma unroll
            for (int n = 0; n < NB; ++n)
                *reinterpret_cast<float2*>(dst + n * 8 + qi * 2) = make_float2(O[n][2 * h], O[n][2 * h + 1]);
            if (qi == 0) {
                dst[D] = l[h] == 0.0f ? -CUDART_INF_F : (m[h] == -CUDART_INF_F ? 0.0f : m[h]);
                dst[D + 1] = l[h];
            }
        }
        const unsigned odds = __ballot_sync(0xffffffffu, odd);
        if (odds) {
            for (int r = 0; r < nr; ++r) {
                if (!((odds >> ((r & 7) * 4)) & 0xFu)) continue;
                const int i = (r_begin + r) / p.G, hd = g * p.G + (r_begin + r) - i * p.G;
                const Seen se = pages::row_seen<SCORED>(p, b.seq, b.q0 + i, b.p0 + i, T);
                float mm, ll, acc[D / 32];
                pages::careful_row<D, SCORED>(p, b.seq, b.q0 + i, hd, b.p0 + i, se, gap, 4, ua + warp,
                                              ub, kWarps, mm, ll, acc);
                float* dst = rows + r * RS;
                __syncwarp();
#pragma unroll
                for (int e = 0; e < D / 32; ++e) dst[lane * (D / 32) + e] = acc[e];
                if (lane == 0) dst[D] = mm, dst[D + 1] = ll;
                __syncwarp();
            }
        }
        __syncthreads();

        // merge of n states `stride` floats apart (or of a cluster's): 4 channels per item
        constexpr int C4 = D / 4;
        auto finish = [&](int r, int c4, float M, float L, float4 a) {
            const int i = (r_begin + r) / p.G;
            const int t = b.q0 + i, hd = g * p.G + (r_begin + r) - i * p.G;
            const long long row = (long long)t * p.Hq + hd;
            if constexpr (STATE) {
                *reinterpret_cast<float4*>(p.st_acc + row * D + c4 * 4) = a;
                if (c4 == 0) *pages::state_ml(p, t, hd) = make_float2(M, L);
            } else {
                const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                *reinterpret_cast<uint2*>(p.out + row * D + c4 * 4) =
                    L == 0.0f ? make_uint2(0u, 0u)
                              : make_uint2(pack_bf2(a.x * inv, a.y * inv), pack_bf2(a.z * inv, a.w * inv));
                if (c4 == 0 && p.lse)
                    p.lse[row] = L == 0.0f ? -CUDART_INF_F : (M + log2f(L)) * 0.6931471805599453f;
            }
        };
        float* merged = reinterpret_cast<float*>(sm) + kWarps * (kRows * RS);
        for (int it = tid; it < nr * C4; it += kWarps * 32) {
            const int r = it / C4, c4 = it % C4;
            const float* src = reinterpret_cast<const float*>(sm) + r * RS;
            float M = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, src[w * (kRows * RS) + D]);
            float L = 0.0f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* x = src + w * (kRows * RS);
                const float lw = x[D + 1];
                const float f = lw == 0.0f ? 0.0f : ptx::ex2(x[D] - M);
                const float4 v = *reinterpret_cast<const float4*>(x + c4 * 4);
                L = fmaf(f, lw, L);
                a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
            }
            if (S == 1) {
                finish(r, c4, M, L, a);
            } else {
                *reinterpret_cast<float4*>(merged + r * RS + c4 * 4) = a;
                if (c4 == 0) merged[r * RS + D] = M, merged[r * RS + D + 1] = L;
            }
        }
        if (S > 1) {
            ptx::cluster_arrive();
            ptx::cluster_wait();
            for (int it = rank * (kWarps * 32) + tid; it < nr * C4; it += S * kWarps * 32) {
                const int r = it / C4, c4 = it % C4;
                float M = -CUDART_INF_F;
                for (int k = 0; k < S; ++k) M = fmaxf(M, ptx::ld_dsmem(ptx::dsmem_addr(merged + r * RS + D, k)));
                float L = 0.0f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < S; ++k) {
                    const float2 ml = ptx::ld_dsmem2(ptx::dsmem_addr(merged + r * RS + D, k));
                    const float4 v = ptx::ld_dsmem4(ptx::dsmem_addr(merged + r * RS + c4 * 4, k));
                    const float f = ml.y == 0.0f ? 0.0f : ptx::ex2(ml.x - M);
                    L = fmaf(f, ml.y, L);
                    a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
                }
                finish(r, c4, M, L, a);
            }
            // no CTA goes on (or away) while another reads its rows
            ptx::cluster_arrive();
            ptx::cluster_wait();
        }
        if (!DIRECT || (b.blk + 1) * kRows >= b.n * p.G) break;
        __syncthreads();
    }
}

template <int D, bool SCORED, bool STATE, bool DIRECT>
cudaError_t launch(const PagedAttend& a, int split, long long blocks, cudaStream_t st) {
    auto kern = pages_rows_kernel<D, SCORED, STATE, DIRECT>;
    // opted in once per instance and device
    static std::once_flag once[kPagedDevices];
    static cudaError_t opt[kPagedDevices];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device >= kPagedDevices) return cudaErrorInvalidDevice;
    std::call_once(once[device], [&] {
        opt[device] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D>());
        if (opt[device] == cudaSuccess)
            opt[device] = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (opt[device] != cudaSuccess) return opt[device];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split * blocks), a.s.Hk, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<D>();
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

}  // namespace

cudaError_t launch_pages_rows(const PagedAttend& a, int head_dim, int max_q, int max_kv, int sm_count,
                              cudaStream_t st) {
    const bool direct = (long long)max_q * a.G <= kRows;
    const long long blocks = direct ? a.s.seqs : (long long)a.s.tokens * a.G / kRows + a.s.seqs;
    // keys split over a cluster as far as all CTAs still run at once, two per SM
    // (their registers), and every warp keeps four units
    const long long jobs = std::min(blocks, a.s.seqs * (((long long)max_q * a.G + kRows - 1) / kRows)) * a.s.Hk;
    long long split = std::min<long long>(2LL * sm_count / std::max(1LL, jobs), max_kv / (4 * kWarps * kUnit));
    split = std::max<long long>(1, std::min<long long>(split, kMaxSplit));
    if (split * blocks > INT_MAX) return cudaErrorInvalidValue;
    const bool scored = paged_scored(a), state = a.st_acc != nullptr;
#define KVP_PG_ROWS(DD, SC, SS) \
    (direct ? launch<DD, SC, SS, true>(a, (int)split, blocks, st) \
            : launch<DD, SC, SS, false>(a, (int)split, blocks, st))
    if (state) return head_dim == 64 ? KVP_PG_ROWS(64, false, true) : KVP_PG_ROWS(128, false, true);
    if (head_dim == 64) return scored ? KVP_PG_ROWS(64, true, false) : KVP_PG_ROWS(64, false, false);
    return scored ? KVP_PG_ROWS(128, true, false) : KVP_PG_ROWS(128, false, false);
#undef KVP_PG_ROWS
}

}  // namespace kvp
