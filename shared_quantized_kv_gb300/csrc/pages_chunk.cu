// Attention of many query rows per sequence over its pages: chunks of new
// tokens, whole prompts (sm_103a, tcgen05).
//
// Mathematics as in pages_rows.cu: one pass over the keys, a running reference
// maximum that moves when the maximum passes it by more than 2^8, p = 2^(x - m)
// rounded to bf16 for the product with V (off by at most 2^-8 of each weight, as
// the output's own rounding is of it), l = sum p in float32.
//
// Bound: the tensor cores, 4 D FLOP per (row, key). A CTA has up to 256 rows
// (new tokens x heads of a group) of one sequence and KV head, as two tiles of
// 128, and walks the keys in tiles of 128. Two slots of tensor memory, each
// with S (128 columns; P, its bf16 weights, overwrites it) and O (D columns),
// are worked on in turn: while the tensor cores do P V and the next Q K^T of
// one slot, the eight softmax warps of the other turn its S into P. With more
// than 128 rows the slots are the two row tiles, and each K and V tile serves
// both; with fewer, both slots have the same rows and take every second key
// tile, and their states are merged at the end.
//   warps 0, 3    loaders of K and of V: pages by TMA, one box of 64 channels
//                 per page, through one ring in the order they are needed
//   warps 1, 2    issuers of the MMAs, one per slot
//   warps 4-19    softmax, two threads per row of a slot: 32 keys of every 64
//                 each, and half the channels of the output
// S_{i+1} of a slot may overwrite P_i because the MMAs of a thread run in the
// order they are issued. V comes as [key][channel], which the MMA takes as an
// MN-major operand. The keys may be split over the CTAs of a cluster, whose
// states meet in distributed shared memory: no workspace, no second launch.
// Every wait on a barrier in memory is bounded; one that expires is recorded in the status word, and
// the CTA runs to its end without waiting again.
//
// Measured on 2,432 new tokens over 16K keys, 32 query heads on 8 KV heads of
// 128 (two full waves of CTAs): 333 us, 1815 TFLOP/s. What got it there: one
// issuer per slot, taking turns (a single one's waits and commits left the
// tensor cores idle: 466 us; two without turns fell into step: 592 us);
// operands of the MMAs in uniform registers (509 us before; not all of them
// known to be uniform and no elected lane: 413 us); two threads per row (402 us
// with one and the same issue, its P too late for its turn); P formed under the
// reference as it is, the maxima looked at after it, and handed over in halves;
// no register spilled (the roles' registers shifted between the warpgroups; 128
// bytes of spill loads cost 3 %). Pages of 16 tokens are 32 boxes per pair of tiles:
// one loader issues them in 1.4 times as long as the rest takes (470 us against
// 340 on 2,048 tokens over 16K when two were tried; now 325), two keep up.
#include <algorithm>
#include <mutex>

#include "pages.cuh"

namespace kvp {
namespace {

using pages::Seen;

constexpr int kThreads = 640;
constexpr int kTile = 128;              // keys per tile, rows per slot
constexpr int kRows = 2 * kTile;        // rows per CTA
constexpr int kFewTiles = 8;            // key tiles that a cluster does not split
constexpr int kMaxParts = 16;           // states of a row: 8 CTAs, 2 slots
// log2 units the reference may trail the maximum: by little where the next tile
// may add to it before it is looked at again, else by what a float32 sum has room
// for (with a bias by distance it moves often)
constexpr float kLazyMax = 8.0f, kLazyScores = 60.0f;
constexpr uint32_t kTryNs = 1000, kTries = 1u << 18;
constexpr uint32_t kCols = 512;         // tensor memory: S0, S1, O0, O1
// named barriers: Q is staged (issuers and softmax warps); every role is done; the merge rows are written;
// a slot's turn at the tensor cores; the two warps of 32 rows (8 barriers)
constexpr uint32_t kBarQ = 1, kBarDone = 2, kBarRows = 3, kBarTurn = 4, kBarPair = 6, kBarLoad = 14;
constexpr int kSoftmax = 512;           // softmax threads
constexpr float kLn2 = 0.6931471805599453f;
// registers: 5 warpgroups launched with 96 each; 64 + 4 x 104 = 5 x 96
constexpr int kRegsFew = 64, kRegsMany = 104;

template <int D>
struct Lay {
    static constexpr int stage = kTile * D * 2;  // a K or V tile
    static constexpr int nst = D == 128 ? 5 : 10;
    static constexpr int ring = 2 * stage;       // after the two Q tiles
    static constexpr int bars = ring + nst * stage;
    // barriers: full, empty per ring stage; per slot S, P (of each half), P V of the first, all done
    static constexpr int bar_s = bars + 2 * nst * 8, bar_p = bar_s + 16, bar_o = bar_p + 32, bar_fin = bar_o + 16;
    static constexpr int info = bar_fin + 16;  // rng[2][2], tensor memory address, prefixes' end, windows' begin
    static constexpr int pair = info + 32;       // per slot a float per row, then a word per 32 rows
    static constexpr int total = pair + 2 * kTile * 4 + 32 + 1024;  // + alignment of the base
    static constexpr int rs = D + 4;             // floats of a merge row: O, m, l
    static_assert(kRows * (rs + kMaxParts) * 4 <= bars, "merge rows and weights fit in the tiles");
    static_assert(total <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float asf(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t asu(float f) { return __float_as_uint(f); }
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < CUDART_INF_F; }

// ring entries of tile i's K and V, of n tiles: K0 K1 V0 K2 V1 K3 ...
__device__ __forceinline__ int k_entry(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_entry(int i, int n) { return min(2 * i + 2, 2 * n - 1); }

// Wait for phase `parity` of the barrier by a whole warp; after kTries tries
// (each suspends the warp for a while; about a quarter of a second in all) `bad` is set, and
// no wait after that waits. One short loop: what is around a wait is on the
// main loop's critical path.
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, bool& bad) {
    if (!bad) {
        uint32_t ok;
        asm volatile(
            "{\n.reg .pred p, q;\n.reg .u32 n;\nmov.u32 n, 0;\n"
            "TRY:\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n@p bra DONE;\n"
            "add.u32 n, n, 1;\nsetp.lt.u32 q, n, %4;\n@q bra TRY;\n"
            "DONE:\nselp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(kTryNs), "n"(kTries) : "memory");
        bad = !ok;
    }
    __syncwarp();
}

// bits k of [32 c, 32 c + 32) with a <= 32 c + k < b
__device__ __forceinline__ uint32_t span_bits(int a, int b, int c) {
    const int x = min(max(a - 32 * c, 0), 32), y = min(max(b - 32 * c, 0), 32);
    if (y <= x) return 0u;
    const uint32_t upto = y == 32 ? 0xffffffffu : (1u << y) - 1u;
    return upto & ~(x == 32 ? 0xffffffffu : (1u << x) - 1u);
}

// KIND: the causal mask alone; other masks too; scores that a cap or a bias by
// distance changes (their costs are apart: 2,432 tokens over 16K keys take
// 333 us, 382 with a window, 793 with a cap, 610 with a bias and 827 with both);
// the same with a cap so wide that each key takes a form of its own.
enum { kPlain, kMasks, kScores, kWideScores };
// STATE: the rows' states for a merge instead of the output; the weights then
// go through the product with V as bf16 hi and lo (16 bits; lo in the half of
// S's columns that hi leaves), as the merged output is float32.
template <int D, int KIND, bool STATE>
__global__ void __launch_bounds__(kThreads, 1)
pages_chunk_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const PagedAttend p) {
    using L = Lay<D>;
    constexpr bool SCORED = KIND != kPlain;
    constexpr bool CHANGED = KIND == kScores || KIND == kWideScores;
    constexpr float kLazy = CHANGED ? kLazyScores : kLazyMax;
    constexpr uint32_t kColS = 0, kColO = 256;  // slot w: 128 w columns on
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const PagedSeqs& s = p.s;
    const int CS = (int)ptx::cluster_size(), rank = (int)ptx::cluster_rank();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    int* rng = reinterpret_cast<int*>(sm + L::info);  // [slot] {first key seen, end of the keys seen}
    uint32_t* tslot = reinterpret_cast<uint32_t*>(rng + 4);
    int* gapped = rng + 5;                              // end of the prefixes, begin of the windows seen
    if (warp == 1) ptx::tmem_alloc(ptx::smem_u32(tslot), kCols);  // beside the search
    if (tid == 0 || tid == 96) ptx::prefetch_map(tid ? &vmap : &kmap);
    // blocks of a sequence from its last (the one that sees most) to its first
    const int job = blockIdx.x / CS, g = job % s.Hk;
    pages::RowBlock b;
    if (!pages::find_block(s, p.G, kRows, job / s.Hk, b)) {  // the whole cluster's
        __syncthreads();
        if (warp == 1) ptx::tmem_dealloc(*tslot, kCols);
        return;
    }
    const int T = b.T;
    const int nblk = (b.n * p.G + kRows - 1) / kRows;
    const int r_begin = (nblk - 1 - b.blk) * kRows;
    const int nr = min(kRows, b.n * p.G - r_begin);
    const bool two = nr > kTile;  // two row tiles, or one in both slots
    // row r of the block: token row b.q0 + i_begin + div_group(j_begin + r), and the head of the group
    const int i_begin = r_begin / p.G, j_begin = r_begin - i_begin * p.G;

    const uint32_t b_full = ptx::smem_u32(sm + L::bars), b_empty = b_full + 8 * L::nst;
    const uint32_t b_s = ptx::smem_u32(sm + L::bar_s), b_p = ptx::smem_u32(sm + L::bar_p);
    const uint32_t b_o = ptx::smem_u32(sm + L::bar_o), b_fin = ptx::smem_u32(sm + L::bar_fin);
    if (tid == 0) {
        for (int i = 0; i < L::nst; ++i) {
            ptx::mbar_init(b_full + 8 * i, 1);
            ptx::mbar_init(b_empty + 8 * i, 2);  // both slots
        }
        for (int w = 0; w < 2; ++w) {
            ptx::mbar_init(b_s + 8 * w, 1);
            ptx::mbar_init(b_p + 16 * w, 8);  // P of the tile's first half, of its second
            ptx::mbar_init(b_p + 16 * w + 8, 8);
            ptx::mbar_init(b_o + 8 * w, 1);
            ptx::mbar_init(b_fin + 8 * w, 1);
            rng[2 * w] = INT_MAX;
            rng[2 * w + 1] = 0;
        }
        gapped[0] = 0;
        gapped[1] = INT_MAX;
        ptx::mbar_init_fence();
    }
    if constexpr (SCORED) __syncthreads();

    // softmax threads: their row and what it sees
    const int w = (warp - 4) / 8;          // slot
    const int part = ((warp - 4) / 4) & 1; // of a row: 32 keys of every 64, half the channels
    const int lr = tid & 127;              // row of the slot
    const int row = two ? w * kTile + lr : lr;
    const bool live = warp >= 4 && row < nr;
    Seen see = {0, INT_MAX, 0, 0};  // rows past the block: nothing to mask, dropped at the end
    int tok = 0, head = 0, pos = 0;
    if (live) {
        const int i = pages::div_group(p, j_begin + row);
        tok = b.q0 + i_begin + i;
        head = g * p.G + j_begin + row - i * p.G;
        pos = b.p0 + i_begin + i;
        see = pages::row_seen<SCORED>(p, b.seq, tok, pos, T);
    }
    // Q on its way to registers: 16-byte pieces, consecutive lanes on consecutive
    // pieces of a row, all of a thread's under way before the first is stored
    // (rows past the block repeat its last: a load under a condition waits for the
    // one before it, 16 thousand cycles in all instead of 4)
    constexpr int CH = D / 8;
    uint4 v[CH / 2];
    if (warp >= 4 && (two || w == 0)) {
        const int first = two ? w * kTile : 0;
#pragma unroll
        for (int k = 0; k < CH / 2; ++k) {
            const int x = k * 256 + (tid & 255), r = min(first + x / CH, nr - 1), c = x % CH;
            const int i = pages::div_group(p, j_begin + r);
            v[k] = ptx::ldg16(p.Q + (long long)(b.q0 + i_begin + i) * p.q_stride +
                              (long long)(g * p.G + j_begin + r - i * p.G) * D + c * 8);
        }
    }
    if constexpr (SCORED) {
        if (warp >= 4) {
            const int lo = __reduce_min_sync(0xffffffffu, live ? see.lo() : INT_MAX);
            const int hi = __reduce_max_sync(0xffffffffu, live ? see.hi() : 0);
            if (lane == 0 && hi > 0) {
                atomicMin(&rng[2 * w], lo);
                atomicMax(&rng[2 * w + 1], hi);
            }
            if (p.prefix && p.window > 0) {
                const int end = __reduce_max_sync(0xffffffffu, live ? see.prefix_end() : 0);
                const int begin = __reduce_min_sync(0xffffffffu, live ? see.window_lo() : INT_MAX);
                if (lane == 0) {
                    atomicMax(&gapped[0], end);
                    atomicMin(&gapped[1], begin);
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tslot;

    // end of the keys that a slot's rows see; with the causal mask alone the
    // last row sees most
    auto seen_end = [&](int slot) {
        if constexpr (SCORED) return rng[2 * slot + 1];
        const int last = two && slot == 0 ? kTile - 1 : nr - 1;
        return max(0, min(T, b.p0 + i_begin + pages::div_group(p, j_begin + last) + 1));
    };
    // this CTA's key tiles [ta, ta + n), counted without the gap: the cluster's
    // share of the tiles that any row sees; a slot takes those that its rows see
    // (two row tiles), or every second one. Few tiles are not split: the cluster's
    // first CTA takes them all, as a merge costs about what kFewTiles cost.
    const int hi = max(seen_end(0), seen_end(1));
    int t_lo = 0;
    if constexpr (SCORED) t_lo = hi > 0 ? min(rng[0], rng[2]) / kTile : 0;
    pages::Gap gap;
    if constexpr (SCORED) gap = pages::Gap(gapped[0], gapped[1], kTile);
    const int t_hi = gap.count((hi + kTile - 1) / kTile);
    const int S = t_hi - t_lo <= kFewTiles ? 1 : CS;
    const int per = (t_hi - t_lo + S - 1) / S;
    const int ta = t_lo + rank * per;
    const int n = max(0, min(t_hi, ta + per) - ta);
    // Modified scores take the tiles from the last to the first: with a bias by
    // distance the first then holds the maxima, and the reference hardly moves.
    auto tile_at = [&](int i) { return gap.number(CHANGED ? ta + n - 1 - i : ta + i); };
    auto tiles_of = [&](int slot) {
        if (!two) return (n - slot + 1) / 2;
        if (CHANGED) return n;  // (of the tiles that the other slot alone sees, the halves are passed over)
        return max(0, min(n, gap.count((seen_end(slot) + kTile - 1) / kTile) - ta));
    };
    if (rank >= S) {  // not a split block's: nothing to do, and nobody waits for this CTA
        if (warp == 1) ptx::tmem_dealloc(tmem, kCols);
        return;
    }
    const bool direct = S == 1 && two;  // a row has one state
    bool bad = false;
    float* rows = reinterpret_cast<float*>(sm);  // merge rows, once the tiles are done with

    if (warp < 4) {
        ptx::regs_dec<kRegsFew>();
        if (warp == 0 || warp == 3) {
            // ------------------------------------------------------- loaders
            const int P = 1 << s.pshift, np = kTile >> s.pshift;  // pages per tile
            const int32_t* table = s.table + (long long)b.seq * s.tstride;
            const int none = s.pages * (s.Hk << s.pshift);  // a row behind the last: reads as zeros
            // first token row of this lane's page of tile i, -1 for none
            auto page_row = [&](int i) {
                const int t = tile_at(i) * kTile + lane * P;
                if (i >= n || lane >= np || t >= T) return -1;
                const int page = __ldg(table + (t >> s.pshift));
                if (page < 0 || page >= s.pages) {
                    pages::flag(s.status, kPgBadPage);
                    return none;
                }
                return (page * s.Hk + g) << s.pshift;
            };
            auto load = [&](int e, int r, const CUtensorMap* map) {
                const int st = e % L::nst;
                const uint32_t bar = b_full + 8 * st;
                const int cnt = __popc(__ballot_sync(0xffffffffu, r >= 0));
                if (e >= L::nst) warp_wait(b_empty + 8 * st, ((e / L::nst) - 1) & 1, bad);
                if (lane == 0) ptx::mbar_expect_tx(bar, (uint32_t)(cnt * P * D * 2));
                __syncwarp();
                if (r >= 0) {
                    const uint32_t dst = ptx::smem_u32(sm + L::ring + st * L::stage) + lane * P * 128;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        ptx::tma_load_2d(dst + c * (kTile * 128), map, c * 64, r, bar);
                }
                __syncwarp();
            };
            // warp 0 loads K, warp 3 V, tile by tile together (a stage's wait by parity
            // needs its load before to be under way)
            int r0 = page_row(0), r1 = page_row(1);
            if (n > 0 && warp == 0) load(0, r0, &kmap);
            for (int i = 0; i < n; ++i) {
                const int r2 = page_row(i + 2);
                ptx::bar_sync(kBarLoad, 64);
                if (warp == 0) {
                    if (i + 1 < n) load(k_entry(i + 1), r1, &kmap);
                } else {
                    load(v_entry(i, n), r0, &vmap);
                }
                r0 = r1;
                r1 = r2;
            }
            ptx::bar_sync(kBarLoad, 64);
            // every requested tile has landed before the CTA may go on
            for (int e = max(0, 2 * n - L::nst); e < 2 * n; ++e) {
                bool late = false;
                warp_wait(b_full + 8 * (e % L::nst), (e / L::nst) & 1, late);
            }
        } else if (warp <= 2) {
            // ------------------------------------------------------ issuers
            // One warp per slot: what one of them waits for costs the other's MMAs
            // nothing (a single issuer's waits and commits, about 1000 cycles per tile,
            // left the tensor cores idle). The whole warp runs this with uniform
            // values; an elected lane issues.
            ptx::bar_sync(kBarQ, 64 + kSoftmax);  // Q is in shared memory
            auto uniform = [](auto x) { return __reduce_max_sync(0xffffffffu, x); };
            const int slot = uniform(warp - 1), nn = uniform(n), nt = uniform(tiles_of(slot));
            const bool pairs = __any_sync(0xffffffffu, two);
            const uint32_t tm = uniform(tmem), base = uniform(ptx::smem_u32(sm)), ring = base + L::ring;
            const uint32_t tS = tm + kColS + 128 * slot, tO = tm + kColO + 128 * slot;
            const uint32_t idS = ptx::idesc_bf16(kTile, kTile, 0, 0);
            const uint32_t idO = ptx::idesc_bf16(kTile, D, 0, 1);
            const uint32_t u_full = base + L::bars, u_empty = u_full + 8 * L::nst;
            const uint32_t u_s = base + L::bar_s + 8 * slot, u_p = base + L::bar_p + 16 * slot;
            const uint32_t u_o = base + L::bar_o + 8 * slot, u_fin = base + L::bar_fin + 8 * slot;
            const uint64_t dq = ptx::sdesc(base + (pairs ? slot : 0) * L::stage, 16, 1024);
            auto full = [&](int e) { warp_wait(u_full + 8 * (e % L::nst), (e / L::nst) & 1, bad); };
            auto release = [&](int e) { ptx::mma_commit_elect(u_empty + 8 * (e % L::nst)); };
            auto qk = [&](int e) {
                const uint64_t dk = ptx::sdesc(ring + (e % L::nst) * L::stage, 16, 1024);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t o = ((ks / 4) * (kTile * 128) + (ks % 4) * 32) >> 4;  // descriptor units
                    ptx::mma_f16_elect(tS, dq + o, dk + o, idS, ks > 0 ? 1u : 0u);
                }
                ptx::mma_commit_elect(u_s);
            };
            auto pv = [&](int e, int it) {
                const uint64_t dv = ptx::sdesc(ring + (e % L::nst) * L::stage, kTile * 128, 1024);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h) {
                        warp_wait(u_p + 8, it & 1, bad);
                        ptx::tc_fence_after();
                    }
#pragma unroll
                    for (int ks = 4 * h; ks < 4 * h + 4; ++ks) {  // P of 32 keys: 16 columns at S's 32
                        const uint32_t tP = tS + 32 * (ks / 2) + 8 * (ks % 2);
                        ptx::mma_f16_ta_elect(tO, tP, dv + ks * (2048 >> 4), idO, (it > 0 || ks > 0) ? 1u : 0u);
                        if constexpr (STATE) ptx::mma_f16_ta_elect(tO, tP + 16, dv + ks * (2048 >> 4), idO, 1u);
                    }
                    if (CHANGED && h == 0) ptx::mma_commit_elect(u_o);  // (it takes over 100 cycles)
                }
            };
            // The slots take turns: P V and the next Q K^T of one, then of the other, so
            // that one's softmax runs beside the other's MMAs. (Left to themselves both
            // run their MMAs and then their softmax at the same time, which took 1.3
            // times as long.) What a turn needs is waited for before it, what can be
            // done after it is.
            // it: turns so far; own: the slot has a tile in this turn, more: and one after it
            auto turn = [&](int it, bool own, int ev, bool more, int ek) {
                if (own) {
                    full(ev);
                    warp_wait(u_p, it & 1, bad);
                }
                if (more) full(ek);
                ptx::tc_fence_after();
                if (slot || it > 0) ptx::bar_sync(kBarTurn + slot, 64);
                if (own) pv(ev, it);
                if (more) qk(ek);
                ptx::bar_arrive(kBarTurn + 1 - slot, 64);
                if (own && !more) ptx::mma_commit_elect(u_fin);  // the slot's last MMAs
                if (own) release(ev);
                if (more) release(ek);
            };
            // a tile that the other slot alone works on: its K or V is not needed here
            auto pass = [&](int e) {
                full(e);
                if (lane == 0) ptx::mbar_arrive(u_empty + 8 * (e % L::nst));
            };
            if (pairs) {
                if (nn > 0) {
                    full(k_entry(0));
                    ptx::tc_fence_after();
                    if (nt > 0) {
                        qk(k_entry(0));
                        release(k_entry(0));
                    } else {
                        pass(k_entry(0));
                    }
                }
                for (int i = 0; i < nn; ++i) {
                    const int ev = v_entry(i, nn), ek = k_entry(i + 1);
                    turn(i, nt > i, ev, nt > i + 1, ek);
                    if (nt <= i) pass(ev);
                    if (nt <= i + 1 && i + 1 < nn) pass(ek);
                }
                if (nn > 0 && !slot) ptx::bar_sync(kBarTurn, 64);
            } else {
                // the other slot's tiles are let pass in the ring's order: a wait by
                // parity needs the stage's load before this one to be done, and the
                // one after it not to be
                for (int i = 0; i < min(nn, 2); ++i) {
                    if (i != slot) {
                        pass(k_entry(i));
                        continue;
                    }
                    full(k_entry(i));
                    ptx::tc_fence_after();
                    qk(k_entry(i));
                    release(k_entry(i));
                }
                for (int i = 0; i < nn; i += 2) {
                    if (slot) {
                        pass(v_entry(i, nn));
                        if (i + 2 < nn) pass(k_entry(i + 2));
                    }
                    turn(i >> 1, i + slot < nn, v_entry(i + slot, nn), i + 2 + slot < nn, k_entry(i + 2 + slot));
                    if (!slot) {
                        if (i + 1 < nn) pass(v_entry(i + 1, nn));
                        if (i + 3 < nn) pass(k_entry(i + 3));
                    }
                }
                if (nn > 0 && !slot) ptx::bar_sync(kBarTurn, 64);
            }
            if (nt > 0) {
                // waited for even after a timeout: no MMA still runs when the CTA goes on
                bool late = false;
                warp_wait(u_fin, 0, late);
                bad = bad || late;
            }
            __syncwarp();
        }
        if (bad && lane == 0) pages::flag(s.status, kPgTimeout);
        if (!direct) {
            ptx::bar_sync(kBarDone, kThreads);
            ptx::bar_sync(kBarRows, kThreads);
        }
    } else {
        ptx::regs_inc<kRegsMany>();
        float m = -CUDART_INF_F, l = 0.0f;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        // ------------------------------------------------------------ softmax
        if (two || w == 0) {
            unsigned char* dst = sm + w * L::stage;
            const int at = tid & 255;
#pragma unroll
            for (int k = 0; k < CH / 2; ++k) {
                const int x = k * 256 + at, r = x / CH, c = x % CH;
                *reinterpret_cast<uint4*>(dst + (c / 8) * (kTile * 128) + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = v[k];
            }
            ptx::fence_proxy_async();  // the MMAs read Q through the async proxy
        }
        ptx::bar_sync(kBarQ, 64 + kSoftmax);
        const int mine = tiles_of(w);
        const bool some = __any_sync(0xffffffffu, live);
        const float slope2 = SCORED && live && p.slopes ? __ldg(p.slopes + head) * 1.4426950408889634f : 0.0f;
        const uint32_t tS = tmem + kColS + 128 * w + lane_off, tO = tmem + kColO + 128 * w + lane_off;
        float* xch = reinterpret_cast<float*>(sm + L::pair) + w * kTile + lr;
        const uint32_t b_pair = kBarPair + 4 * w + (warp & 3);
        // both threads of a row: the maximum (or the sum, part 0's first) of their values
        auto joined = [&](float x, bool add) {
            if (!part) *xch = x;
            ptx::bar_sync(b_pair, 64);
            if (part) *xch = x = add ? *xch + x : fmaxf(*xch, x);
            ptx::bar_sync(b_pair, 64);
            return part ? x : *xch;
        };
        // keys of the part's 32 from k0 on that the row does not see: `unseen`
        auto mask = [&](int k0, uint32_t (&u)[32], float unseen) {
            uint32_t bits = span_bits(see.a1 - k0, see.b1 - k0, 0);
            if constexpr (SCORED) bits |= span_bits(see.a2 - k0, see.b2 - k0, 0);
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if (!(bits >> k & 1u)) u[k] = asu(unseen);
        };
        auto max_of = [&](const uint32_t (&u)[32]) {
            auto f = [&](int k) { return asf(u[k]); };
            float x[11];
#pragma unroll
            for (int k = 0; k < 10; ++k) x[k] = ptx::max3(f(3 * k), f(3 * k + 1), f(3 * k + 2));
            x[10] = fmaxf(f(30), f(31));
            return ptx::max3(ptx::max3(ptx::max3(x[0], x[1], x[2]), ptx::max3(x[3], x[4], x[5]), x[6]),
                             ptx::max3(x[7], x[8], x[9]), x[10]);
        };
        // the row's reference becomes mt (its maximum in both parts) where that passes
        // it; O, which no MMA works on, follows
        auto move_ref = [&](float mine_max, bool summed) {
            const float mt = joined(mine_max, false);
            const bool move = mt > m + kLazy || (m == -CUDART_INF_F && mt > m);
            if (summed) {
                // (in two steps: a maximum may have passed the reference by up to 2^128, and
                // ex2 gives 0 below 2^-126)
                const float al = move && m != -CUDART_INF_F ? ptx::ex2(0.5f * (m - mt)) : 1.0f;
                l = l * al * al;
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 32) {
                    uint32_t o[32];
                    ptx::tmem_ld32(tO + part * (D / 2) + c, o);
                    ptx::tmem_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = asu(asf(o[k]) * al * al);
                    ptx::tmem_st32x(tO + part * (D / 2) + c, o);
                }
                ptx::tmem_wait_st();
            }
            if (move) m = mt;
        };
        if (!SCORED && mine > 0 && some) {
            // The first reference is the maximum of the first half tile. (A row that
            // sees none of its keys sees none at all: the causal mask alone.)
            const int t0 = (ta + (two ? 0 : w)) * kTile;  // (plain scores: no gap)
            warp_wait(b_s + 8 * w, 0, bad);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
                uint32_t u[32];
                ptx::tmem_ld32(tS + c, u);
                ptx::tmem_wait_ld(u);
                mask(t0 + c, u, -CUDART_INF_F);
                m = fmaxf(m, max_of(u));
            }
            m *= p.scale_log2;
            // products of minus infinity alone are no reference: such a row is done again
            if (live && m == -CUDART_INF_F && see.some(t0, t0 + 64)) l = CUDART_NAN_F;
            ptx::bar_sync(b_pair, 64);  // P of either part overwrites what both have read
        }
        float top = -CUDART_INF_F;  // the part's maximum in the tile before
        const float scale = CHANGED ? 1.0f : p.scale_log2;  // of scores in units of log2 already, or not
        // the scores of the part's 32 keys from k0 on, -inf where the row sees none
        auto in_log2 = [&](int k0, bool whole, uint32_t (&u)[32]) {
            if constexpr (CHANGED) {
                const bool behind = p.slopes && __all_sync(0xffffffffu, !live || pos >= k0 + 31);
                // (what an unseen place holds has no say in the form that a cap takes)
                if (!whole && p.cap2 > 0.0f) mask(k0, u, 0.0f);
                pages::scores32<KIND == kWideScores>(p, *reinterpret_cast<float (*)[32]>(u), slope2, pos, k0, behind, live);
            }
            if (!whole) mask(k0, u, -CUDART_INF_F);
        };
        for (int it = 0; it < mine; ++it) {
            const int i = two ? it : 2 * it + w;  // tile of this CTA
            const int t0 = tile_at(i) * kTile;
            // A maximum that passes the reference by 2^8 moves it: where scores cost much
            // to form or may rise fast (CHANGED) at once, else before the next tile (until
            // then the weights are that much larger, which float32 has room for up to 2^128;
            // rows beyond it come out infinite and are done again). The two threads of a row
            // ask one another while S is on its way.
            const bool moves = !CHANGED && it > 0 && some && ptx::bar_or(b_pair, 64, top > m + kLazy);
            warp_wait(b_s + 8 * w, it & 1, bad);
            ptx::tc_fence_after();
            // keys behind the sequence's end: whatever their V holds becomes 0 (a
            // weight of 0 times NaN would be NaN); each slot for itself. (After S: what
            // the ring's stage held before this V has then been used, so the parity
            // waited for is this load's and not that of the one before the last.)
            if (t0 + kTile > T) {
                const int e = v_entry(i, n);
                warp_wait(b_full + 8 * (e % L::nst), (e / L::nst) & 1, bad);
                if (t0 + lr >= T) {
                    unsigned char* v = sm + L::ring + (e % L::nst) * L::stage + lr * 128;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const int ch = part * (D / 16) + c;
                        *reinterpret_cast<uint4*>(v + (ch / 8) * (kTile * 128) + (ch % 8) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                ptx::fence_proxy_async();
            }
            if (!some) {  // no row of this warp: only the barriers' counts
                __syncwarp();
                if (lane < 2) ptx::mbar_arrive(b_p + 16 * w + 8 * lane);
                continue;
            }
            // (S came after every P V before it: O rests)
            if (moves) move_ref(top, true);
            top = -CUDART_INF_F;
            // a row's first keys are its first reference (both of its warps see that)
            if (KIND == kMasks && __any_sync(0xffffffffu, live && m == -CUDART_INF_F && see.some(t0, t0 + kTile))) {
#pragma unroll 1
                for (int k0 = t0 + 32 * part; k0 < t0 + kTile; k0 += 64) {
                    uint32_t u[32];
                    ptx::tmem_ld32(tS + (k0 - t0), u);
                    ptx::tmem_wait_ld(u);
                    in_log2(k0, false, u);
                    top = fmaxf(top, max_of(u) * scale);
                }
                if (ptx::bar_or(b_pair, 64, top > m + kLazy || (m == -CUDART_INF_F && top > m))) move_ref(top, it > 0);
            }
            // The tile's keys in two halves, so that P V of the first runs while P of
            // the second is formed; a thread has 32 keys of each.
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int half = t0 + 64 * h, k0 = half + 32 * part;  // first keys of the half, of the part
                const uint32_t tSh = tS + 64 * h + 32 * part;
                const bool whole = __all_sync(0xffffffffu, see.all(k0, k0 + 32));
                // nothing seen by either part (beyond the diagonal, other documents): weights
                // of 0 whatever S holds (with the causal mask alone these are the diagonal's
                // few, and the test costs every tile more than they save)
                const bool any = !SCORED || __any_sync(0xffffffffu, live && see.some(half, half + 64));
                uint32_t pw[16], pl[STATE ? 16 : 1];
                float2 sum[2] = {};
                if (any) {
                    uint32_t u[32];
                    ptx::tmem_ld32(tSh, u);
                    ptx::tmem_wait_ld(u);
                    in_log2(k0, whole, u);
                    const float x = max_of(u) * scale;
                    if constexpr (CHANGED) {
                        if (ptx::bar_or(b_pair, 64, x > m + kLazy || (m == -CUDART_INF_F && x > m))) {
                            if (h) {  // (S came after every P V but the first half's)
                                warp_wait(b_o + 8 * w, it & 1, bad);
                                ptx::tc_fence_after();
                            }
                            move_ref(x, it > 0 || h > 0);
                        }
                    } else {
                        top = fmaxf(top, x);
                    }
                    const float ref = m == -CUDART_INF_F ? 0.0f : m;
                    const float2 sc = make_float2(scale, scale), nm = make_float2(-ref, -ref);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 d = __ffma2_rn(make_float2(asf(u[2 * k]), asf(u[2 * k + 1])), sc, nm);
                        const float2 e = make_float2(ptx::ex2(d.x), ptx::ex2(d.y));
                        sum[k & 1] = __fadd2_rn(sum[k & 1], e);
                        pw[k] = pack_bf2(e.x, e.y);
                        if constexpr (STATE)
                            pl[k] = pack_bf2(e.x - asf(pw[k] << 16), e.y - asf(pw[k] & 0xFFFF0000u));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) pw[k] = 0u;
                }
                // P over the part's own columns of S
                ptx::tmem_st16(tSh, pw);
                if constexpr (STATE) ptx::tmem_st16(tSh + 16, pl);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_p + 16 * w + 8 * h);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
        }
        if (mine > 0) {
            warp_wait(b_fin + 8 * w, 0, bad);  // every MMA of the slot
            ptx::tc_fence_after();
        }
        if (bad && lane == 0) pages::flag(s.status, kPgTimeout);
        __syncwarp();

        // careful_row of this warp's row `of` (a lane), over the slot's tiles or all of the CTA's
        auto careful = [&](int of, bool all, float& cm, float& cl, float (&acc)[D / 32]) {
            Seen se;
            se.a1 = __shfl_sync(0xffffffffu, see.a1, of);
            se.b1 = __shfl_sync(0xffffffffu, see.b1, of);
            se.a2 = __shfl_sync(0xffffffffu, see.a2, of);
            se.b2 = __shfl_sync(0xffffffffu, see.b2, of);
            pages::careful_row<D, SCORED>(p, b.seq, __shfl_sync(0xffffffffu, tok, of),
                                          __shfl_sync(0xffffffffu, head, of), __shfl_sync(0xffffffffu, pos, of), se,
                                          gap, 7, two || all ? ta : ta + (CHANGED ? (n - 1 - w) & 1 : w), ta + n,
                                          two || all ? 1 : 2, cm, cl, acc);
        };
        l = joined(l, true);
        bool odd = live && l != 0.0f && !finite(l);  // sums that a masked key may have spoilt
        uint32_t* flags = reinterpret_cast<uint32_t*>(sm + L::pair + 2 * kTile * 4) + 4 * w + (warp & 3);
        // A state that another is merged with has its l within 2^-32 ... 2^64 of its m:
        // a last tile's maxima may lie far above the reference, up to where the other
        // state's weight of it (ex2 of the references' difference, 0 below 2^-126) would
        // lose the larger part of a row.
        const bool high = l > 0x1p32f;
        const float down = high ? 0x1p-64f : 1.0f;
        const float state_m =
            l == 0.0f ? -CUDART_INF_F : (m == -CUDART_INF_F ? 0.0f : m) + (high ? 64.0f : 0.0f);
        // a row's last numbers: m and l, or their logarithm
        auto finish = [&](int t, int hd, float rm, float rl) {
            if constexpr (STATE)
                *pages::state_ml(p, t, hd) = make_float2(rm, rl);
            else if (p.lse)
                p.lse[(long long)t * p.Hq + hd] = rl == 0.0f ? -CUDART_INF_F : (rm + log2f(rl)) * kLn2;
        };
        // rows `odds` of the warp again, over the CTA's tiles, and their output
        auto again = [&](unsigned odds) {
            for (; odds; odds &= odds - 1) {
                const int of = __ffs(odds) - 1;
                float cm, cl, acc[D / 32];
                careful(of, true, cm, cl, acc);
                const int ct = __shfl_sync(0xffffffffu, tok, of), ch = __shfl_sync(0xffffffffu, head, of);
                const long long at = ((long long)ct * p.Hq + ch) * D + lane * (D / 32);
#pragma unroll
                for (int e = 0; e < D / 32; ++e) {
                    if constexpr (STATE) p.st_acc[at + e] = acc[e];
                    else p.out[at + e] = cl == 0.0f ? (uint16_t)0 : __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] / cl));
                }
                if (lane == 0) finish(ct, ch, cm, cl);
            }
        };
        // 32 channels from c on of this thread's row
        auto store32 = [&](int c, const float (&y)[32]) {
            const long long at = ((long long)tok * p.Hq + head) * D + c;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                if constexpr (STATE) {
                    *reinterpret_cast<float4*>(p.st_acc + at + k) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                    *reinterpret_cast<float4*>(p.st_acc + at + k + 4) = make_float4(y[k + 4], y[k + 5], y[k + 6], y[k + 7]);
                } else {
                    *reinterpret_cast<uint4*>(p.out + at + k) =
                        make_uint4(pack_bf2(y[k], y[k + 1]), pack_bf2(y[k + 2], y[k + 3]), pack_bf2(y[k + 4], y[k + 5]),
                                   pack_bf2(y[k + 6], y[k + 7]));
                }
            }
        };
        // a row's channels of this thread
        constexpr int HC = D / 2;
        const int c0 = part * HC;
        if (direct) {
            // The slot's Q (no MMA reads it any more) takes the output as bf16, and the
            // two warps write whole rows of it, 16 each.
            const float inv = STATE ? down : 1.0f / l;  // (not used where l is 0)
            unsigned char* stage = sm + w * L::stage + (warp & 3) * 32 * (D * 2);
#pragma unroll 1
            for (int c = c0; c < c0 + HC; c += 32) {
                uint32_t o[32];
                float y[32];
                ptx::tmem_ld32(tO + c, o);
                ptx::tmem_wait_ld(o);
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    odd = odd || (live && l != 0.0f && !finite(asf(o[k])));
                    y[k] = l == 0.0f ? 0.0f : asf(o[k]) * inv;
                }
                if constexpr (STATE) {
                    if (live) store32(c, y);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
                        *reinterpret_cast<uint4*>(stage + lane * (D * 2) + ((((c + k) / 8) ^ (lane & 7)) << 4)) =
                            make_uint4(pack_bf2(y[k], y[k + 1]), pack_bf2(y[k + 2], y[k + 3]),
                                       pack_bf2(y[k + 4], y[k + 5]), pack_bf2(y[k + 6], y[k + 7]));
                }
            }
            if (live && !part) finish(tok, head, state_m, l * down);
            const unsigned odds = __ballot_sync(0xffffffffu, odd);
            if (part && lane == 0) *flags = odds;
            ptx::bar_sync(b_pair, 64);
            if constexpr (!STATE) {
                const long long at = live ? ((long long)tok * p.Hq + head) * D : -1;
#pragma unroll
                for (int k = 0; k < CH / 2; ++k) {
                    const int x = k * 32 + lane, r = 16 * part + x / CH, c = x % CH;
                    const long long to = __shfl_sync(0xffffffffu, at, r);
                    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * (D * 2) + ((c ^ (r & 7)) << 4));
                    if (to >= 0) *reinterpret_cast<uint4*>(p.out + to + c * 8) = v;
                }
                ptx::bar_sync(b_pair, 64);  // both warps' rows are written
            }
            if (!part) again(odds | *flags);  // (writes odd rows once more)
        } else {
            // states into shared memory, once no MMA reads the tiles any more and
            // every load has landed
            ptx::bar_sync(kBarDone, kThreads);
            float* dst = rows + (w * kTile + lr) * L::rs;
#pragma unroll
            for (int c = c0; c < c0 + HC; c += 32) {
                uint32_t o[32];
                ptx::tmem_ld32(tO + c, o);
                ptx::tmem_wait_ld(o);
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 v = make_float4(asf(o[k]), asf(o[k + 1]), asf(o[k + 2]), asf(o[k + 3]));
                    odd = odd || (live && l != 0.0f && !(finite(v.x) && finite(v.y) && finite(v.z) && finite(v.w)));
                    *reinterpret_cast<float4*>(dst + c + k) =
                        make_float4(v.x * down, v.y * down, v.z * down, v.w * down);
                }
            }
            if (!part) {
                dst[D] = state_m;
                dst[D + 1] = l * down;
            }
            const unsigned mine_odd = __ballot_sync(0xffffffffu, odd);
            if (part && lane == 0) *flags = mine_odd;
            ptx::bar_sync(b_pair, 64);
            for (unsigned odds = part ? 0u : mine_odd | *flags; odds; odds &= odds - 1) {
                const int of = __ffs(odds) - 1;
                float cm, cl, acc[D / 32];
                careful(of, false, cm, cl, acc);
                float* to = rows + (w * kTile + (warp & 3) * 32 + of) * L::rs;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) to[lane * (D / 32) + e] = acc[e];
                if (lane == 0) to[D] = cm, to[D + 1] = cl;
                __syncwarp();
            }
            ptx::bar_sync(kBarRows, kThreads);
        }
    }

    if (!direct) {
        // The rows' states, merged over the slots and the cluster: each CTA takes
        // a share of the rows. First a thread per row: the states' weights (with
        // the division by the sum in them); then 4 channels per item, the states'
        // loads all under way before the first is used.
        if (S > 1) {
            ptx::cluster_arrive();
            ptx::cluster_wait();
        }
        const int slots = two ? 1 : 2, parts = slots * S;  // states of a row; k-th: slot k % slots of CTA k / slots
        const int share = (nr + S - 1) / S, r0 = rank * share, cnt = max(0, min(nr - r0, share));
        float* weights = rows + kRows * L::rs;  // [share][parts]
        auto state = [&](int r, int k) {
            return ptx::dsmem_addr(rows + (r0 + r + (k % slots) * kTile) * L::rs, k / slots);
        };
        auto out_at = [&](int r) {  // the share's row r: token row and head
            const int i = pages::div_group(p, j_begin + r0 + r);
            return make_int2(b.q0 + i_begin + i, g * p.G + j_begin + r0 + r - i * p.G);
        };
        for (int r = tid; r < cnt; r += kThreads) {
            float2 ml[kMaxParts];
#pragma unroll
            for (int k = 0; k < kMaxParts; ++k)
                ml[k] = k < parts ? ptx::ld_dsmem2(state(r, k) + D * 4) : make_float2(-CUDART_INF_F, 0.0f);
            float M = -CUDART_INF_F, Lt = 0.0f;
#pragma unroll
            for (int k = 0; k < kMaxParts; ++k) M = fmaxf(M, ml[k].x);
#pragma unroll
            for (int k = 0; k < kMaxParts; ++k) {
                ml[k].x = ml[k].y == 0.0f ? 0.0f : ptx::ex2(ml[k].x - M);  // a state of nothing: 0
                Lt = fmaf(ml[k].x, ml[k].y, Lt);
            }
            const float inv = STATE ? 1.0f : Lt == 0.0f ? 0.0f : 1.0f / Lt;
#pragma unroll
            for (int k = 0; k < kMaxParts; ++k)
                if (k < parts) weights[r * parts + k] = ml[k].y == 0.0f ? -1.0f : ml[k].x * inv;
            const int2 at = out_at(r);
            if constexpr (STATE)
                *pages::state_ml(p, at.x, at.y) = make_float2(M, Lt);
            else if (p.lse)
                p.lse[(long long)at.x * p.Hq + at.y] = Lt == 0.0f ? -CUDART_INF_F : (M + log2f(Lt)) * kLn2;
        }
        __syncthreads();
        constexpr int C4 = D / 4;
#pragma unroll 2
        for (int x = tid; x < cnt * C4; x += kThreads) {
            const int r = x / C4, c4 = x % C4;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < parts; k0 += 4) {
                float4 v[4];
                float f[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    f[u] = -1.0f;
                    if (k0 + u < parts) {
                        v[u] = ptx::ld_dsmem4(state(r, k0 + u) + c4 * 16);
                        f[u] = weights[r * parts + k0 + u];
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (f[u] < 0.0f) continue;  // a state of nothing, whatever its O holds
                    a.x = fmaf(f[u], v[u].x, a.x), a.y = fmaf(f[u], v[u].y, a.y);
                    a.z = fmaf(f[u], v[u].z, a.z), a.w = fmaf(f[u], v[u].w, a.w);
                }
            }
            const int2 ot = out_at(r);
            const long long at = ((long long)ot.x * p.Hq + ot.y) * D + c4 * 4;
            if constexpr (STATE) *reinterpret_cast<float4*>(p.st_acc + at) = a;
            else *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf2(a.x, a.y), pack_bf2(a.z, a.w));
        }
        if (S > 1) {  // no CTA goes away while another reads its rows
            ptx::cluster_arrive();
            ptx::cluster_wait();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kCols);
    }
}

// Per instance and device, once: the shared memory opted in, and how many
// clusters of 1, 2, 4 and 8 CTAs the GPU holds at once (a cluster's CTAs share
// a group of SMs whose number need not be a multiple).
struct Fit {
    cudaError_t err = cudaSuccess;
    int clusters[4] = {};
};
template <int D, int KIND, bool STATE>
const Fit& fit(int device) {
    static std::once_flag once[kPagedDevices];
    static Fit fits[kPagedDevices];
    std::call_once(once[device], [device] {
        auto kern = pages_chunk_kernel<D, KIND, STATE>;
        Fit& x = fits[device];
        x.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::total);
        for (int i = 0; i < 4 && x.err == cudaSuccess; ++i) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1 << i, 1, 1);
            cfg.blockDim = dim3(kThreads, 1, 1);
            cfg.dynamicSmemBytes = Lay<D>::total;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1 << i;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            x.err = cudaOccupancyMaxActiveClusters(&x.clusters[i], kern, &cfg);
        }
    });
    return fits[device];
}

template <int D, int KIND, bool STATE>
cudaError_t launch(const PagedAttend& a, int max_q, int max_kv, cudaStream_t st) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device >= kPagedDevices) return cudaErrorInvalidDevice;
    const Fit& f = fit<D, KIND, STATE>(device);
    if (f.err != cudaSuccess) return f.err;
    const long long rows = (long long)a.s.tokens * a.G;
    const long long blocks = rows / kRows + a.s.seqs;  // at least as many as there are
    // about as many as there are, and the key tiles of one (in halves where one
    // row tile has both slots)
    const long long per_seq = ((long long)max_q * a.G + kRows - 1) / kRows;
    const long long jobs = std::min(rows / kRows + (a.s.seqs + 1) / 2, a.s.seqs * per_seq) * a.s.Hk;
    const bool one = (long long)max_q * a.G <= kTile;
    const int ntiles = std::max(1, (max_kv + kTile - 1) / kTile);
    int split = 1;
    long long best = -1;
    for (int i = 0; i < 4 && f.clusters[i] > 0; ++i) {
        const int S = 1 << i;
        if (S > 1 && ntiles <= kFewTiles) break;
        // the time of the GPU's slots in key tiles (2.5 thousand cycles): waves x
        // (tiles of a CTA, and about five for its start and end, ten with a merge
        // over the cluster; seven and fourteen choose the same)
        const long long tiles = (ntiles + S - 1) / S;
        const long long cost =
            (std::max(1LL, jobs) + f.clusters[i] - 1) / f.clusters[i] * ((one ? (tiles + 1) / 2 : tiles) + (S > 1 ? 10 : 5));
        if (best < 0 || cost < best) best = cost, split = S;
    }
    if (split * blocks * a.s.Hk > INT_MAX) return cudaErrorInvalidValue;
    CUtensorMap kmap, vmap;
    const long long trows = (long long)a.s.pages * a.s.Hk << a.s.pshift;
    if (!make_page_map(&kmap, a.K, D, trows, 1 << a.s.pshift) || !make_page_map(&vmap, a.V, D, trows, 1 << a.s.pshift))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split * blocks * a.s.Hk), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Lay<D>::total;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pages_chunk_kernel<D, KIND, STATE>, kmap, vmap, a);
}

}  // namespace

cudaError_t launch_pages_chunk(const PagedAttend& a, int head_dim, int max_q, int max_kv, cudaStream_t st) {
    const int kind = a.cap2 > pages::kWideCap2        ? kWideScores
                     : a.cap2 > 0.0f || a.slopes ? kScores
                     : paged_scored(a)           ? kMasks
                                                 : kPlain;
#define KVP_PG_CHUNK(KK, SS) \
    (head_dim == 64 ? launch<64, KK, SS>(a, max_q, max_kv, st) : launch<128, KK, SS>(a, max_q, max_kv, st))
    if (a.st_acc) return KVP_PG_CHUNK(kPlain, true);
    if (kind == kWideScores) return KVP_PG_CHUNK(kWideScores, false);
    if (kind == kScores) return KVP_PG_CHUNK(kScores, false);
    return kind == kMasks ? KVP_PG_CHUNK(kMasks, false) : KVP_PG_CHUNK(kPlain, false);
#undef KVP_PG_CHUNK
}

}  // namespace kvp
