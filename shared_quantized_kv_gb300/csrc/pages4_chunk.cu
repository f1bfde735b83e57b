// Attention of many query rows per sequence over its pages in 4 bits: chunks of
// new tokens, whole prompts (sm_103a, tcgen05).
//
// Mathematics as in pages4_rows.cu for the values: O = H (sum p t' c'), c = u -
// 7.5 of the codes, one pass with a running reference maximum; V's operand is bf16
// c, exactly, and the weights p t' are rounded to bf16 once (off by 2^-8 of each at
// most). The scores are taken the other way round: <q, k> = t <q, H c>, as H c = H
// (u - 8) + (D / 2) e_0 is a vector of whole numbers up to 8 D + D / 2, which fp16
// holds exactly, and so is q (bf16) once a power of two has brought the row's
// largest value into [8, 16) (what lies 2^18 and more below it loses bits that are
// 2^-29 of it). So the products are exact, with one MMA per operand pair;
// transformed queries would need two fp16 parts (one alone is off by 2^-11, which
// the log of the sum of a row with few keys shows), for which shared memory has no
// room. The transform is H16 x H8 (H4 with D = 64): the first by small matrix
// products, the second by additions.
//
// Bound: the tensor cores, 4 D FLOP per (row, key), with the instructions that
// make operands of codes and weights of scores close behind. The frame is that
// of pages_chunk.cu: up to 256 rows of one sequence and KV head per CTA, two
// slots of tensor memory worked on in turn, key tiles of 128 in two stages of K and
// two of V, a cluster's CTAs on shares of the keys. What differs is where tiles come
// from. With a workspace a kernel before makes each once (codes expanded into the
// swizzled tile that the MMAs read, and its scales), and loaders copy them in bulk.
// Without, or for sequences longer than it has room for, six warps of the CTA read
// the codes (by copies into small rings of their own) and expand them, which each
// CTA does anew.
//   warps 1, 2    issuers of the MMAs, one per slot
//   warps 4-19    softmax, two threads per row of a slot: 32 keys of every 64
//                 each, and half the channels of the output
//   warps 0, 3    loaders of K with the scales, and of V; or expanders of V, 64
//                 keys of every tile each
//   warps 20-23   expanders of K, 32 keys of every tile each (without a workspace)
// Every wait on a barrier in memory is bounded; one that expires is recorded in
// the status word, and the CTA runs to its end without waiting again.
//
// Measured on 2,048 new tokens over 16K keys, 32 query heads on 8 of 128: 443 us
// with a workspace, 15 of them to make it (1.16 PFLOP/s; the bf16 pages take 352), 748
// without. The scales cost most beside the products: a version without their
// multiplications took 344 us. What got it there, without a workspace at first: one
// warp group for K and V 1001 us, V by the two warps that had nothing to do 765,
// registers for K's expanders 743; the workspace 546; scales asked for while S is on
// its way 521; four rows to a lane and no test of the scales 467; queries asked for at
// once and the output's transform in registers 448; K's and V's tiles made apart 442.
// Keys' operands with their scales in them, in fp16 (652 us against 743 without a
// workspace), leave the log of the sum 1e-5 off, which rows of few keys show.
#include <algorithm>
#include <mutex>

#include "pages4.cuh"

namespace kvp {
namespace {

using pages::Seen;

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
// a slot's turn at the tensor cores; the two warps of 32 rows (8 barriers); the rows' factors are read
constexpr uint32_t kBarQ = 1, kBarDone = 2, kBarRows = 3, kBarTurn = 4, kBarPair = 6, kBarRead = 14;
constexpr int kSoftmax = 512;           // softmax threads
constexpr int kEarly = 4;               // scales (in fours) asked for before S has come
// expander warps of K (20 to 23, 32 keys of a tile each) and of V (0 and 3, 64 each), and how many times 32 keys'
// codes their own rings hold
constexpr int kWarpsK = 4, kWarpsV = 2, kRawK = 2, kRawV = 3;
constexpr float kLn2 = 0.6931471805599453f;
// MADE: the tiles lie in a workspace, made before (no expanders). Registers of the warpgroups of warps 0 to 3, of the
// softmax (4 of them), of K's expanders: 56 + 4 x 88 + 72 = 6 x 80, and 64 + 4 x 104 = 5 x 96 at launch.
template <bool MADE>
struct Shape {
    static constexpr int threads = MADE ? 640 : 768;
    static constexpr int regs_issue = MADE ? 64 : 56, regs_many = MADE ? 104 : 88, regs_expand = 72;
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < CUDART_INF_F; }

// What the softmax needs to know of a tile's scales, beside the ring: a slot per tile
// (where V's is not finite: 0, and K's NaN. A row that sees the key then has a sum that is NaN and is done again key by
// key; for others, whose weight of it is 0, nothing has to be looked at. The same where K's scale is so
// large that it may overflow times the sum of a row's values, up to 16, and the key's whole numbers, 2^18 at most,
// although the row's factor would bring the score back.)
constexpr float kMostScale = 0x1p108f;
struct TileScales {
    float v[kTile];
    float k[kTile];
    __device__ __forceinline__ void set(int key, float tk, float tv) {
        v[key] = finite(tv) ? tv : 0.0f;
        k[key] = finite(tv) && fabsf(tk) <= kMostScale ? tk : CUDART_NAN_F;
    }
};
// A tile in the workspace, as shared memory takes it: K, V, the scales.
template <int D>
constexpr int made_bytes() { return 2 * kTile * D * 2 + (int)sizeof(TileScales); }
static_assert(made_bytes<64>() % 128 == 0 && made_bytes<128>() % 128 == 0 && sizeof(TileScales) % 16 == 0, "alignment");

template <int D, bool MADE>
struct Lay {
    static constexpr int stage = kTile * D * 2;  // a K or V tile
    static constexpr int nst = D == 128 ? 2 : 4; // of K, and as many of V
    // A tile's scales are written before its K: by then the K of nst tiles before is
    // released, and a softmax may still be at the tile before that one (where the
    // slots take every second tile, one lets the other's next K pass early).
    static constexpr int slots = nst + 2;
    static constexpr int ring = 2 * stage;       // after the two Q tiles: K's stages, then V's
    static constexpr int codes = 32 * D / 2;     // of 32 keys
    static constexpr int raw = ring + 2 * nst * stage;
    static constexpr int scales = raw + (MADE ? 0 : (kWarpsK * kRawK + kWarpsV * kRawV) * codes);
    static constexpr int bars = scales + slots * (int)sizeof(TileScales);
    // barriers: full, empty per stage of K, of V; per slot S, P (of each half), P V of the first, all done
    static constexpr int bar_s = bars + 4 * nst * 8, bar_p = bar_s + 16, bar_o = bar_p + 32, bar_fin = bar_o + 16;
    static constexpr int info = bar_fin + 16;  // rng[2][2], tensor memory address, prefixes' end, windows' begin
    static constexpr int pair = info + 32;       // per slot a float per row (the rows' factors before), then a word per 32 rows
    static constexpr int total = pair + 2 * kTile * 4 + 32 + 1024;  // + alignment of the base
    static constexpr int rs = D + 4;             // floats of a merge row: O, m, l
    static_assert(kRows * (rs + kMaxParts) * 4 <= raw, "merge rows and weights fit in the tiles");
    static_assert(total <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float asf(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t asu(float f) { return __float_as_uint(f); }

// Wait for phase `parity` of the barrier by a whole warp; after kTries tries
// (each suspends the warp for a while; about a quarter of a second in all) `bad` is set, and
// no wait after that waits.
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// bits k of [32 c, 32 c + 32) with a <= 32 c + k < b
__device__ __forceinline__ uint32_t span_bits(int a, int b, int c) {
    const int x = min(max(a - 32 * c, 0), 32), y = min(max(b - 32 * c, 0), 32);
    if (y <= x) return 0u;
    const uint32_t upto = y == 32 ? 0xffffffffu : (1u << y) - 1u;
    return upto & ~(x == 32 ? 0xffffffffu : (1u << x) - 1u);
}

__device__ __forceinline__ uint32_t mask_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
    return y;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
// codes in bits 0-3 of both halves -> fp16 u - 8
__device__ __forceinline__ uint32_t k_pair(uint32_t x) {
    return hadd2(mask_or(x, 0x000F000Fu, 0x64006400u), 0xE408E408u);
}
// d = A (16 keys x 16 channels) B (16 x 8) in fp16: whole numbers, exactly
__device__ __forceinline__ void mma_half(uint32_t& d0, uint32_t& d1, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f16.f16.f16.f16 {%0,%1}, {%2,%3,%4,%5}, {%6,%7}, {%8,%8};"
        : "=r"(d0), "=r"(d1)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0u));
}
// a word's eight channels as bf16 u - 7.5, exactly: 64 + u - 71.5
__device__ __forceinline__ uint4 v_operand(uint32_t w) {
    auto one = [](uint32_t x) {
        const uint32_t y = mask_or(x, 0x001E001Eu, 0x42804280u);
        uint32_t z;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(y), "r"(0xC28FC28Fu));
        return z;
    };
    return make_uint4(one(w << 1), one(w >> 3), one(w >> 7), one(w >> 11));
}

// H16's columns as operands: entry (k, n) is -1 to the ones that k and n share.
__device__ __forceinline__ void h16_operands(uint32_t (&h16)[2][2]) {
    const int lane = threadIdx.x & 31, quad = lane >> 2, qi = lane & 3;
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            auto sign = [&](int k) { return __popc(k & (quad + 8 * nb)) & 1 ? 0xBC00u : 0x3C00u; };
            h16[nb][y] = sign(2 * qi + 8 * y) | sign(2 * qi + 8 * y + 1) << 16;
        }
}
// A warp's 32 keys from key0 of a tile on: H (u - 7.5) of their codes `own`, into
// the tile. 16 keys at a time are a matrix operand (u - 8) whose 16 channels of a
// group the product with H16 transforms; the groups' results then go through the
// last stages in registers. half_sum: D / 2 where the lane has channel 0.
template <int D>
__device__ __forceinline__ void expand_k(const unsigned char* own, unsigned char* stage, int key0, const uint32_t (&h16)[2][2],
                                         uint32_t half_sum) {
    const int lane = threadIdx.x & 31, quad = lane >> 2, qi = lane & 3;
    constexpr int kGroups = D / 16;
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {  // keys 16 x + quad and + 8
        uint32_t z[2][kGroups][2];  // [key][group][half of its channels]
#pragma unroll
        for (int g2 = 0; g2 < kGroups / 2; ++g2) {  // two groups: four words
            uint4 w[2];
#pragma unroll
            for (int y = 0; y < 2; ++y)
                w[y] = *reinterpret_cast<const uint4*>(own + (16 * x + 8 * y + quad) * (D / 2) + g2 * 16);
            const int sh = 4 * qi;
            const uint32_t a0 = k_pair(w[0].x >> sh), a1 = k_pair(w[1].x >> sh);
            const uint32_t a2 = k_pair(w[0].y >> sh), a3 = k_pair(w[1].y >> sh);
            const uint32_t c0 = k_pair(w[0].z >> sh), c1 = k_pair(w[1].z >> sh);
            const uint32_t c2 = k_pair(w[0].w >> sh), c3 = k_pair(w[1].w >> sh);
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
                mma_half(z[0][2 * g2][nb], z[1][2 * g2][nb], a0, a1, a2, a3, h16[nb][0], h16[nb][1]);
                mma_half(z[0][2 * g2 + 1][nb], z[1][2 * g2 + 1][nb], c0, c1, c2, c3, h16[nb][0], h16[nb][1]);
            }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int h = 1; h < kGroups; h <<= 1)
#pragma unroll
                    for (int q = 0; q < kGroups; ++q)
                        if (!(q & h)) {
                            const uint32_t a = z[y][q][nb], c = z[y][q + h][nb];
                            z[y][q][nb] = hadd2(a, c), z[y][q + h][nb] = hsub2(a, c);
                        }
            z[y][0][0] = hadd2(z[y][0][0], half_sum);
            // channels 16 q + 8 nb + 2 qi and the next: 4 bytes of piece 2 q + nb
            const int key = key0 + 16 * x + 8 * y + quad;  // (key & 7 is quad)
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    const int pc = 2 * q + nb;
                    *reinterpret_cast<uint32_t*>(stage + (pc / 8) * (kTile * 128) + key * 128 +
                                                 (((pc % 8) ^ quad) << 4) + 4 * qi) = z[y][q][nb];
                }
        }
    }
}
// The same of V: u - 7.5 as they are. D / 8 lanes take a key, a word each, which becomes 16 bytes of its row.
template <int D>
__device__ __forceinline__ void expand_v(const unsigned char* own, unsigned char* stage, int key0) {
    constexpr int kLanes = D / 8, kKeys = 32 / kLanes;  // lanes of a key, keys at a time
    const int lane = threadIdx.x & 31, in_row = lane % kLanes, in_key = lane / kLanes;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(own) + lane;
    unsigned char* to = stage + (in_row / 8) * (kTile * 128) + (key0 + in_key) * 128;
    const uint32_t piece = (in_row % 8) ^ (in_key & 7);  // ((key & 7) changes by kKeys at a time)
#pragma unroll 8
    for (int j = 0; j < 32 / kKeys; ++j)
        *reinterpret_cast<uint4*>(to + j * kKeys * 128 + ((piece ^ ((j * kKeys) & 7)) << 4)) = v_operand(words[32 * j]);
}

// An expander warp's share of every tile, 16 * BLOCKS keys from key0 on: where its
// codes lie (a page holds 16 keys at least), and copies of them on their way into
// the warp's own ring, 32 keys to an entry. RECORD: page numbers out of range go to
// the status word.
template <int D, int BLOCKS, bool RECORD = true>
struct CodeReader {
    static constexpr int kTiles = 32 / BLOCKS;  // of one lookup, a lane per 16 keys
    static constexpr int kEntries = BLOCKS / 2, kDepth = BLOCKS == 2 ? kRawK : kRawV;
    static constexpr int kBytes = 32 * D / 2;
    const PagedSeqs& s;
    const int32_t* table;
    int g, T, n, key0, lane, now, next, batch;
    unsigned char* raw;
    __device__ __forceinline__ CodeReader(const PagedAttend& p, const PagedSeqs& s_, int g_, int seq, int T_, int n_, int key0_,
                                          int lane_, unsigned char* raw_)
        : s(s_), table(s_.table + (long long)seq * s_.tstride), g(g_), T(T_), n(n_), key0(key0_), lane(lane_), raw(raw_) {}
    // index of the vector of the first of the lane's 16 keys, -1 for none, in the m-th kTiles tiles
    template <class F>
    __device__ __forceinline__ int lookup(int m, F tile_at) const {
        const int i = kTiles * m + lane / BLOCKS, t = i < n ? tile_at(i) * kTile + key0 + 16 * (lane % BLOCKS) : T;
        if (t >= T) return -1;
        const int page = __ldg(table + (t >> s.pshift));
        if (page < 0 || page >= s.pages) {
            if (RECORD) pages::flag(s.status, kPgBadPage);
            return -1;
        }
        return ((page * s.Hk + g) << s.pshift) + (t & ((1 << s.pshift) - 1));
    }
    template <class F>
    __device__ __forceinline__ void start(F tile_at) {
        batch = 0, now = lookup(0, tile_at), next = lookup(1, tile_at);
    }
    // tile i is under way: no tile before it is asked for any more
    template <class F>
    __device__ __forceinline__ void next_batch(int i, F tile_at) {
        if (i < kTiles * (batch + 1)) return;
        ++batch;
        now = next, next = lookup(batch + 1, tile_at);
    }
    __device__ __forceinline__ int vector_of(int i, int block) const {
        return __shfl_sync(0xffffffffu, i / kTiles == batch ? now : next, (i % kTiles) * BLOCKS + block);
    }
    __device__ __forceinline__ unsigned char* slot(int i, int c) const {
        return raw + ((i * kEntries + c) % kDepth) * kBytes;
    }
    __device__ __forceinline__ void ask(const uint16_t* codes, int i, int c) const {
        const uint32_t to = ptx::smem_u32(slot(i, c)) + lane * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = vector_of(i, 2 * c + h);
            const unsigned char* src = reinterpret_cast<const unsigned char*>(codes) + (long long)max(at, 0) * (D / 2) + lane * 16;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) cp_async16(to + (h * (D / 64) + j) * 512, src + j * 512, at < 0 ? 0 : 16);
        }
    }
};

// The workspace: room for so many tiles of each sequence and KV head. Sequences
// that fit are the MADE kernel's, others the other one's.
struct Made {
    unsigned char* tiles;
    int room;
    __host__ __device__ bool has(long long tokens) const { return room > 0 && tokens <= (long long)room * kTile; }
};

// KIND: the causal mask alone; other masks too; scores that a cap or a bias by
// distance changes; the same with a cap so wide that each key takes a form of its own.
enum { kPlain, kMasks, kScores, kWideScores };
template <int D, int KIND, bool MADE>
__global__ void __launch_bounds__(Shape<MADE>::threads, 1)
pages4_chunk_kernel(const PagedAttend4 p4, const Made made) {
    using L = Lay<D, MADE>;
    using SH = Shape<MADE>;
    constexpr int kThreads = SH::threads;
    const PagedAttend& p = p4.a;
    constexpr bool SCORED = KIND != kPlain;
    constexpr bool CHANGED = KIND == kScores || KIND == kWideScores;
    constexpr bool kQuad = KIND == kPlain;  // the softmax has four rows to a lane, else a row to a lane
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
    // blocks of a sequence from its last (the one that sees most) to its first
    const int job = blockIdx.x / CS, g = job % s.Hk;
    pages::RowBlock b;
    if (!pages::find_block(s, p.G, kRows, job / s.Hk, b) || made.has(b.T) != MADE) {  // the whole cluster's
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

    // full, empty: of K's stages, V's nst further on
    const uint32_t b_full = ptx::smem_u32(sm + L::bars), b_empty = b_full + 16 * L::nst;
    const uint32_t b_s = ptx::smem_u32(sm + L::bar_s), b_p = ptx::smem_u32(sm + L::bar_p);
    const uint32_t b_o = ptx::smem_u32(sm + L::bar_o), b_fin = ptx::smem_u32(sm + L::bar_fin);
    if (tid == 0) {
        for (int i = 0; i < 2 * L::nst; ++i) {
            ptx::mbar_init(b_full + 8 * i, MADE ? 1 : i < L::nst ? kWarpsK : kWarpsV);
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
    const bool soft = warp >= 4 && warp < 20;
    const int w = (warp - 4) / 8;          // slot
    const int part = ((warp - 4) / 4) & 1; // of a row: 32 keys of every 64, half the channels
    const int lr = tid & 127;              // row of the slot
    const int row = two ? w * kTile + lr : lr;
    const bool live = soft && row < nr;
    Seen see = {0, INT_MAX, 0, 0};  // rows past the block: nothing to mask, dropped at the end
    int tok = 0, head = 0, pos = 0;
    if (live) {
        const int i = pages::div_group(p, j_begin + row);
        tok = b.q0 + i_begin + i;
        head = g * p.G + j_begin + row - i * p.G;
        pos = b.p0 + i_begin + i;
        see = pages::row_seen<SCORED>(p, b.seq, tok, pos, T);
    }
    if constexpr (SCORED) {
        if (soft) {
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
    TileScales* tile_scales = reinterpret_cast<TileScales*>(sm + L::scales);

    if (warp < 4) {
        ptx::regs_dec<SH::regs_issue>();
        if (warp == 1 || warp == 2) {
            // ------------------------------------------------------ issuers
            // One warp per slot; the whole warp runs this with uniform values, an elected lane issues.
            ptx::bar_sync(kBarQ, 64 + kSoftmax);  // Q is in shared memory
            auto uniform = [](auto x) { return __reduce_max_sync(0xffffffffu, x); };
            const int slot = uniform(warp - 1), nn = uniform(n), nt = uniform(tiles_of(slot));
            const bool pairs = __any_sync(0xffffffffu, two);
            const uint32_t tm = uniform(tmem), base = uniform(ptx::smem_u32(sm)), ring = base + L::ring;
            const uint32_t tS = tm + kColS + 128 * slot, tO = tm + kColO + 128 * slot;
            const uint32_t idS = ptx::idesc_f16(kTile, kTile, 0, 0);
            const uint32_t idO = ptx::idesc_bf16(kTile, D, 0, 1);
            const uint32_t u_full = base + L::bars, u_empty = u_full + 16 * L::nst;
            const uint32_t u_s = base + L::bar_s + 8 * slot, u_p = base + L::bar_p + 16 * slot;
            const uint32_t u_o = base + L::bar_o + 8 * slot, u_fin = base + L::bar_fin + 8 * slot;
            const uint64_t dq = ptx::sdesc(base + (pairs ? slot : 0) * L::stage, 16, 1024);
            // an entry: K of tile i is 2 i, its V 2 i + 1; the stage that has it
            auto k_entry = [](int i) { return 2 * i; };
            auto v_entry = [](int i) { return 2 * i + 1; };
            auto stage_of = [](int e) { return (e >> 1) % L::nst + (e & 1) * L::nst; };
            auto full = [&](int e) { warp_wait(u_full + 8 * stage_of(e), ((e >> 1) / L::nst) & 1, bad); };
            auto release = [&](int e) { ptx::mma_commit_elect(u_empty + 8 * stage_of(e)); };
            auto qk = [&](int e) {
                const uint64_t dk = ptx::sdesc(ring + stage_of(e) * L::stage, 16, 1024);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t o = ((ks / 4) * (kTile * 128) + (ks % 4) * 32) >> 4;  // descriptor units
                    ptx::mma_f16_elect(tS, dq + o, dk + o, idS, ks > 0 ? 1u : 0u);
                }
                ptx::mma_commit_elect(u_s);
            };
            auto pv = [&](int e, int it) {
                const uint64_t dv = ptx::sdesc(ring + stage_of(e) * L::stage, kTile * 128, 1024);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h) {
                        warp_wait(u_p + 8, it & 1, bad);
                        ptx::tc_fence_after();
                    }
#pragma unroll
                    for (int ks = 4 * h; ks < 4 * h + 4; ++ks)  // P of 32 keys: 16 columns at S's 32
                        ptx::mma_f16_ta_elect(tO, tS + 32 * (ks / 2) + 8 * (ks % 2), dv + ks * (2048 >> 4), idO,
                                              (it > 0 || ks > 0) ? 1u : 0u);
                    if (CHANGED && h == 0) ptx::mma_commit_elect(u_o);  // (it takes over 100 cycles)
                }
            };
            // The slots take turns: P V and the next Q K^T of one, then of the other, so
            // that one's softmax runs beside the other's MMAs. What a turn needs is waited
            // for before it, what can be done after it is.
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
                if (lane == 0) ptx::mbar_arrive(u_empty + 8 * stage_of(e));
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
                    const int ev = v_entry(i), ek = k_entry(i + 1);
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
                        pass(v_entry(i));
                        if (i + 2 < nn) pass(k_entry(i + 2));
                    }
                    turn(i >> 1, i + slot < nn, v_entry(i + slot), i + 2 + slot < nn, k_entry(i + 2 + slot));
                    if (!slot) {
                        if (i + 1 < nn) pass(v_entry(i + 1));
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
        } else if constexpr (MADE) {
            // ------------------------------------------------------- loaders
            // Warp 0: K and the scales, warp 3: V; a tile in one or two bulk copies. Warp 3 looks at
            // the tile's table entries too, a lane per 16 keys: those out of range are recorded where a
            // tile is read, not where it is made (more tiles are made than rows see). An
            // entry is asked for after a tile's copies and looked at after the next one's.
            const bool v = warp == 3;
            int page = 0;
            auto look = [&] {
                if (page < 0 || page >= s.pages) pages::flag(s.status, kPgBadPage);
            };
            const unsigned char* tiles = made.tiles + ((long long)b.seq * s.Hk + g) * made.room * made_bytes<D>() + (v ? L::stage : 0);
            for (int i = 0; i < n; ++i) {
                const int st = i % L::nst + (v ? L::nst : 0);
                if (i >= L::nst) warp_wait(b_empty + 8 * st, ((i / L::nst) - 1) & 1, bad);
                if (lane == 0) {
                    const unsigned char* src = tiles + (long long)tile_at(i) * made_bytes<D>();
                    ptx::mbar_expect_tx(b_full + 8 * st, L::stage + (v ? 0 : (int)sizeof(TileScales)));
                    ptx::bulk_g2s(ptx::smem_u32(sm + L::ring + st * L::stage), src, L::stage, b_full + 8 * st);
                    if (!v)
                        ptx::bulk_g2s(ptx::smem_u32(tile_scales + i % L::slots), src + 2 * L::stage, sizeof(TileScales), b_full + 8 * st);
                }
                __syncwarp();
                if (v) {
                    look();
                    const int t = tile_at(i) * kTile + 16 * lane;
                    page = lane < kTile / 16 && t < T ? __ldg(s.table + (long long)b.seq * s.tstride + (t >> s.pshift)) : 0;
                }
            }
            look();
            // every requested tile has landed before the CTA may go on
            for (int i = max(0, n - L::nst); i < n; ++i) {
                bool late = false;
                warp_wait(b_full + 8 * (i % L::nst + (v ? L::nst : 0)), (i / L::nst) & 1, late);
            }
        } else {
            // ---------------------------------------------- expanders of V
            const int vw = warp / 3;
            CodeReader<D, 4> in(p, s, g, b.seq, T, n, vw * 64, lane,
                                sm + L::raw + (kWarpsK * kRawK + vw * kRawV) * L::codes);
            auto tile_of = [&](int i) { return tile_at(i); };
            in.start(tile_of);
            if (n > 0) in.ask(p.V, 0, 0);
            cp_commit();
            if (n > 0) in.ask(p.V, 0, 1);
            cp_commit();
            for (int i = 0; i < n; ++i) {
                const int st = i % L::nst;
                unsigned char* stage = sm + L::ring + (L::nst + st) * L::stage;
                if (i >= L::nst) warp_wait(b_empty + 8 * (L::nst + st), ((i / L::nst) - 1) & 1, bad);
                in.next_batch(i, tile_of);
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // 32 keys
                    if (i + 1 < n) in.ask(p.V, i + 1, c);
                    cp_commit();
                    cp_wait<2>();
                    __syncwarp();
                    expand_v<D>(in.slot(i, c), stage, vw * 64 + 32 * c);
                    __syncwarp();  // (the codes are read)
                }
                ptx::fence_proxy_async();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_full + 8 * (L::nst + st));
            }
            cp_wait<0>();
        }
        if (bad && lane == 0) pages::flag(s.status, kPgTimeout);
        if (!direct) {
            ptx::bar_sync(kBarDone, kThreads);
            ptx::bar_sync(kBarRows, kThreads);
        }
    } else if (!MADE && warp >= 20) {
        ptx::regs_dec<SH::regs_expand>();
        // -------------------------------------------------- expanders of K
        const int key0 = (warp - 20) * 32;
        CodeReader<D, 2> in(p, s, g, b.seq, T, n, key0, lane, sm + L::raw + (warp - 20) * (kRawK * L::codes));
        auto tile_of = [&](int i) { return tile_at(i); };
        in.start(tile_of);
        float tk = 0.0f, tv = 0.0f;
        auto ask_scales = [&](int i) {  // lane: key key0 + lane
            const int at = in.vector_of(i, lane >> 4);
            const bool held = at >= 0 && i < n && tile_at(i) * kTile + key0 + lane < T;
            tk = held ? __ldg(p4.Kt + at + (lane & 15)) : 0.0f;
            tv = held ? __ldg(p4.Vt + at + (lane & 15)) : 0.0f;
        };
        uint32_t h16[2][2];
        h16_operands(h16);
        const uint32_t half_sum = (lane & 3) == 0 ? (D == 128 ? 0x5400u : 0x5000u) : 0u;  // D / 2 to channel 0
        ask_scales(0);
        in.ask(p.K, 0, 0);
        cp_commit();
        for (int i = 0; i < n; ++i) {
            if (i + 1 < n) in.ask(p.K, i + 1, 0);
            cp_commit();
            cp_wait<1>();
            __syncwarp();
            const int st = i % L::nst;
            unsigned char* stage = sm + L::ring + st * L::stage;
            if (i >= L::nst) warp_wait(b_empty + 8 * st, ((i / L::nst) - 1) & 1, bad);
            TileScales& ts = tile_scales[i % L::slots];
            ts.set(key0 + lane, tk, tv);
            in.next_batch(i, tile_of);
            ask_scales(i + 1);
            expand_k<D>(in.slot(i, 0), stage, key0, h16, half_sum);
            ptx::fence_proxy_async();
            __syncwarp();  // (and the codes are read)
            if (lane == 0) ptx::mbar_arrive(b_full + 8 * st);
        }
        cp_wait<0>();
        if (bad && lane == 0) pages::flag(s.status, kPgTimeout);
        if (!direct) {
            ptx::bar_sync(kBarDone, kThreads);
            ptx::bar_sync(kBarRows, kThreads);
        }
    } else {
        ptx::regs_inc<SH::regs_many>();
        float m = -CUDART_INF_F, l = 0.0f;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        // ------------------------------------------------------------ softmax
        // the rows, a warp each, in fp16 times a power of two (rows past the block repeat its last)
        float* rowf = reinterpret_cast<float*>(sm + L::pair);
        {
            // (all of a warp's rows are asked for before the first is looked at: 4 at a time took 6 us of a CTA's start)
            constexpr int kEach = kRows / (kSoftmax / 32);
            const int nq = two ? kRows : kTile;
            uint2 v[kEach];
#pragma unroll
            for (int u = 0; u < kEach; ++u) {
                const int rr = min(warp - 4 + u * (kSoftmax / 32), nr - 1), i = pages::div_group(p, j_begin + rr);
                const uint16_t* src = p.Q + (long long)(b.q0 + i_begin + i) * p.q_stride +
                                      (long long)(g * p.G + j_begin + rr - i * p.G) * D;
                v[u] = make_uint2(0u, 0u);
                if (lane < D / 4 && (two || u < kEach / 2)) v[u] = __ldg(reinterpret_cast<const uint2*>(src) + lane);
            }
#pragma unroll
            for (int u = 0; u < kEach; ++u) {
                const int r = warp - 4 + u * (kSoftmax / 32);
                if (r >= nq) break;
                const float4 x = make_float4(asf(v[u].x << 16), asf(v[u].x & 0xFFFF0000u), asf(v[u].y << 16), asf(v[u].y & 0xFFFF0000u));
                const uint32_t top = __reduce_max_sync(
                    0xffffffffu, max(max(asu(fabsf(x.x)), asu(fabsf(x.y))), max(asu(fabsf(x.z)), asu(fabsf(x.w)))));
                const int e = min(max((int)(top >> 23) - 126, -122), 126);
                const float up = asf((uint32_t)(127 + 4 - e) << 23);
                const __half2 a = __floats2half2_rn(x.x * up, x.y * up), c = __floats2half2_rn(x.z * up, x.w * up);
                if (lane < D / 4) {
                    const int q = r & 127, ch = lane * 4;
                    *reinterpret_cast<uint2*>(sm + (r >> 7) * L::stage + (ch / 64) * (kTile * 128) + q * 128 +
                                              ((((ch % 64) / 8) ^ (q & 7)) << 4) + (ch & 4) * 2) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
                }
                if (lane == 0) rowf[r] = asf((uint32_t)(127 - 4 + e) << 23);
            }
            ptx::fence_proxy_async();  // the MMAs read Q through the async proxy
        }
        ptx::bar_sync(kBarQ, 64 + kSoftmax);
        const int mine = tiles_of(w);
        const bool some = __any_sync(0xffffffffu, live);
        const float slope2 = SCORED && live && p.slopes ? __ldg(p.slopes + head) * 1.4426950408889634f : 0.0f;
        const float mul = rowf[two ? w * kTile + lr : lr] * (CHANGED ? 1.0f : p.scale_log2);
        float mul4[4];  // kQuad: of rows quad + 8 a of the warp's 32
        if constexpr (kQuad)
#pragma unroll
            for (int a = 0; a < 4; ++a)
                mul4[a] = rowf[(two ? w * kTile : 0) + (warp & 3) * 32 + (lane >> 2) + 8 * a] * p.scale_log2;
        ptx::bar_sync(kBarRead, kSoftmax);  // (its place is used for other things from here on)
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
        // scores of 32 keys times their scales t, the first of which have been asked for
        auto times = [&](const float4 (&early)[kEarly], const float* t, uint32_t (&u)[32]) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                const float4 f = k / 4 < kEarly ? early[k / 4 < kEarly ? k / 4 : 0] : *reinterpret_cast<const float4*>(t + k);
                const float2 x = __fmul2_rn(make_float2(asf(u[k]), asf(u[k + 1])), make_float2(f.x, f.y));
                const float2 y = __fmul2_rn(make_float2(asf(u[k + 2]), asf(u[k + 3])), make_float2(f.z, f.w));
                u[k] = asu(x.x), u[k + 1] = asu(x.y), u[k + 2] = asu(y.x), u[k + 3] = asu(y.y);
            }
        };
        // (while the scores are on their way from tensor memory: what a tile's scales cost
        // is the loads' place in the path from S to P)
        auto ask_early = [&](float4 (&early)[kEarly], const float* t) {
#pragma unroll
            for (int k = 0; k < kEarly; ++k)
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(early[k].x), "=f"(early[k].y), "=f"(early[k].z), "=f"(early[k].w)
                             : "r"(ptx::smem_u32(t + 4 * k)));
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
        if constexpr (kQuad) {
            // A lane has keys 8 j + 2 qi and the next of 32 in four rows, quad + 8 a of the
            // warp's 32 (the layout of 16 rows x 256 bits): a scale then serves four scores,
            // not one, and what the loads of scales give each lane is a quarter (2,048
            // tokens over 16K keys: 466 us, 538 with a row to a lane).
            const int quad = lane >> 2, qi = lane & 3;
            constexpr uint32_t k16 = 16u << 16;  // 16 rows on, in tensor memory
            float qm[4], ql[4], top4[4];
            int end4[4];
            const int row0 = (two ? w * kTile : 0) + (warp & 3) * 32 + quad;
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                qm[a] = top4[a] = -CUDART_INF_F, ql[a] = 0.0f;
                const int i = pages::div_group(p, j_begin + row0 + 8 * a);
                end4[a] = row0 + 8 * a < nr ? min(b.p0 + i_begin + i + 1, T) : INT_MAX;
            }
            const int all_see = __reduce_min_sync(0xffffffffu, min(min(end4[0], end4[1]), min(end4[2], end4[3])));
            // scores (without the rows' factors) of the 32 keys at `in` of the tile, which are keys k0 and on
            auto load4 = [&](const TileScales& ts, int in, int k0, float2 (&x)[4][4], float2 (&tv)[4]) {  // [row][keys]; V's scales
                uint32_t u[32];
                ptx::tmem_ld_16x256(tS + in, u);
                ptx::tmem_ld_16x256(tS + in + k16, u + 16);
                float2 t[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // (while S is on its way)
                    const uint32_t at = ptx::smem_u32(ts.k + in + 8 * j + 2 * qi), at_v = ptx::smem_u32(ts.v + in + 8 * j + 2 * qi);
                    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(t[j].x), "=f"(t[j].y) : "r"(at));
                    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(tv[j].x), "=f"(tv[j].y) : "r"(at_v));
                }
                ptx::tmem_wait_ld(u);
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int e = 16 * (a >> 1) + 4 * j + 2 * (a & 1);
                        x[a][j] = __fmul2_rn(make_float2(asf(u[e]), asf(u[e + 1])), t[j]);
                    }
                if (k0 + 32 > all_see) {
#pragma unroll
                    for (int a = 0; a < 4; ++a)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int key = k0 + 8 * j + 2 * qi;
                            if (key >= end4[a]) x[a][j].x = -CUDART_INF_F;
                            if (key + 1 >= end4[a]) x[a][j].y = -CUDART_INF_F;
                        }
                }
            };
            auto max8 = [](const float2 (&x)[4]) {
                return ptx::max3(ptx::max3(x[0].x, x[0].y, x[1].x), ptx::max3(x[1].y, x[2].x, x[2].y), fmaxf(x[3].x, x[3].y));
            };
            auto over_lanes = [](float v) {  // the largest of a row's four lanes
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            };
            // of this lane's row in the layout of a row per lane
            auto per_row = [&](const float (&v)[4]) {
                float r = 0.0f;
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const float y = __shfl_sync(0xffffffffu, v[a], (lane & 7) * 4);
                    if (lane >> 3 == a) r = y;
                }
                return r;
            };
            // The references become the maxima of both parts where these have passed them; O follows.
            auto move4 = [&] {
                float* x = reinterpret_cast<float*>(sm + L::pair) + w * kTile + (warp & 3) * 32;
                float al[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    top4[a] = over_lanes(top4[a]);
                    if (!part && qi == 0) x[quad + 8 * a] = top4[a];
                }
                ptx::bar_sync(b_pair, 64);
                if (part) {
#pragma unroll
                    for (int a = 0; a < 4; ++a) top4[a] = fmaxf(top4[a], x[quad + 8 * a]);
                    __syncwarp();
                    if (qi == 0)
#pragma unroll
                        for (int a = 0; a < 4; ++a) x[quad + 8 * a] = top4[a];
                }
                ptx::bar_sync(b_pair, 64);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const float mt = part ? top4[a] : x[quad + 8 * a];
                    const bool move = mt > qm[a] + kLazy || (qm[a] == -CUDART_INF_F && mt > qm[a]);
                    // (in two steps: a maximum may have passed the reference by up to 2^128, and ex2 gives 0 below 2^-126)
                    al[a] = move && qm[a] != -CUDART_INF_F ? ptx::ex2(0.5f * (qm[a] - mt)) : 1.0f;
                    ql[a] = ql[a] * al[a] * al[a];
                    if (move) qm[a] = mt;
                }
                const float of = per_row(al);
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 32) {
                    uint32_t o[32];
                    ptx::tmem_ld32(tO + part * (D / 2) + c, o);
                    ptx::tmem_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = asu(asf(o[k]) * of * of);
                    ptx::tmem_st32x(tO + part * (D / 2) + c, o);
                }
                ptx::tmem_wait_st();
            };
            if (mine > 0 && some) {
                // The first reference is the maximum of the first half tile, which both parts look at.
                const int i0 = two ? 0 : w, t0 = (ta + i0) * kTile;  // (plain scores: no gap)
                warp_wait(b_s + 8 * w, 0, bad);
                ptx::tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 64; c += 32) {
                    float2 x[4][4], none[4];
                    load4(tile_scales[i0 % L::slots], c, t0 + c, x, none);
#pragma unroll
                    for (int a = 0; a < 4; ++a) qm[a] = fmaxf(qm[a], max8(x[a]) * mul4[a]);
                }
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    qm[a] = over_lanes(qm[a]);
                    // products of minus infinity alone are no reference: such a row is done again
                    if (row0 + 8 * a < nr && qm[a] == -CUDART_INF_F && end4[a] > t0) ql[a] = CUDART_NAN_F;
                }
                ptx::bar_sync(b_pair, 64);  // P of either part overwrites what both have read
            }
            for (int it = 0; it < mine; ++it) {
                const int i = two ? it : 2 * it + w;  // tile of this CTA
                const int t0 = tile_at(i) * kTile;
                const TileScales& ts = tile_scales[i % L::slots];
                // A maximum that passes the reference by 2^8 moves it before the next tile
                // (until then the weights are that much larger, which float32 has room for up to
                // 2^128; rows beyond it come out infinite and are done again).
                const bool far = top4[0] > qm[0] + kLazy || top4[1] > qm[1] + kLazy || top4[2] > qm[2] + kLazy || top4[3] > qm[3] + kLazy;
                const bool moves = it > 0 && some && ptx::bar_or(b_pair, 64, far);
                warp_wait(b_s + 8 * w, it & 1, bad);
                ptx::tc_fence_after();
                if (!some) {  // no row of this warp: only the barriers' counts
                    __syncwarp();
                    if (lane < 2) ptx::mbar_arrive(b_p + 16 * w + 8 * lane);
                    continue;
                }
                // (S came after every P V before it: O rests)
                if (moves) move4();
#pragma unroll
                for (int a = 0; a < 4; ++a) top4[a] = -CUDART_INF_F;
                // The tile's keys in two halves, so that P V of the first runs while P of the second is formed.
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int in = 64 * h + 32 * part;
                    float2 x[4][4], t[4];
                    load4(ts, in, t0 + in, x, t);
                    uint32_t pw[2][8];  // rows quad + 16 hh and + 8
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        top4[a] = fmaxf(top4[a], max8(x[a]) * mul4[a]);
                        const float ref = qm[a] == -CUDART_INF_F ? 0.0f : qm[a];
                        const float2 sc = make_float2(mul4[a], mul4[a]), nm = make_float2(-ref, -ref);
                        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 d = __ffma2_rn(x[a][j], sc, nm);
                            const float2 e = make_float2(ptx::ex2(d.x), ptx::ex2(d.y)), y = __fmul2_rn(e, t[j]);
                            sum = __fadd2_rn(sum, e);
                            pw[a >> 1][2 * j + (a & 1)] = pack_bf2(y.x, y.y);
                        }
                        ql[a] += sum.x + sum.y;
                    }
                    // P over the part's own columns of S
                    ptx::tmem_st_16x128(tS + in, pw[0]);
                    ptx::tmem_st_16x128(tS + in + k16, pw[1]);
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(b_p + 16 * w + 8 * h);
                }
            }
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                ql[a] += __shfl_xor_sync(0xffffffffu, ql[a], 1);
                ql[a] += __shfl_xor_sync(0xffffffffu, ql[a], 2);
            }
            l = per_row(ql);
            m = per_row(qm);
        } else {
        float top = -CUDART_INF_F;  // the part's maximum in the tile before
        constexpr bool kLeft = !CHANGED;  // the row's factor is left for the exponent
        const float f = kLeft ? mul : 1.0f;
        // the scores of the part's 32 keys from k0 on, -inf where the row sees none
        auto scores_of = [&](const float4 (&early)[kEarly], const float* t, int k0, bool whole, uint32_t (&u)[32]) {
            times(early, t, u);
            if constexpr (CHANGED) {
#pragma unroll
                for (int k = 0; k < 32; ++k) u[k] = asu(asf(u[k]) * mul);
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
            const TileScales& ts = tile_scales[i % L::slots];
            // A maximum that passes the reference by 2^8 moves it: where scores cost much
            // to form or may rise fast (CHANGED) at once, else before the next tile (until
            // then the weights are that much larger, which float32 has room for up to 2^128;
            // rows beyond it come out infinite and are done again). The two threads of a row
            // ask one another while S is on its way.
            const bool moves = !CHANGED && it > 0 && some && ptx::bar_or(b_pair, 64, top > m + kLazy);
            warp_wait(b_s + 8 * w, it & 1, bad);
            ptx::tc_fence_after();
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
                for (int c = 32 * part; c < kTile; c += 64) {
                    uint32_t u[32];
                    float4 early[kEarly];
                    ptx::tmem_ld32(tS + c, u);
                    ask_early(early, ts.k + c);
                    ptx::tmem_wait_ld(u);
                    scores_of(early, ts.k + c, t0 + c, false, u);
                    top = fmaxf(top, max_of(u) * f);
                }
                if (ptx::bar_or(b_pair, 64, top > m + kLazy || (m == -CUDART_INF_F && top > m))) move_ref(top, it > 0);
            }
            // The tile's keys in two halves, so that P V of the first runs while P of
            // the second is formed; a thread has 32 keys of each.
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int half = t0 + 64 * h, in = 64 * h + 32 * part, k0 = t0 + in;
                const uint32_t tSh = tS + in;
                const bool whole = __all_sync(0xffffffffu, see.all(k0, k0 + 32));
                // nothing seen by either part (beyond the diagonal, other documents): weights
                // of 0 whatever S holds
                const bool any = __any_sync(0xffffffffu, live && see.some(half, half + 64));
                uint32_t pw[16];
                float2 sum[2] = {};
                if (any) {
                    uint32_t u[32];
                    float4 early[kEarly];
                    ptx::tmem_ld32(tSh, u);
                    ask_early(early, ts.k + in);
                    ptx::tmem_wait_ld(u);
                    scores_of(early, ts.k + in, k0, whole, u);
                    const float x = max_of(u) * f;
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
                    const float2 sc = make_float2(f, f), nm = make_float2(-ref, -ref);
                    auto weights = [&](int k) {  // of keys 2 k and 2 k + 1
                        const float2 d = __ffma2_rn(make_float2(asf(u[2 * k]), asf(u[2 * k + 1])), sc, nm);
                        const float2 e = make_float2(ptx::ex2(d.x), ptx::ex2(d.y));
                        sum[k & 1] = __fadd2_rn(sum[k & 1], e);
                        return e;
                    };
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const float4 t = *reinterpret_cast<const float4*>(&ts.v[in + 2 * k]);
                        const float2 a = __fmul2_rn(weights(k), make_float2(t.x, t.y));
                        const float2 c = __fmul2_rn(weights(k + 1), make_float2(t.z, t.w));
                        pw[k] = pack_bf2(a.x, a.y), pw[k + 1] = pack_bf2(c.x, c.y);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) pw[k] = 0u;
                }
                // P over the part's own columns of S
                ptx::tmem_st16(tSh, pw);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_p + 16 * w + 8 * h);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
        }
        }
        if (mine > 0) {
            warp_wait(b_fin + 8 * w, 0, bad);  // every MMA of the slot
            ptx::tc_fence_after();
        }
        if (bad && lane == 0) pages::flag(s.status, kPgTimeout);
        __syncwarp();

        // careful_row4 of this warp's row `of` (a lane), over the slot's tiles or all of the CTA's
        auto careful = [&](int of, bool all, float& cm, float& cl, float (&acc)[D / 32]) {
            Seen se;
            se.a1 = __shfl_sync(0xffffffffu, see.a1, of);
            se.b1 = __shfl_sync(0xffffffffu, see.b1, of);
            se.a2 = __shfl_sync(0xffffffffu, see.a2, of);
            se.b2 = __shfl_sync(0xffffffffu, see.b2, of);
            pages::careful_row4<D, SCORED>(p4, b.seq, __shfl_sync(0xffffffffu, tok, of),
                                           __shfl_sync(0xffffffffu, head, of), __shfl_sync(0xffffffffu, pos, of), se,
                                           gap, 7, two || all ? ta : ta + (CHANGED ? (n - 1 - w) & 1 : w), ta + n,
                                           two || all ? 1 : 2, cm, cl, acc);
        };
        l = joined(l, true);
        bool again = live && l != 0.0f && !finite(l);  // sums that are not finite: done again key by key
        uint32_t* flags = reinterpret_cast<uint32_t*>(sm + L::pair + 2 * kTile * 4) + 4 * w + (warp & 3);
        // A state that another is merged with has its l within 2^-32 ... 2^64 of its m:
        // a last tile's maxima may lie far above the reference, up to where the other
        // state's weight of it (ex2 of the references' difference, 0 below 2^-126) would
        // lose the larger part of a row.
        const bool high = l > 0x1p32f;
        const float down = high ? 0x1p-64f : 1.0f;
        const float state_m =
            l == 0.0f ? -CUDART_INF_F : (m == -CUDART_INF_F ? 0.0f : m) + (high ? 64.0f : 0.0f);
        auto finish = [&](int t, int hd, float rm, float rl) {
            if (p.lse) p.lse[(long long)t * p.Hq + hd] = rl == 0.0f ? -CUDART_INF_F : (rm + log2f(rl)) * kLn2;
        };
        // a row's channels of this thread
        constexpr int HC = D / 2;
        const int c0 = part * HC;
        if (direct) {
            // Both threads of a row read all of its O: the transform's stage over channels D / 2
            // apart leaves part 0 the sums and part 1 the differences, the other stages stay in
            // registers. The slot's Q (no MMA reads it any more) takes the rows in bf16, pieces of
            // 8 channels exchanged by the row's number, and the two warps write them in whole
            // lines. (Over lanes, four channels to each, the transform took 6 us.)
            const float inv = 1.0f / l, sign = part ? -1.0f : 1.0f;  // (inv: not used where l is 0)
            unsigned char* stage = sm + w * L::stage + (warp & 3) * 32 * (D * 2);
            constexpr int C8 = D / 8, kPer = 32 / C8;  // pieces of a row, rows of a warp at a time
            if (live && !part) finish(tok, head, state_m, l * down);
            const long long at = live ? ((long long)tok * p.Hq + head) * D : -1;
            float2 y[HC / 2];
#pragma unroll
            for (int c = 0; c < HC; c += 16) {
                uint32_t u[32];  // 16 channels, and those D / 2 on
                ptx::tmem_ld16(tO + c, *reinterpret_cast<uint32_t(*)[16]>(u));
                ptx::tmem_ld16(tO + HC + c, *reinterpret_cast<uint32_t(*)[16]>(u + 16));
                ptx::tmem_wait_ld(u);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float a = fmaf(sign, asf(u[16 + 2 * k]), asf(u[2 * k])) * inv;
                    const float d = fmaf(sign, asf(u[17 + 2 * k]), asf(u[2 * k + 1])) * inv;
                    y[c / 2 + k] = make_float2(a + d, a - d);
                }
            }
#pragma unroll
            for (int h = 1; h < HC / 2; h <<= 1)
#pragma unroll
                for (int i = 0; i < HC / 2; ++i)
                    if (!(i & h)) {
                        const float2 a = y[i], d = y[i + h];
                        y[i] = __fadd2_rn(a, d);
                        y[i + h] = __ffma2_rn(d, make_float2(-1.0f, -1.0f), a);
                    }
            // (an infinity or NaN in O is in the row's every output)
            again = again || (live && l != 0.0f && !finite(y[0].x));
#pragma unroll
            for (int k = 0; k < HC / 8; ++k) {
                uint4 v = make_uint4(pack_bf2(y[4 * k].x, y[4 * k].y), pack_bf2(y[4 * k + 1].x, y[4 * k + 1].y),
                                     pack_bf2(y[4 * k + 2].x, y[4 * k + 2].y), pack_bf2(y[4 * k + 3].x, y[4 * k + 3].y));
                if (l == 0.0f) v = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(stage + lane * (D * 2) + (((part * (HC / 8) + k) ^ (lane & (C8 - 1))) << 4)) = v;
            }
            ptx::bar_sync(b_pair, 64);
#pragma unroll 4
            for (int k = 0; k < 16 / kPer; ++k) {
                const int r = 16 * part + kPer * k + lane / C8, c8 = lane % C8;  // of the 32
                const uint4 v = *reinterpret_cast<const uint4*>(stage + r * (D * 2) + ((c8 ^ (r & (C8 - 1))) << 4));
                const long long row_at = __shfl_sync(0xffffffffu, at, r);
                if (row_at >= 0) *reinterpret_cast<uint4*>(p.out + row_at + c8 * 8) = v;
            }
            const unsigned odds = __ballot_sync(0xffffffffu, again);
            if (part && lane == 0) *flags = odds;
            ptx::bar_sync(b_pair, 64);
            if (!part) {  // (writes odd rows once more)
                for (unsigned left = odds | *flags; left; left &= left - 1) {
                    const int of = __ffs(left) - 1;
                    float cm, cl, acc[D / 32];
                    careful(of, true, cm, cl, acc);
                    pages::transform_row<D>(acc);
                    const int ct = __shfl_sync(0xffffffffu, tok, of), ch = __shfl_sync(0xffffffffu, head, of);
                    const long long to = ((long long)ct * p.Hq + ch) * D + lane * (D / 32);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e)
                        p.out[to + e] = cl == 0.0f ? (uint16_t)0 : __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] / cl));
                    if (lane == 0) finish(ct, ch, cm, cl);
                }
            }
        } else {
            // states into shared memory, once no MMA reads the tiles any more and
            // every tile has been written
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
                    again = again || (live && l != 0.0f && !(finite(v.x) && finite(v.y) && finite(v.z) && finite(v.w)));
                    *reinterpret_cast<float4*>(dst + c + k) =
                        make_float4(v.x * down, v.y * down, v.z * down, v.w * down);
                }
            }
            if (!part) {
                dst[D] = state_m;
                dst[D + 1] = l * down;
            }
            const unsigned mine_odd = __ballot_sync(0xffffffffu, again);
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
        // loads all under way before the first is used, and the transform.
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
            const float inv = Lt == 0.0f ? 0.0f : 1.0f / Lt;
#pragma unroll
            for (int k = 0; k < kMaxParts; ++k)
                if (k < parts) weights[r * parts + k] = ml[k].y == 0.0f ? -1.0f : ml[k].x * inv;
            const int2 at = out_at(r);
            if (p.lse) p.lse[(long long)at.x * p.Hq + at.y] = Lt == 0.0f ? -CUDART_INF_F : (M + log2f(Lt)) * kLn2;
        }
        __syncthreads();
        constexpr int C4 = D / 4;
        for (int x0 = 0; x0 < cnt * C4; x0 += kThreads) {  // whole warps: the transform crosses lanes
            const int x = x0 + tid, r = min(x / C4, cnt - 1), c4 = x % C4;
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
            pages::transform4<D>(a);
            if (x < cnt * C4) {
                const int2 ot = out_at(r);
                *reinterpret_cast<uint2*>(p.out + ((long long)ot.x * p.Hq + ot.y) * D + c4 * 4) =
                    make_uint2(pack_bf2(a.x, a.y), pack_bf2(a.z, a.w));
            }
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
template <int D, int KIND, bool MADE>
const Fit& fit(int device) {
    static std::once_flag once[kPagedDevices];
    static Fit fits[kPagedDevices];
    std::call_once(once[device], [device] {
        auto kern = pages4_chunk_kernel<D, KIND, MADE>;
        Fit& x = fits[device];
        x.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (Lay<D, MADE>::total));
        for (int i = 0; i < 4 && x.err == cudaSuccess; ++i) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1 << i, 1, 1);
            cfg.blockDim = dim3(Shape<MADE>::threads, 1, 1);
            cfg.dynamicSmemBytes = (Lay<D, MADE>::total);
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

template <int D, int KIND, bool MADE>
cudaError_t launch(const PagedAttend4& p4, const Made& made, int max_q, int max_kv, cudaStream_t st) {
    const PagedAttend& a = p4.a;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device >= kPagedDevices) return cudaErrorInvalidDevice;
    const Fit& f = fit<D, KIND, MADE>(device);
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
        // the time of the GPU's slots in key tiles: waves x (tiles of a CTA, and about
        // seven for its start and end, twelve with a merge over the cluster)
        const long long tiles = (ntiles + S - 1) / S;
        const long long cost =
            (std::max(1LL, jobs) + f.clusters[i] - 1) / f.clusters[i] * ((one ? (tiles + 1) / 2 : tiles) + (S > 1 ? 12 : 7));
        if (best < 0 || cost < best) best = cost, split = S;
    }
    if (split * blocks * a.s.Hk > INT_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(split * blocks * a.s.Hk), 1, 1);
    cfg.blockDim = dim3(Shape<MADE>::threads, 1, 1);
    cfg.dynamicSmemBytes = (Lay<D, MADE>::total);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pages4_chunk_kernel<D, KIND, MADE>, p4, made);
}

// Tiles of the workspace: K expanded, V expanded, the scales, as the kernel takes
// them. A CTA per tile's K with the scales, or V, of a sequence and KV head, four
// warps of 32 keys, through shared memory and out in bulk. Memory bound, 650 bytes per
// key and head of 128, 512 of them written: 4,096 keys of 8 heads of 19 sequences in 62
// us, 6.6 TB/s (88 with K and V made by one CTA, two of which an SM has room for).
constexpr int kMakeThreads = 128;
constexpr int kMadeSeqs = 65535;  // a grid's third extent: more sequences go without a workspace
template <int D>
__global__ void __launch_bounds__(kMakeThreads)
pages4_make_kernel(const PagedAttend4 p4, const Made made) {
    constexpr int kStage = kTile * D * 2, kCodes = 32 * D / 2;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const PagedAttend& p = p4.a;
    const PagedSeqs& s = p.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, key0 = warp * 32;
    const int seq = blockIdx.z, g = blockIdx.y, tile = blockIdx.x / 2;
    const bool values = blockIdx.x & 1;
    const int len = pages::length_of(s, seq), T = pages::held_tokens(s, len);
    if (pages::row_begin(s, seq + 1) <= pages::row_begin(s, seq)) return;  // no rows, nobody reads it
    if (!made.has(T) || tile * kTile >= T) return;
    CodeReader<D, 2, false> in(p, s, g, seq, T, 1, key0, lane, sm + kStage + sizeof(TileScales) + warp * kCodes);
    in.start([&](int) { return tile; });
    in.ask(values ? p.V : p.K, 0, 0);
    cp_commit();
    if (values) {
        cp_wait<0>();
        __syncwarp();
        expand_v<D>(in.raw, sm, key0);
    } else {
        const int at = in.vector_of(0, lane >> 4);
        const bool held = at >= 0 && tile * kTile + key0 + lane < T;
        const float tk = held ? __ldg(p4.Kt + at + (lane & 15)) : 0.0f, tv = held ? __ldg(p4.Vt + at + (lane & 15)) : 0.0f;
        reinterpret_cast<TileScales*>(sm + kStage)->set(key0 + lane, tk, tv);
        uint32_t h16[2][2];
        h16_operands(h16);
        cp_wait<0>();
        __syncwarp();
        expand_k<D>(in.raw, sm, key0, h16, (lane & 3) == 0 ? (D == 128 ? 0x5400u : 0x5000u) : 0u);
    }
    ptx::fence_proxy_async();
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned char* dst = made.tiles + (((long long)seq * s.Hk + g) * made.room + tile) * made_bytes<D>();
        auto copy = [](unsigned char* to, const unsigned char* from, int bytes) {
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(ptx::smem_u32(from)),
                         "r"(bytes) : "memory");
        };
        copy(dst + (values ? kStage : 0), sm, kStage);
        if (!values) copy(dst + 2 * kStage, sm + kStage, (int)sizeof(TileScales));
        ptx::bulk_commit();
        ptx::bulk_wait_read();  // (shared memory stays until it has been read)
    }
}

template <int D>
cudaError_t launch_make(const PagedAttend4& p4, const Made& made, cudaStream_t st) {
    constexpr int smem = kTile * D * 2 + (int)sizeof(TileScales) + 4 * (32 * D / 2) + 128;
    static std::once_flag once[kPagedDevices];
    static cudaError_t opt[kPagedDevices];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device >= kPagedDevices) return cudaErrorInvalidDevice;
    std::call_once(once[device], [&] {
        opt[device] = cudaFuncSetAttribute(pages4_make_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (opt[device] != cudaSuccess) return opt[device];
    pages4_make_kernel<D><<<dim3(2 * made.room, p4.a.s.Hk, p4.a.s.seqs), kMakeThreads, smem, st>>>(p4, made);
    return cudaGetLastError();
}

template <int D, int KIND>
cudaError_t launch_kind(const PagedAttend4& p4, const Made& made, int max_q, int max_kv, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (made.room > 0) {
        e = launch_make<D>(p4, made, st);
        if (e == cudaSuccess) e = launch<D, KIND, true>(p4, made, max_q, max_kv, st);
        // no sequence can be longer than the workspace's room: the other kernel has nothing to do
        if (made.has((long long)p4.a.s.tstride << p4.a.s.pshift)) return e;
    }
    return e == cudaSuccess ? launch<D, KIND, false>(p4, made, max_q, max_kv, st) : e;
}

}  // namespace

// Bytes of a workspace with room for max_kv tokens of every sequence.
long long pages4_chunk_ws_bytes(const PagedSeqs& s, int head_dim, int max_kv) {
    if (s.seqs > kMadeSeqs) return 0;
    const long long tiles = (max_kv + kTile - 1) / kTile * (long long)s.Hk * s.seqs;
    return tiles * (head_dim == 64 ? made_bytes<64>() : made_bytes<128>());
}

cudaError_t launch_pages4_chunk(const PagedAttend4& p4, int head_dim, int max_q, int max_kv, void* ws, size_t ws_bytes,
                                cudaStream_t st) {
    const PagedAttend& a = p4.a;
    const int kind = a.cap2 > pages::kWideCap2        ? kWideScores
                     : a.cap2 > 0.0f || a.slopes ? kScores
                     : paged_scored(a)           ? kMasks
                                                 : kPlain;
    // room for no more tiles than max_kv has: longer sequences are the kernel's that makes its tiles itself
    Made made{static_cast<unsigned char*>(ws), 0};
    if (ws) {
        const long long each = (long long)a.s.seqs * a.s.Hk * (head_dim == 64 ? made_bytes<64>() : made_bytes<128>());
        made.room = (int)std::min<long long>((long long)ws_bytes / each, (max_kv + kTile - 1) / kTile);
        if (a.s.seqs > kMadeSeqs) made.room = 0;
    }
#define KVP_PG4_CHUNK(KK) \
    (head_dim == 64 ? launch_kind<64, KK>(p4, made, max_q, max_kv, st) : launch_kind<128, KK>(p4, made, max_q, max_kv, st))
    if (kind == kWideScores) return KVP_PG4_CHUNK(kWideScores);
    if (kind == kScores) return KVP_PG4_CHUNK(kScores);
    return kind == kMasks ? KVP_PG4_CHUNK(kMasks) : KVP_PG4_CHUNK(kPlain);
#undef KVP_PG4_CHUNK
}

}  // namespace kvp
