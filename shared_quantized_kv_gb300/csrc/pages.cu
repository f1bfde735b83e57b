// Paged private caches: writing new tokens into their pages, copying pages,
// and the host side of the paged attention.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <new>
#include <vector>

#include "pages4.cuh"

namespace kvp {
namespace {

using pages::flag;

// ------------------------------------------------------------------- append
// One warp per new token: its K and its V row (kv_heads * D values each) are
// read as 16-byte pieces, all requested before the lookups that say where they
// go have come back, and written to the token's slot. Memory bound: every byte
// is read once and written once.
constexpr int kAppWarps = 4;
constexpr int kAppPieces = 4;  // pieces of K and of V in flight per lane

__global__ void __launch_bounds__(kAppWarps * 32)
pages_append_kernel(const PagedSeqs s, uint4* __restrict__ Kp, uint4* __restrict__ Vp,
                    const uint4* __restrict__ K, long long k_stride, const uint4* __restrict__ V,
                    long long v_stride, int chshift) {
    const int tok = blockIdx.x * kAppWarps + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (tok >= s.tokens) return;
    const int pieces = s.Hk << chshift;  // 16-byte pieces of a row, D / 8 = 1 << chshift per head
    const uint4* ks = K + (long long)tok * k_stride;
    const uint4* vs = V + (long long)tok * v_stride;
    uint4 kv[kAppPieces], vv[kAppPieces];
#pragma unroll
    for (int u = 0; u < kAppPieces; ++u) {
        const int i = lane + 32 * u;
        if (i < pieces) kv[u] = ks[i], vv[u] = vs[i];
    }
    pages::RowBlock b;
    if (!pages::find_block(s, 1, 1, tok, b)) return;  // a row behind the last sequence
    // blocks of one row each are numbered over the sequences' rows alone; rows
    // that belong to nobody lie behind them, so the block's row is the token
    // (q_start ascending from 0, as documented)
    const int pos = b.p0 + b.blk;
    if (pos < 0 || pos >= b.T || b.q0 + b.blk != tok) return;  // (at T and behind it: no room in the table)
    const int page = __ldg(s.table + (long long)b.seq * s.tstride + (pos >> s.pshift));
    if (page < 0 || page >= s.pages) {
        if (lane == 0) flag(s.status, kPgBadPage);
        return;
    }
    const int slot = pos & ((1 << s.pshift) - 1);
    // piece i: head i >> chshift
    auto at = [&](int i) {
        const int h = i >> chshift, c = i & ((1 << chshift) - 1);
        return (((((long long)page * s.Hk + h) << s.pshift) + slot) << chshift) + c;
    };
#pragma unroll
    for (int u = 0; u < kAppPieces; ++u) {
        const int i = lane + 32 * u;
        if (i < pieces) Kp[at(i)] = kv[u], Vp[at(i)] = vv[u];
    }
    for (int i0 = 32 * kAppPieces; i0 < pieces; i0 += 32 * kAppPieces) {
#pragma unroll
        for (int u = 0; u < kAppPieces; ++u) {
            const int i = i0 + lane + 32 * u;
            if (i < pieces) kv[u] = ks[i], vv[u] = vs[i];
        }
#pragma unroll
        for (int u = 0; u < kAppPieces; ++u) {
            const int i = i0 + lane + 32 * u;
            if (i < pieces) Kp[at(i)] = kv[u], Vp[at(i)] = vv[u];
        }
    }
}

// --------------------------------------------------------------------- copy
// The pairs travel in the launch's parameters: nothing to upload, and a
// captured launch keeps its own. Two sizes, as a small parameter block
// launches sooner.
template <int NP>
struct CopyPairs {
    int src[NP], dst[NP];
};
constexpr int kCopyFew = 64, kCopyMany = 3840;
constexpr int kCopyThreads = 256, kCopyUnroll = 4;
constexpr int kCopyPiece = kCopyThreads * kCopyUnroll;  // 16-byte pieces per CTA

// grid (parts of a page, pairs, layers x {K, V})
template <int NP>
__global__ void __launch_bounds__(kCopyThreads)
pages_copy_kernel(uint4* __restrict__ K, uint4* __restrict__ V, long long layer_stride, int page_pieces,
                  const __grid_constant__ CopyPairs<NP> pr) {
    uint4* base = (blockIdx.z & 1 ? V : K) + (long long)(blockIdx.z >> 1) * layer_stride;
    const uint4* src = base + (long long)pr.src[blockIdx.y] * page_pieces;
    uint4* dst = base + (long long)pr.dst[blockIdx.y] * page_pieces;
    const int i0 = blockIdx.x * kCopyPiece + threadIdx.x;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
        if (i0 + u * kCopyThreads < page_pieces) v[u] = __ldcs(src + i0 + u * kCopyThreads);
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
        if (i0 + u * kCopyThreads < page_pieces) __stcs(dst + i0 + u * kCopyThreads, v[u]);
}

template <int NP>
cudaError_t copy_some(void* K, void* V, int layers, int pages, int pieces, const int32_t* src, const int32_t* dst, int n,
                      cudaStream_t st) {
    CopyPairs<NP> pr;
    for (int i = 0; i < n; ++i) pr.src[i] = src[i], pr.dst[i] = dst[i];
    pages_copy_kernel<NP><<<dim3((pieces + kCopyPiece - 1) / kCopyPiece, n, 2 * layers), kCopyThreads, 0, st>>>(
        static_cast<uint4*>(K), static_cast<uint4*>(V), (long long)pages * pieces, pieces, pr);
    return cudaGetLastError();
}

}  // namespace

cudaError_t copy_pages(void* K, void* V, int layers, int pages, int pieces, const int32_t* src, const int32_t* dst, int n,
                       cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < n && e == cudaSuccess;) {
        const int m = std::min(n - i, n <= kCopyFew ? kCopyFew : kCopyMany);
        e = m <= kCopyFew ? copy_some<kCopyFew>(K, V, layers, pages, pieces, src + i, dst + i, m, st)
                          : copy_some<kCopyMany>(K, V, layers, pages, pieces, src + i, dst + i, m, st);
        i += m;
    }
    return e;
}

cudaError_t launch_pages_append(const PagedSeqs& s, int head_dim, uint16_t* Kp, uint16_t* Vp, const void* K,
                                long long k_stride, const void* V, long long v_stride, cudaStream_t st) {
    pages_append_kernel<<<(s.tokens + kAppWarps - 1) / kAppWarps, kAppWarps * 32, 0, st>>>(
        s, reinterpret_cast<uint4*>(Kp), reinterpret_cast<uint4*>(Vp), static_cast<const uint4*>(K), k_stride / 8,
        static_cast<const uint4*>(V), v_stride / 8, head_dim == 128 ? 4 : 3);
    return cudaGetLastError();
}

}  // namespace kvp

// ------------------------------------------------------------------ C entries
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_pages(const kvpool_pages_t* pg, int layer) {
    if (!pg || !pg->K || !pg->V || !aligned(pg->K, 16) || !aligned(pg->V, 16) || !aligned(pg->status, 4))
        return KVPOOL_ERR_INVALID_ARG;
    if (pg->layers < 1 || pg->layers > 32767 || pg->pages < 1 || pg->kv_heads < 1 || pg->kv_heads > 65535 ||
        (pg->head_dim != 64 && pg->head_dim != 128) ||
        (pg->page_tokens != 16 && pg->page_tokens != 32 && pg->page_tokens != 64 && pg->page_tokens != 128))
        return KVPOOL_ERR_INVALID_ARG;
    // a layer's token rows (one per page, head and slot) are counted in 31 bits
    if ((long long)pg->pages * pg->kv_heads > ((1LL << 31) - 1) / pg->page_tokens) return KVPOOL_ERR_INVALID_ARG;
    if (layer < 0 || layer >= pg->layers) return KVPOOL_ERR_INVALID_ARG;
    return KVPOOL_OK;
}

int check_seqs(const kvpool_seqs_t* s) {
    if (!s || s->seqs < 1 || s->table_stride < 1 || s->tokens < 1 || s->max_q < 0 || s->max_kv < 0 ||
        !s->page_table || !s->kv_len || !s->q_start || !aligned(s->page_table, 4) || !aligned(s->kv_len, 4) ||
        !aligned(s->q_start, 4))
        return KVPOOL_ERR_INVALID_ARG;
    return KVPOOL_OK;
}

// The current device: sm_103 or KVPOOL_ERR_UNSUPPORTED; its SM count (asked
// for once per device: a device's properties do not change).
int check_device(int& sms) {
    static std::atomic<int> known[kvp::kPagedDevices];  // SM count, -1 for another architecture, 0 not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kvp::kPagedDevices) return KVPOOL_ERR_UNSUPPORTED;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return KVPOOL_ERR_CUDA;
        if (major * 10 + minor != 103) n = -1;
        known[dev].store(n, std::memory_order_relaxed);
    }
    sms = n;
    return n > 0 ? KVPOOL_OK : KVPOOL_ERR_UNSUPPORTED;
}

int map_cuda(cudaError_t e) { return e == cudaSuccess ? KVPOOL_OK : KVPOOL_ERR_CUDA; }

long long layer_elems(const kvpool_pages_t* pg) {
    return (long long)pg->pages * pg->kv_heads * pg->page_tokens * pg->head_dim;
}

kvp::PagedSeqs seqs_view(const kvpool_pages_t* pg, const kvpool_seqs_t* s) {
    kvp::PagedSeqs v{};
    v.pages = pg->pages;
    v.Hk = pg->kv_heads;
    while ((1 << v.pshift) < pg->page_tokens) ++v.pshift;
    v.seqs = s->seqs;
    v.tstride = s->table_stride;
    v.tokens = s->tokens;
    v.table = s->page_table;
    v.kv_len = s->kv_len;
    v.q_start = s->q_start;
    v.status = pg->status;
    return v;
}

}  // namespace

int kvp::check_pages_args(const kvpool_pages_t* pg, int layer) { return check_pages(pg, layer); }
int kvp::check_seqs_args(const kvpool_seqs_t* s) { return check_seqs(s); }
int kvp::check_sm103(int& sms) { return check_device(sms); }
kvp::PagedSeqs kvp::paged_seqs_view(const kvpool_pages_t* pg, const kvpool_seqs_t* s) { return seqs_view(pg, s); }

int kvp::check_copy_args(const kvpool_pages_t* pg, const int32_t* src, const int32_t* dst, int n) {
    if (n < 0 || n > pg->pages || (n > 0 && (!src || !dst))) return KVPOOL_ERR_INVALID_ARG;
    // every page at most once a destination, and then no source. Few pairs are
    // compared with one another (the decode path: a fork or two); many are
    // marked in a table of the pages.
    for (int i = 0; i < n; ++i)
        if (src[i] < 0 || src[i] >= pg->pages || dst[i] < 0 || dst[i] >= pg->pages) return KVPOOL_ERR_INVALID_ARG;
    if (n <= 64) {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < n; ++j)
                if (dst[i] == src[j] || (i != j && dst[i] == dst[j])) return KVPOOL_ERR_INVALID_ARG;
    } else {
        try {
            std::vector<bool> is_dst(pg->pages, false);
            for (int i = 0; i < n; ++i) {
                if (is_dst[dst[i]]) return KVPOOL_ERR_INVALID_ARG;
                is_dst[dst[i]] = true;
            }
            for (int i = 0; i < n; ++i)
                if (is_dst[src[i]]) return KVPOOL_ERR_INVALID_ARG;
        } catch (...) {
            return KVPOOL_ERR_OOM;
        }
    }
    return KVPOOL_OK;
}

int kvp::pages_status(int32_t* status, void* stream) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int32_t bits = 0;
    cudaError_t e = cudaMemcpyAsync(&bits, status, sizeof(bits), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, sizeof(bits), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return KVPOOL_ERR_CUDA;
    if (bits & kPgTimeout) return KVPOOL_ERR_TIMEOUT;
    if (bits & (kPgBadPage | kPgBadPosition)) return KVPOOL_ERR_INVALID_ARG;
    return KVPOOL_OK;
}

int kvp::paged_attend_args(const kvpool_pages_t* pg, int layer, const kvpool_seqs_t* seqs, const void* Q,
                           long long q_stride, int q_heads, const kvpool_score_t* score, float softmax_scale,
                           PagedAttend& a, int& max_q, int& max_kv) {
    int rc = check_pages(pg, layer);
    if (rc) return rc;
    rc = check_seqs(seqs);
    if (rc) return rc;
    if (!Q || !aligned(Q, 16)) return KVPOOL_ERR_INVALID_ARG;
    if (q_heads < pg->kv_heads || q_heads % pg->kv_heads || q_stride % 8 ||
        q_stride < (long long)q_heads * pg->head_dim)
        return KVPOOL_ERR_INVALID_ARG;
    if (!(softmax_scale >= 0.0f) || isinf(softmax_scale)) return KVPOOL_ERR_INVALID_ARG;
    if (score && (!(score->cap >= 0.0f) || isinf(score->cap) || score->window < 0 || !aligned(score->slopes, 4) ||
                  !aligned(score->first, 4) || !aligned(score->prefix, 4)))
        return KVPOOL_ERR_INVALID_ARG;
    const int group = q_heads / pg->kv_heads;
    // rows (tokens x heads of a group) are counted in 31 bits, a group in 16
    if ((long long)seqs->tokens * group > (1LL << 31) - 1024 || group > 65535) return KVPOOL_ERR_INVALID_ARG;
    a = PagedAttend{};
    a.s = seqs_view(pg, seqs);
    const long long at = layer * layer_elems(pg);
    a.K = static_cast<const uint16_t*>(pg->K) + at;
    a.V = static_cast<const uint16_t*>(pg->V) + at;
    a.Q = static_cast<const uint16_t*>(Q);
    a.q_stride = q_stride;
    a.Hq = q_heads;
    a.G = group;
    a.g_magic = (uint32_t)(((1ull << 32) + group - 1) / group);
    const float scale = softmax_scale > 0.0f ? softmax_scale : 1.0f / sqrtf((float)pg->head_dim);
    a.scale_log2 = scale * 1.4426950408889634f;
    if (isinf(a.scale_log2)) return KVPOOL_ERR_INVALID_ARG;
    if (score) {
        if (score->cap > 0.0f) {
            a.cap2 = score->cap * 1.4426950408889634f;
            a.cap_in = 2.0f * 1.4426950408889634f * scale / score->cap;
            a.cap_z = scale / score->cap;
            if (isinf(a.cap_in)) return KVPOOL_ERR_INVALID_ARG;  // (0 times it would be NaN)
            a.cap_near = 0.7f * score->cap / scale;
            for (int i = 0; i < 5; ++i) a.cap_q[i] = kTanh[i] * a.scale_log2;
        }
        a.slopes = score->slopes;
        a.window = score->window;
        a.first = score->first;
        a.prefix = score->prefix;
    }
    const long long room = std::min<long long>((long long)seqs->table_stride * pg->page_tokens, 1LL << 30);
    max_kv = (int)(seqs->max_kv > 0 ? std::min<long long>(seqs->max_kv, room) : room);
    max_q = seqs->max_q > 0 ? std::min(seqs->max_q, seqs->tokens) : seqs->tokens;
    return KVPOOL_OK;
}

cudaError_t kvp::launch_pages_attend(const PagedAttend& a, int head_dim, int max_q, int max_kv, int sm_count,
                                     cudaStream_t st) {
    // The kernel for few rows takes 16 at a time, each block of 16 through all
    // its keys: one block per sequence always; more of them while the keys read
    // over and over (from L2) stay below 128 MiB. On one sequence of 1,024 keys
    // and 128 rows per KV head it takes 14 us against 22 of the kernel for many
    // rows, of 16K keys and 32 rows 31 against 33; on 16K keys and 128 rows 59
    // against 39, on 16 sequences of 1,024 keys and 32 rows 29 against 27.
    const double blocks = (double)a.s.seqs * (((long long)max_q * a.G + 15) / 16);
    const double reads = blocks * a.s.Hk * max_kv * head_dim * 4;
    if ((long long)max_q * a.G <= 16 || reads < (double)(1 << 27))
        return launch_pages_rows(a, head_dim, max_q, max_kv, sm_count, st);
    return launch_pages_chunk(a, head_dim, max_q, max_kv, st);
}

extern "C" {

int kvpool_pages_append(const kvpool_pages_t* pg, int layer, const kvpool_seqs_t* seqs, const void* K,
                        long long k_stride, const void* V, long long v_stride, void* stream) {
    int rc = check_pages(pg, layer);
    if (rc) return rc;
    rc = check_seqs(seqs);
    if (rc) return rc;
    const long long row = (long long)pg->kv_heads * pg->head_dim;
    if (!K || !V || !aligned(K, 16) || !aligned(V, 16) || k_stride < row || v_stride < row || k_stride % 8 ||
        v_stride % 8)
        return KVPOOL_ERR_INVALID_ARG;
    int sms = 0;
    rc = check_device(sms);
    if (rc) return rc;
    const long long at = layer * layer_elems(pg);
    return map_cuda(kvp::launch_pages_append(seqs_view(pg, seqs), pg->head_dim, static_cast<uint16_t*>(pg->K) + at,
                                             static_cast<uint16_t*>(pg->V) + at, K, k_stride, V, v_stride,
                                             static_cast<cudaStream_t>(stream)));
}

int kvpool_pages_append_rotary(const kvpool_pages_t* pg, int layer, const kvpool_seqs_t* seqs,
                               const kvpool_rotary_t* rotary, const void* K, long long k_stride, const void* V,
                               long long v_stride, const void* Q, long long q_stride, int q_heads, void* Q_out,
                               long long q_out_stride, void* stream) {
    int rc = check_pages(pg, layer);
    if (rc) return rc;
    kvp::AppendArgs a{};
    rc = kvp::append_args(pg, seqs, rotary, K, k_stride, V, v_stride, Q, q_stride, q_heads, Q_out, q_out_stride, a);
    if (rc) return rc;
    if (!rotary) return KVPOOL_ERR_INVALID_ARG;
    int sms = 0;
    rc = check_device(sms);
    if (rc) return rc;
    const long long at = layer * layer_elems(pg);
    a.Kp = static_cast<uint16_t*>(pg->K) + at;
    a.Vp = static_cast<uint16_t*>(pg->V) + at;
    return map_cuda(kvp::launch_append(a, pg->head_dim, false, static_cast<cudaStream_t>(stream)));
}

int kvpool_pages_copy(const kvpool_pages_t* pg, const int32_t* src, const int32_t* dst, int n, void* stream) {
    int rc = check_pages(pg, 0);
    if (rc) return rc;
    rc = kvp::check_copy_args(pg, src, dst, n);
    if (rc) return rc;
    if (n == 0) return KVPOOL_OK;
    int sms = 0;
    rc = check_device(sms);
    if (rc) return rc;
    return map_cuda(kvp::copy_pages(pg->K, pg->V, pg->layers, pg->pages,
                                    pg->kv_heads * pg->page_tokens * pg->head_dim / 8, src, dst, n,
                                    static_cast<cudaStream_t>(stream)));
}

int kvpool_pages_attend(const kvpool_pages_t* pg, int layer, const kvpool_seqs_t* seqs, const void* Q,
                        long long q_stride, int q_heads, const kvpool_score_t* score, void* out, float* lse,
                        float softmax_scale, void* stream) {
    kvp::PagedAttend a{};
    int max_q = 0, max_kv = 0, sms = 0;
    int rc = kvp::paged_attend_args(pg, layer, seqs, Q, q_stride, q_heads, score, softmax_scale, a, max_q, max_kv);
    if (rc) return rc;
    if (!out || !aligned(out, 16) || !aligned(lse, 4)) return KVPOOL_ERR_INVALID_ARG;
    rc = check_device(sms);
    if (rc) return rc;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    return map_cuda(
        kvp::launch_pages_attend(a, pg->head_dim, max_q, max_kv, sms, static_cast<cudaStream_t>(stream)));
}

int kvpool_pages_status(const kvpool_pages_t* pg, void* stream) {
    if (!pg || !pg->status || !aligned(pg->status, 4)) return KVPOOL_ERR_INVALID_ARG;
    return kvp::pages_status(pg->status, stream);
}

}  // extern "C"
