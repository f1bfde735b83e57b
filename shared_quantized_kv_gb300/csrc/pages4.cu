// Paged private caches in 4 bits, host side: what the calls check and hand on.
#include <math.h>

#include <algorithm>

#include "pages4.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int map_cuda(cudaError_t e) { return e == cudaSuccess ? KVPOOL_OK : KVPOOL_ERR_CUDA; }

// The pages as the checks of the bf16 ones take them.
kvpool_pages_t view(const kvpool_pages4_t* pg) {
    return {pg->K, pg->V, pg->layers, pg->pages, pg->kv_heads, pg->page_tokens, pg->head_dim, pg->status};
}

int check_pages4(const kvpool_pages4_t* pg, int layer, kvpool_pages_t& v) {
    if (!pg) return KVPOOL_ERR_INVALID_ARG;
    v = view(pg);
    const int rc = kvp::check_pages_args(&v, layer);
    if (rc) return rc;
    if (!pg->K_scale || !pg->V_scale || !aligned(pg->K_scale, 16) || !aligned(pg->V_scale, 16))
        return KVPOOL_ERR_INVALID_ARG;
    return KVPOOL_OK;
}

// Blocks of 8 rows, each through all its keys, are the kernel's for few rows while
// these are few: one sequence of 16K keys, 8 KV heads of 128: 51 us against 56 with
// 64 rows per head, 81 against 57 with 128; of 2,048 keys 24 against 25 with 256
// rows, 52 against 28 with 640. 32 heads of 64, 8,192 keys: 30 against 35 with 32
// rows, 37 against 35 with 40, 41 against 35 with 64. 2 heads of 64, 8,192 keys: 21
// against 34 with 256, 40 against 33 with 1,024. 4 heads of 128 in groups of 7,
// 20,011 keys: 31 against 65 with 56, 74 against 61 with 280. (Both kernels go by
// keys and rows; channels hardly move the border. The lengths do, which the rule
// leaves out: of 4 sequences of 2,048 keys and 128 rows the other kernel would take
// 27 us, not 41; 16 of 8,192 keys and 24 rows would take 122 here, not 167.)
constexpr double kRowsReads = 5 << 18;
bool few_rows(const kvp::PagedAttend& a, int max_q, int max_kv) {
    const long long rows = (long long)max_q * a.G, blocks = a.s.seqs * ((rows + 7) / 8);
    return rows <= 16 || (double)blocks * a.s.Hk * max_kv < kRowsReads;
}
// Rows of a sequence and KV head from which a workspace pays: more than one CTA's.
constexpr long long kMadeRows = 256;

long long layer_vectors(const kvpool_pages4_t* pg) { return (long long)pg->pages * pg->kv_heads * pg->page_tokens; }

}  // namespace

int kvp::append_args(const kvpool_pages_t* pg, const kvpool_seqs_t* seqs, const kvpool_rotary_t* rotary, const void* K,
                     long long k_stride, const void* V, long long v_stride, const void* Q, long long q_stride, int q_heads,
                     void* Q_out, long long q_out_stride, AppendArgs& a) {
    const int rc = check_seqs_args(seqs);
    if (rc) return rc;
    const long long row = (long long)pg->kv_heads * pg->head_dim;
    if (!K || !V || !aligned(K, 16) || !aligned(V, 16) || k_stride < row || v_stride < row || k_stride % 8 ||
        v_stride % 8)
        return KVPOOL_ERR_INVALID_ARG;
    if (rotary) {
        if (!rotary->cos || !rotary->sin || !aligned(rotary->cos, 16) || !aligned(rotary->sin, 16) ||
            !aligned(rotary->at, 4) || rotary->positions < 1 || rotary->dim < 16 || rotary->dim % 16 ||
            rotary->dim > pg->head_dim)
            return KVPOOL_ERR_INVALID_ARG;
        a.r = {rotary->cos, rotary->sin, rotary->at, rotary->positions, rotary->dim / 2, rotary->interleaved != 0,
               rotary->offset};
    }
    if (Q) {
        const long long qrow = (long long)q_heads * pg->head_dim;
        if (!rotary || !Q_out || q_heads < 1 || !aligned(Q, 16) || !aligned(Q_out, 16) || q_stride < qrow ||
            q_out_stride < qrow || q_stride % 8 || q_out_stride % 8)
            return KVPOOL_ERR_INVALID_ARG;
    } else if (Q_out) {
        return KVPOOL_ERR_INVALID_ARG;
    }
    a.s = paged_seqs_view(pg, seqs);
    a.K = static_cast<const uint16_t*>(K);
    a.V = static_cast<const uint16_t*>(V);
    a.Q = static_cast<const uint16_t*>(Q);
    a.Q_out = static_cast<uint16_t*>(Q_out);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.Hq = q_heads;
    return KVPOOL_OK;
}

extern "C" {

int kvpool_pages4_append(const kvpool_pages4_t* pg, int layer, const kvpool_seqs_t* seqs, const kvpool_rotary_t* rotary,
                         const void* K, long long k_stride, const void* V, long long v_stride, const void* Q,
                         long long q_stride, int q_heads, void* Q_out, long long q_out_stride, void* stream) {
    kvpool_pages_t v;
    int rc = check_pages4(pg, layer, v);
    if (rc) return rc;
    kvp::AppendArgs a{};
    rc = kvp::append_args(&v, seqs, rotary, K, k_stride, V, v_stride, Q, q_stride, q_heads, Q_out, q_out_stride, a);
    if (rc) return rc;
    int sms = 0;
    rc = kvp::check_sm103(sms);
    if (rc) return rc;
    const long long at = layer * layer_vectors(pg);
    a.Kc = static_cast<uint32_t*>(pg->K) + at * (pg->head_dim / 8);
    a.Vc = static_cast<uint32_t*>(pg->V) + at * (pg->head_dim / 8);
    a.Kt = pg->K_scale + at;
    a.Vt = pg->V_scale + at;
    return map_cuda(kvp::launch_append(a, pg->head_dim, true, static_cast<cudaStream_t>(stream)));
}

int kvpool_pages4_read(const kvpool_pages4_t* pg, int layer, const kvpool_seqs_t* seqs, void* K, void* V, void* stream) {
    kvpool_pages_t v;
    int rc = check_pages4(pg, layer, v);
    if (rc) return rc;
    rc = kvp::check_seqs_args(seqs);
    if (rc) return rc;
    if (!K || !V || !aligned(K, 16) || !aligned(V, 16)) return KVPOOL_ERR_INVALID_ARG;
    int sms = 0;
    rc = kvp::check_sm103(sms);
    if (rc) return rc;
    const long long at = layer * layer_vectors(pg);
    return map_cuda(kvp::launch_pages4_read(
        kvp::paged_seqs_view(&v, seqs), pg->head_dim, static_cast<const uint32_t*>(pg->K) + at * (pg->head_dim / 8),
        static_cast<const uint32_t*>(pg->V) + at * (pg->head_dim / 8), pg->K_scale + at, pg->V_scale + at,
        static_cast<uint16_t*>(K), static_cast<uint16_t*>(V), static_cast<cudaStream_t>(stream)));
}

int kvpool_pages4_copy(const kvpool_pages4_t* pg, const int32_t* src, const int32_t* dst, int n, void* stream) {
    kvpool_pages_t v;
    int rc = check_pages4(pg, 0, v);
    if (rc) return rc;
    rc = kvp::check_copy_args(&v, src, dst, n);
    if (rc || n == 0) return rc;
    int sms = 0;
    rc = kvp::check_sm103(sms);
    if (rc) return rc;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int vectors = pg->kv_heads * pg->page_tokens;
    cudaError_t e = kvp::copy_pages(pg->K, pg->V, pg->layers, pg->pages, vectors * pg->head_dim / 32, src, dst, n, st);
    if (e == cudaSuccess)
        e = kvp::copy_pages(pg->K_scale, pg->V_scale, pg->layers, pg->pages, vectors / 4, src, dst, n, st);
    return map_cuda(e);
}

int kvpool_pages4_attend(const kvpool_pages4_t* pg, int layer, const kvpool_seqs_t* seqs, const void* Q,
                         long long q_stride, int q_heads, const kvpool_score_t* score, void* out, float* lse,
                         float softmax_scale, void* workspace, size_t workspace_bytes, void* stream) {
    kvpool_pages_t v;
    int rc = check_pages4(pg, layer, v);
    if (rc) return rc;
    kvp::PagedAttend4 a{};
    int max_q = 0, max_kv = 0, sms = 0;
    rc = kvp::paged_attend_args(&v, layer, seqs, Q, q_stride, q_heads, score, softmax_scale, a.a, max_q, max_kv);
    if (rc) return rc;
    if (!out || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16)) return KVPOOL_ERR_INVALID_ARG;
    rc = kvp::check_sm103(sms);
    if (rc) return rc;
    const long long at = layer * layer_vectors(pg);
    a.a.K = static_cast<const uint16_t*>(pg->K) + at * (pg->head_dim / 4);
    a.a.V = static_cast<const uint16_t*>(pg->V) + at * (pg->head_dim / 4);
    a.Kt = pg->K_scale + at;
    a.Vt = pg->V_scale + at;
    a.a.out = static_cast<uint16_t*>(out);
    a.a.lse = lse;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (few_rows(a.a, max_q, max_kv)) return map_cuda(kvp::launch_pages4_rows(a, pg->head_dim, max_q, max_kv, sms, st));
    return map_cuda(kvp::launch_pages4_chunk(a, pg->head_dim, max_q, max_kv, workspace, workspace_bytes, st));
}

size_t kvpool_pages4_attend_ws_bytes(const kvpool_pages4_t* pg, const kvpool_seqs_t* seqs, int q_heads) {
    kvpool_pages_t v;
    if (check_pages4(pg, 0, v) || kvp::check_seqs_args(seqs)) return 0;
    kvp::PagedAttend a{};
    int max_q = 0, max_kv = 0;
    const long long row = (long long)q_heads * pg->head_dim;
    // (any aligned address stands for Q: nothing is read)
    if (kvp::paged_attend_args(&v, 0, seqs, pg->K, row, q_heads, nullptr, 0.0f, a, max_q, max_kv)) return 0;
    if (few_rows(a, max_q, max_kv) || (long long)max_q * a.G <= kMadeRows) return 0;
    return (size_t)kvp::pages4_chunk_ws_bytes(a.s, pg->head_dim, max_kv);
}

int kvpool_pages4_status(const kvpool_pages4_t* pg, void* stream) {
    if (!pg || !pg->status || !aligned(pg->status, 4)) return KVPOOL_ERR_INVALID_ARG;
    return kvp::pages_status(pg->status, stream);
}

}  // extern "C"
