// The paged private caches held in 4 bits: what their kernels share.
//
// A head-vector x of D channels is held as D / 8 words of eight codes u and a
// float32 scale t, and stands for t H (u - 7.5), H the Walsh-Hadamard matrix in
// Sylvester's order. Word w holds channels 8 w ... 8 w + 7 of y = H x: channel
// 8 w + 2 k in bits 4 k ... 4 k + 3, channel 8 w + 2 k + 1 sixteen bits above,
// so that one mask leaves two neighbouring channels as the halves of a register.
#pragma once

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
cudaError_t launch_pages4_rows(const PagedAttend4& a, int head_dim, int max_q, int max_kv, int sm_count,
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

}  // namespace kvp
