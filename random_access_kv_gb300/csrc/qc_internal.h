// Internal declarations of the quantised paged cache, shared by its kernels and its C ABI (qc_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qcache.h"

struct qc_ctx {
    int device = 0;
    int num_sms = 0;
    int fmt = 0;
    int d = 0;
    int heads = 0;
    int page = 0;           // tokens per page, a power of two
    int shift = 0;          // log2(page)
    uint32_t *flags = nullptr;   // [0] sticky QC_FLAG_* word, [1] the copy qc_status takes
};

namespace fq {
// flags[1] = atomic exchange of flags[0] with 0, by one device thread (defined in fq_selftest.cu).
cudaError_t launch_take_flags(uint32_t *flags, cudaStream_t s);
}  // namespace fq

namespace qc {

constexpr int kMaxHeads = 1024, kMaxNodes = 1024, kMaxGroup = 64;

// Where things lie in one head's part of a page (bytes from the part's start).
struct Geometry {
    int d, page, shift, heads;
    int row;        // bytes of a row's codes
    int blocks;     // bytes of a row's block scales (0 unless e2m1)
    int part;       // bytes of one head's part
    __host__ __device__ int codes(int which) const { return which * page * row; }
    __host__ __device__ int scales(int which) const { return 2 * page * row + which * page * 4; }
    __host__ __device__ int block_scales(int which) const { return 2 * page * (row + 4) + which * page * blocks; }
};

inline Geometry geometry(const qc_ctx *c) {
    Geometry g;
    g.d = c->d;
    g.page = c->page;
    g.shift = c->shift;
    g.heads = c->heads;
    g.row = c->fmt == QC_E2M1 ? c->d / 2 : c->d;
    g.blocks = c->fmt == QC_E2M1 ? c->d / 16 : 0;
    g.part = 2 * c->page * (g.row + 4 + g.blocks);
    return g;
}

struct Heads {              // rows [n][heads][d] of one tensor
    const void *x;
    void *out;
    const float *w;
    int heads;
    int64_t token, head;            // strides in elements
    int64_t out_token, out_head;
};

struct NormRope {
    int64_t n;
    Heads q, k;
    float eps;
    const int64_t *pos;
    const float *table;
    int64_t max_pos;
    int rot;
    int interleaved;
    uint32_t *flags;
};

struct Rows {               // a write or a read of n tokens
    int64_t n;
    const void *k, *v;              // qc_write
    int64_t k_token, k_head, v_token, v_head;
    void *k_out, *v_out;            // qc_read
    const int64_t *slots;
    unsigned char *pages;
    int64_t slots_end;              // n_pages * page
    Geometry g;
    uint32_t *flags;
};

struct Attend {
    int n_seq, n_nodes, n_q_heads, group;
    const void *q;
    int64_t q_seq, q_node, q_head;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens, *nodes;
    const uint32_t *tree;
    int words;                      // 32-bit words of a tree row
    const unsigned char *pages;
    int64_t n_pages;
    float scale;
    int64_t max_len;
    void *out;
    float *lse;
    void *workspace;
    Geometry g;
    uint32_t *flags;
};

// Kernel launches on stream s; arguments already validated by the caller.
cudaError_t launch_norm_rope(const qc_ctx *c, int type, const NormRope &p, cudaStream_t s);
cudaError_t launch_write(const qc_ctx *c, int type, const Rows &p, cudaStream_t s);
cudaError_t launch_read(const qc_ctx *c, int type, const Rows &p, cudaStream_t s);
cudaError_t launch_attend(const qc_ctx *c, int type, const Attend &p, cudaStream_t s);
int64_t attend_workspace(const qc_ctx *c, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len);

}  // namespace qc
