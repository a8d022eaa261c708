// C ABI of the quantised paged cache (include/qcache.h): argument checks, context set-up, kernel
// dispatch. The kernels are in qc_norm_rope.cu, qc_rows.cu and qc_attend*.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <new>

#include "qc_internal.h"

namespace {

struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    cudaError_t err = cudaSuccess;
    explicit DeviceGuard(int dev) {
        err = cudaGetDevice(&prev);
        if (err == cudaSuccess && prev != dev) {
            err = cudaSetDevice(dev);
            changed = err == cudaSuccess;
        }
    }
    ~DeviceGuard() {
        if (changed) cudaSetDevice(prev);
    }
};

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int size_of(int type) { return type == QC_F32 ? 4 : 2; }

// A stride that keeps rows on 16-byte boundaries and whose offsets over `count` rows fit 63 bits.
int check_stride(int64_t stride, int64_t count, int size) {
    if (stride < 0 || (count > 1 && stride > INT64_MAX / 16 / count)) return FQ_EINVAL;
    return count > 1 && stride * size % 16 ? FQ_EALIGN : FQ_OK;
}

int check_rows(const void *x, int64_t n, int heads, int64_t token, int64_t head, int size) {
    if (!x) return FQ_EINVAL;
    if (!aligned(x, 16)) return FQ_EALIGN;
    const int a = check_stride(token, n, size), b = check_stride(head, heads, size);
    return a != FQ_OK ? a : b;
}

int check_pages(const qc_ctx *ctx, const void *pages, int64_t n_pages) {
    if (n_pages < 0 || n_pages > INT64_MAX / 2 / qc_page_bytes(ctx) || (n_pages > 0 && !pages)) return FQ_EINVAL;
    return aligned(pages, 16) ? FQ_OK : FQ_EALIGN;
}

// What the kernels' grids take.
constexpr int64_t kMaxTokens = int64_t(1) << 32, kMaxRows = int64_t(1) << 35, kMaxPos = int64_t(1) << 40;

bool too_many(const qc_ctx *ctx, int64_t n) { return n < 0 || n > kMaxTokens || n * ctx->heads > kMaxRows; }

}  // namespace

extern "C" {

int qc_create(qc_ctx **out, int format, int d, int n_heads, int page_tokens, int device) {
    if (!out) return FQ_EINVAL;
    *out = nullptr;
    if (format < QC_INT8 || format > QC_E2M1 || (d != 64 && d != 128) || n_heads < 1 || n_heads > qc::kMaxHeads)
        return FQ_EINVAL;
    if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1))) return FQ_EINVAL;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev) return FQ_ENODEV;
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        return FQ_ENODEV;
    if (major != 10 || minor != 3) return FQ_ENODEV;
    DeviceGuard g(device);
    if (g.err != cudaSuccess) return FQ_ECUDA;
    qc_ctx *c = new (std::nothrow) qc_ctx();
    if (!c) return FQ_ENOMEM;
    c->device = device;
    c->num_sms = sms;
    c->fmt = format;
    c->d = d;
    c->heads = n_heads;
    c->page = page_tokens;
    while ((1 << c->shift) < page_tokens) ++c->shift;
    cudaError_t e = cudaMalloc((void **)&c->flags, 2 * sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemset(c->flags, 0, 2 * sizeof(uint32_t));
    if (e != cudaSuccess) {
        cudaFree(c->flags);
        delete c;
        return e == cudaErrorMemoryAllocation ? FQ_ENOMEM : FQ_ECUDA;
    }
    *out = c;
    return FQ_OK;
}

int64_t qc_page_bytes(const qc_ctx *ctx) {
    return ctx ? (int64_t)ctx->heads * qc::geometry(ctx).part : -1;
}

int qc_norm_rope(qc_ctx *ctx, int type, int64_t n, const void *q, int hq, int64_t q_token, int64_t q_head,
                 const float *wq, const void *k, int hk, int64_t k_token, int64_t k_head, const float *wk, float eps,
                 const int64_t *pos, const float *table, int64_t max_pos, int rot, int interleaved, void *q_out,
                 int64_t qo_token, int64_t qo_head, void *k_out, int64_t ko_token, int64_t ko_head, void *stream) {
    if (!ctx || type < QC_F16 || type > QC_F32 || n < 0 || n > kMaxTokens) return FQ_EINVAL;
    if (hq < 0 || hk < 0 || hq > qc::kMaxHeads || hk > qc::kMaxHeads) return FQ_EINVAL;
    if (rot < 0 || rot > ctx->d || rot % 16 || !isfinite(eps) || eps < 0.f) return FQ_EINVAL;
    if (rot > 0 && (max_pos < 0 || max_pos > kMaxPos)) return FQ_EINVAL;
    if (n == 0 || hq + hk == 0) return FQ_OK;
    const int size = size_of(type);
    for (int i = 0; i < 4; ++i) {
        const int heads = i & 1 ? hk : hq;
        if (!heads) continue;
        const void *x = i == 0 ? q : i == 1 ? k : i == 2 ? q_out : k_out;
        const int64_t tok = i == 0 ? q_token : i == 1 ? k_token : i == 2 ? qo_token : ko_token;
        const int64_t hd = i == 0 ? q_head : i == 1 ? k_head : i == 2 ? qo_head : ko_head;
        const int rc = check_rows(x, n, heads, tok, hd, size);
        if (rc != FQ_OK) return rc;
    }
    if (rot > 0 && (!pos || (!table && max_pos > 0))) return FQ_EINVAL;
    if (!aligned(wq, 16) || !aligned(wk, 16)) return FQ_EALIGN;
    if (rot > 0 && (!aligned(pos, 8) || !aligned(table, 16))) return FQ_EALIGN;
    qc::NormRope p = {};
    p.n = n;
    p.q = {q, q_out, wq, hq, q_token, q_head, qo_token, qo_head};
    p.k = {k, k_out, wk, hk, k_token, k_head, ko_token, ko_head};
    p.eps = eps;
    p.pos = pos;
    p.table = table;
    p.max_pos = max_pos;
    p.rot = rot;
    p.interleaved = interleaved != 0;
    p.flags = ctx->flags;
    DeviceGuard g(ctx->device);
    if (g.err != cudaSuccess) return FQ_ECUDA;
    return qc::launch_norm_rope(ctx, type, p, (cudaStream_t)stream) == cudaSuccess ? FQ_OK : FQ_ECUDA;
}

int qc_write(qc_ctx *ctx, int type, int64_t n, const void *k, int64_t k_token, int64_t k_head, const void *v,
             int64_t v_token, int64_t v_head, const int64_t *slots, void *pages, int64_t n_pages, void *stream) {
    if (!ctx || type < QC_F16 || type > QC_F32 || too_many(ctx, n)) return FQ_EINVAL;
    int rc = check_pages(ctx, pages, n_pages);
    if (rc != FQ_OK) return rc;
    if (n == 0) return FQ_OK;
    if ((rc = check_rows(k, n, ctx->heads, k_token, k_head, size_of(type))) != FQ_OK) return rc;
    if ((rc = check_rows(v, n, ctx->heads, v_token, v_head, size_of(type))) != FQ_OK) return rc;
    if (!slots) return FQ_EINVAL;
    if (!aligned(slots, 8)) return FQ_EALIGN;
    qc::Rows p = {};
    p.n = n;
    p.k = k;
    p.v = v;
    p.k_token = k_token;
    p.k_head = k_head;
    p.v_token = v_token;
    p.v_head = v_head;
    p.slots = slots;
    p.pages = (unsigned char *)pages;
    p.slots_end = n_pages * ctx->page;
    p.g = qc::geometry(ctx);
    p.flags = ctx->flags;
    DeviceGuard g(ctx->device);
    if (g.err != cudaSuccess) return FQ_ECUDA;
    return qc::launch_write(ctx, type, p, (cudaStream_t)stream) == cudaSuccess ? FQ_OK : FQ_ECUDA;
}

int qc_read(qc_ctx *ctx, int type, int64_t n, const int64_t *slots, const void *pages, int64_t n_pages, void *k_out,
            void *v_out, void *stream) {
    if (!ctx || type < QC_F16 || type > QC_F32 || too_many(ctx, n)) return FQ_EINVAL;
    const int rc = check_pages(ctx, pages, n_pages);
    if (rc != FQ_OK) return rc;
    if (n == 0 || (!k_out && !v_out)) return FQ_OK;
    if (!slots) return FQ_EINVAL;
    if (!aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16)) return FQ_EALIGN;
    qc::Rows p = {};
    p.n = n;
    p.k_out = k_out;
    p.v_out = v_out;
    p.slots = slots;
    p.pages = (unsigned char *)pages;
    p.slots_end = n_pages * ctx->page;
    p.g = qc::geometry(ctx);
    p.flags = ctx->flags;
    DeviceGuard g(ctx->device);
    if (g.err != cudaSuccess) return FQ_ECUDA;
    return qc::launch_read(ctx, type, p, (cudaStream_t)stream) == cudaSuccess ? FQ_OK : FQ_ECUDA;
}

int64_t qc_attend_workspace(const qc_ctx *ctx, int64_t n_seq, int n_nodes, int n_q_heads, int64_t max_len) {
    if (!ctx || n_seq < 0 || n_seq > 65535 || n_nodes < 1 || n_nodes > qc::kMaxNodes) return -1;
    if (n_q_heads < 1 || n_q_heads % ctx->heads || n_q_heads / ctx->heads > qc::kMaxGroup) return -1;
    if (max_len < 0 || max_len > INT32_MAX - 2 * qc::kMaxNodes) return -1;
    if (n_seq * n_nodes * n_q_heads > INT32_MAX) return -1;
    return qc::attend_workspace(ctx, n_seq, n_nodes, n_q_heads, max_len);
}

int qc_attend(qc_ctx *ctx, int type, int64_t n_seq, int n_nodes, int n_q_heads, const void *q, int64_t q_seq,
              int64_t q_node, int64_t q_head, const int32_t *table, int64_t table_stride, const int32_t *lens,
              const int32_t *nodes, const uint32_t *tree, const void *pages, int64_t n_pages, float scale,
              int64_t max_len, void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
    if (!ctx || (type != QC_F16 && type != QC_BF16) || !isfinite(scale)) return FQ_EINVAL;
    const int64_t want = qc_attend_workspace(ctx, n_seq, n_nodes, n_q_heads, max_len);
    if (want < 0) return FQ_EINVAL;
    int rc = check_pages(ctx, pages, n_pages);
    if (rc != FQ_OK) return rc;
    if (n_seq == 0) return FQ_OK;
    if (table_stride < (max_len + n_nodes + ctx->page - 1) / ctx->page || table_stride > INT64_MAX / 8 / n_seq)
        return FQ_EINVAL;
    if (!q || !table || !lens || !out || workspace_bytes < want || (want > 0 && !workspace)) return FQ_EINVAL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
        !aligned(nodes, 4) || !aligned(tree, 4) || !aligned(lse, 4))
        return FQ_EALIGN;
    if ((rc = check_stride(q_seq, n_seq, 2)) != FQ_OK || (rc = check_stride(q_node, n_nodes, 2)) != FQ_OK ||
        (rc = check_stride(q_head, n_q_heads, 2)) != FQ_OK)
        return rc;
    qc::Attend p = {};
    p.n_seq = (int)n_seq;
    p.n_nodes = n_nodes;
    p.n_q_heads = n_q_heads;
    p.group = n_q_heads / ctx->heads;
    p.q = q;
    p.q_seq = q_seq;
    p.q_node = q_node;
    p.q_head = q_head;
    p.table = table;
    p.table_stride = table_stride;
    p.lens = lens;
    p.nodes = nodes;
    p.tree = tree;
    p.words = (n_nodes + 31) / 32;
    p.pages = (const unsigned char *)pages;
    p.n_pages = n_pages;
    p.scale = scale;
    p.max_len = max_len;
    p.out = out;
    p.lse = lse;
    p.workspace = workspace;
    p.g = qc::geometry(ctx);
    p.flags = ctx->flags;
    DeviceGuard g(ctx->device);
    if (g.err != cudaSuccess) return FQ_ECUDA;
    return qc::launch_attend(ctx, type, p, (cudaStream_t)stream) == cudaSuccess ? FQ_OK : FQ_ECUDA;
}

int qc_status(qc_ctx *ctx, void *stream, uint32_t *flags) {
    if (!ctx || !flags) return FQ_EINVAL;
    DeviceGuard g(ctx->device);
    if (g.err != cudaSuccess) return FQ_ECUDA;
    cudaStream_t s = (cudaStream_t)stream;
    uint32_t h = 0;
    // One atomic read-and-clear on the device (see fq_status).
    cudaError_t e = fq::launch_take_flags(ctx->flags, s);
    if (e == cudaSuccess) e = cudaMemcpyAsync(&h, ctx->flags + 1, sizeof(uint32_t), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return FQ_ECUDA;
    *flags = h;
    return FQ_OK;
}

void qc_destroy(qc_ctx *ctx) {
    if (!ctx) return;
    DeviceGuard g(ctx->device);
    cudaDeviceSynchronize();
    cudaFree(ctx->flags);
    delete ctx;
}

}  // extern "C"
