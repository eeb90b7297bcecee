// mx4_api.cu -- the extern "C" entry points of the microscaled 4-bit (mx4) calls:
// argument validation and launch sequences.
#include <cstdio>

#include "mx4.cuh"

namespace moe {
namespace {

int mx_fail(int code, const char *fn, const char *what)
{
    char msg[256];
    snprintf(msg, sizeof msg, "%s: %s", fn, what);
    return report_error(code, msg);
}

// a required device pointer: not NULL, 16-byte aligned
int mx_ptr(const char *fn, const void *ptr, const char *name)
{
    char msg[128];
    if (ptr == nullptr) {
        snprintf(msg, sizeof msg, "argument '%s' is NULL", name);
        return mx_fail(MOE_ERR_INVALID_ARG, fn, msg);
    }
    if ((reinterpret_cast<uintptr_t>(ptr) & 15u) != 0) {
        snprintf(msg, sizeof msg, "argument '%s' is not 16-byte aligned", name);
        return mx_fail(MOE_ERR_ALIGN, fn, msg);
    }
    return MOE_OK;
}

#define MX_PTR(ptr)                                       \
    do {                                                  \
        const int rc_ = mx_ptr(fn, (ptr), #ptr);          \
        if (rc_ != MOE_OK)                                \
            return rc_;                                   \
    } while (0)

// Token-sized buffers may be NULL when the batch is empty (T == 0).
#define MX_TOK(ptr)                                       \
    do {                                                  \
        if (p->T > 0 || (ptr) != nullptr)                 \
            MX_PTR(ptr);                                  \
    } while (0)

#define MX_OPT(ptr)                                       \
    do {                                                  \
        if ((ptr) != nullptr)                             \
            MX_PTR(ptr);                                  \
    } while (0)

int mx_after(const char *fn, cudaError_t e)
{
    if (e == cudaSuccess)
        e = cudaGetLastError();
    return e == cudaSuccess ? report_ok() : report_cuda(e, fn);
}

// the layer as the mx4 calls take it
int mx_params(const char *fn, const moe_params_t *p)
{
    const int rc = validate_params(fn, p);
    if (rc != MOE_OK)
        return rc;
    if (p->d % kMx4Block != 0)
        return mx_fail(MOE_ERR_SHAPE, fn, "d is not a multiple of 32");
    return MOE_OK;
}

// a bf16 layer and its workspace
int mx_layer(const char *fn, const moe_params_t *p, void *ws, size_t ws_bytes)
{
    const int rc = mx_params(fn, p);
    if (rc != MOE_OK)
        return rc;
    if (p->dtype != MOE_BF16)
        return mx_fail(MOE_ERR_DTYPE, fn, "the mx4 experts are bf16 layers");
    if (mx_ptr(fn, ws, "ws") != MOE_OK)
        return mx_ptr(fn, ws, "ws");
    if (ws_bytes < ws_layout(p).total)
        return mx_fail(MOE_ERR_WORKSPACE, fn, "the workspace is below moe_workspace_size");
    return MOE_OK;
}

int mx_matrix(const char *fn, int32_t dtype, int32_t G, int32_t rows, int32_t K, int64_t ld)
{
    if (dtype != MOE_BF16 && dtype != MOE_F32)
        return mx_fail(MOE_ERR_DTYPE, fn, "dtype is neither MOE_BF16 nor MOE_F32");
    if (G < 1 || rows < 1)
        return mx_fail(MOE_ERR_INVALID_ARG, fn, "G or rows is below 1");
    if (K < 8 || K % 8 != 0 || K > 1 << 22 || rows > 1 << 28)
        return mx_fail(MOE_ERR_SHAPE, fn, "K is not a positive multiple of 8, or too large");
    if (ld < K || ld % 8 != 0)
        return mx_fail(MOE_ERR_SHAPE, fn, "ld is below K or not a multiple of 8");
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_mx4_codes_bytes(int32_t G, int32_t rows, int32_t K)
{
    if (G < 1 || rows < 1 || K < 8 || K % 8 != 0)
        return 0;
    return (size_t)G * rows * (mx4_k32(K) / 2);
}

size_t moe_mx4_scales_bytes(int32_t G, int32_t rows, int32_t K)
{
    if (G < 1 || rows < 1 || K < 8 || K % 8 != 0)
        return 0;
    return (size_t)G * ((rows + 127) / 128) * ((K + 127) / 128) * kMx4Tile;
}

size_t moe_mx4_rows_bytes(const moe_params_t *p, int32_t K)
{
    if (validate_params("moe_mx4_rows_bytes", p) != MOE_OK || K < 1)
        return 0;
    const size_t rows = (size_t)p->T * p->k;
    return (rows > 0 ? rows : 1) * (mx4_k32(K) / 2);
}

size_t moe_mx4_row_scales_bytes(const moe_params_t *p, int32_t K)
{
    if (validate_params("moe_mx4_row_scales_bytes", p) != MOE_OK || K < 1)
        return 0;
    return (size_t)mx4_row_tiles((int64_t)p->T * p->k, p->E) * ((K + 127) / 128) * kMx4Tile;
}

int moe_mx4_quantize(const void *src, int32_t dtype, int32_t G, int32_t rows, int32_t K,
                     int64_t ld, void *codes, void *scales, void *stream)
{
    const char *fn = "moe_mx4_quantize";
    const int rc = mx_matrix(fn, dtype, G, rows, K, ld);
    if (rc != MOE_OK)
        return rc;
    MX_PTR(src);
    MX_PTR(codes);
    MX_PTR(scales);
    return mx_after(fn, launch_mx4_quantize(src, dtype, G, rows, K, ld, codes, scales,
                                            (cudaStream_t)stream));
}

int moe_mx4_dequantize(const void *codes, const void *scales, int32_t dtype, int32_t G,
                       int32_t rows, int32_t K, int64_t ld, void *dst, void *stream)
{
    const char *fn = "moe_mx4_dequantize";
    const int rc = mx_matrix(fn, dtype, G, rows, K, ld);
    if (rc != MOE_OK)
        return rc;
    MX_PTR(codes);
    MX_PTR(scales);
    MX_PTR(dst);
    return mx_after(fn, launch_mx4_dequantize(codes, scales, dtype, G, rows, K, ld, dst,
                                              (cudaStream_t)stream));
}

int moe_mx4_dispatch(const moe_params_t *p, const void *x, const int32_t *topk_idx,
                     const int32_t *slot_row, const int32_t *offsets, void *x_q, void *x_s,
                     void *stream)
{
    const char *fn = "moe_mx4_dispatch";
    const int rc = mx_params(fn, p);
    if (rc != MOE_OK)
        return rc;
    MX_TOK(x);
    MX_TOK(topk_idx);
    MX_TOK(slot_row);
    MX_PTR(offsets);
    MX_TOK(x_q);
    MX_TOK(x_s);
    if (p->T == 0)
        return report_ok();
    return mx_after(fn, launch_mx4_dispatch(p, x, topk_idx, slot_row, offsets, x_q, x_s,
                                            (cudaStream_t)stream));
}

int moe_expert_up_mx4(const moe_params_t *p, const void *x_q, const void *x_s,
                      const int32_t *offsets, const void *W13_q, const void *W13_s, void *h_q,
                      void *h_s, void *ws, size_t ws_bytes, void *stream)
{
    const char *fn = "moe_expert_up_mx4";
    const int rc = mx_layer(fn, p, ws, ws_bytes);
    if (rc != MOE_OK)
        return rc;
    MX_TOK(x_q);
    MX_TOK(x_s);
    MX_PTR(offsets);
    MX_PTR(W13_q);
    MX_PTR(W13_s);
    MX_TOK(h_q);
    MX_TOK(h_s);
    if (p->T == 0)
        return report_ok();
    return mx_after(fn, launch_mx4_up(p, x_q, x_s, offsets, W13_q, W13_s, h_q, h_s,
                                      reinterpret_cast<int32_t *>(ws), (cudaStream_t)stream));
}

int moe_expert_down_mx4(const moe_params_t *p, const void *h_q, const void *h_s,
                        const int32_t *offsets, const void *W2_q, const void *W2_s, void *out,
                        void *ws, size_t ws_bytes, void *stream)
{
    const char *fn = "moe_expert_down_mx4";
    const int rc = mx_layer(fn, p, ws, ws_bytes);
    if (rc != MOE_OK)
        return rc;
    MX_TOK(h_q);
    MX_TOK(h_s);
    MX_PTR(offsets);
    MX_PTR(W2_q);
    MX_PTR(W2_s);
    MX_TOK(out);
    if (p->T == 0)
        return report_ok();
    return mx_after(fn, launch_mx4_down(p, h_q, h_s, offsets, W2_q, W2_s, out, false,
                                        reinterpret_cast<int32_t *>(ws), (cudaStream_t)stream));
}

int moe_expert_ffn_mx4(const moe_params_t *p, const void *x_q, const void *x_s,
                       const int32_t *offsets, const void *W13_q, const void *W13_s,
                       const void *W2_q, const void *W2_s, void *h_q, void *h_s, void *out,
                       void *ws, size_t ws_bytes, void *stream)
{
    const char *fn = "moe_expert_ffn_mx4";
    int rc = mx_layer(fn, p, ws, ws_bytes);
    if (rc != MOE_OK)
        return rc;
    MX_PTR(W2_q);  // the second half's arguments before the first half is launched
    MX_PTR(W2_s);
    MX_TOK(out);
    if ((rc = moe_expert_up_mx4(p, x_q, x_s, offsets, W13_q, W13_s, h_q, h_s, ws, ws_bytes,
                                stream)) != MOE_OK || p->T == 0)
        return rc;
    return mx_after(fn, launch_mx4_down(p, h_q, h_s, offsets, W2_q, W2_s, out, true,
                                        reinterpret_cast<int32_t *>(ws), (cudaStream_t)stream));
}

int moe_forward_mx4(const moe_params_t *p, const moe_mx4_buffers_t *b, int32_t act, void *ws,
                    size_t ws_bytes, void *stream)
{
    const char *fn = "moe_forward_mx4";
    int rc = mx_layer(fn, p, ws, ws_bytes);
    if (rc != MOE_OK)
        return rc;
    if (b == nullptr)
        return mx_fail(MOE_ERR_INVALID_ARG, fn, "buffers is NULL");
    if (act != MOE_MX4_ACT_BF16 && act != MOE_MX4_ACT_MX4)
        return mx_fail(MOE_ERR_INVALID_ARG, fn, "act is neither MOE_MX4_ACT_BF16 nor MOE_MX4_ACT_MX4");
    MX_TOK(b->x);
    MX_PTR(b->Wg);
    MX_OPT(b->Wnoise);
    MX_OPT(b->noise);
    MX_OPT(b->bias);
    MX_OPT(b->router_packed);
    MX_PTR(b->W13_q);
    MX_PTR(b->W13_s);
    MX_PTR(b->W2_q);
    MX_PTR(b->W2_s);
    MX_TOK(b->y);
    MX_PTR(b->loss);
    MX_PTR(b->counts);
    MX_PTR(b->importance);
    MX_PTR(b->f);
    MX_PTR(b->P);
    MX_TOK(b->topk_idx);
    MX_TOK(b->topk_w);
    MX_PTR(b->probs_sum);
    MX_TOK(b->row_token);
    MX_TOK(b->slot_row);
    MX_PTR(b->kept);
    MX_PTR(b->offsets);
    if (b->Wnoise != nullptr && b->noise == nullptr && p->T > 0)
        return mx_fail(MOE_ERR_INVALID_ARG, fn, "Wnoise given without the noise draws");
    if (act == MOE_MX4_ACT_BF16 && p->T > 0) {
        if (p->T > MOE_MX4_FEW_TOKENS)
            return mx_fail(MOE_ERR_UNSUPPORTED, fn, "MOE_MX4_ACT_BF16 takes at most 16 tokens");
        if (!mx4_few_fits(p, b->Wnoise != nullptr))
            return mx_fail(MOE_ERR_UNSUPPORTED, fn,
                           "MOE_MX4_ACT_BF16 takes at most 32 experts, 16 with noise");
        MX_PTR(b->h);
        return mx_after(fn, launch_mx4_few(p, b, static_cast<char *>(ws), (cudaStream_t)stream));
    }
    MX_TOK(b->x_q);
    MX_TOK(b->x_s);
    MX_TOK(b->h_q);
    MX_TOK(b->h_s);
    MX_TOK(b->out);
    char *w = static_cast<char *>(ws);
    int32_t *status = reinterpret_cast<int32_t *>(ws);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = launch_route(p, b->x, b->Wg, b->Wnoise, b->router_packed, b->noise, b->bias,
                                 b->topk_idx, b->topk_w, b->probs_sum, b->importance, w, status, s);
    if (e == cudaSuccess)
        e = launch_dispatch(p, nullptr, b->topk_idx, nullptr, b->row_token, b->slot_row, b->counts,
                            b->kept, b->offsets, w, status, true, s);
    if (e == cudaSuccess && p->T > 0) {
        if ((e = launch_mx4_dispatch(p, b->x, b->topk_idx, b->slot_row, b->offsets, b->x_q, b->x_s,
                                     s)) == cudaSuccess &&
            (e = launch_mx4_up(p, b->x_q, b->x_s, b->offsets, b->W13_q, b->W13_s, b->h_q, b->h_s,
                               status, s)) == cudaSuccess &&
            (e = launch_mx4_down(p, b->h_q, b->h_s, b->offsets, b->W2_q, b->W2_s, b->out, true,
                                 status, s)) == cudaSuccess)
            e = launch_combine(p, b->out, b->slot_row, b->topk_w, b->y, s);
    }
    if (e == cudaSuccess)
        e = launch_gate_stats(p, b->counts, b->probs_sum, b->f, b->P, b->loss, s);
    return mx_after(fn, e);
}

}  // extern "C"
