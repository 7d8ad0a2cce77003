// C-ABI entry points of the MXFP4 quantiser and product, the experts on MXFP4 activations, and the
// layer's gradients: argument checks on the host before any launch, workspace carving, launch order.
#include "kernels.h"
#include "mx4.cuh"

namespace ftmoe {

static bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// shape and T of a layer call; rows R = T k + S T must be an int32
static ft_status check_layer(const ft_moe_shape* s, int32_t T, int64_t* rows) {
    ft_status r = check_shape(s);
    if (r) return r;
    if (T < 0) return fail(FT_ERR_INVALID_ARG, "T < 0");
    *rows = int64_t(T) * (s->top_k + s->num_shared);
    if (*rows > 0x7FFFFFFFll) return fail(FT_ERR_UNSUPPORTED, "%lld rows: T * (k + S) must fit in 31 bits", (long long)*rows);
    return FT_OK;
}

static ft_status product_status(int r, const char* what) {
    if (r == 1) return fail(FT_ERR_CUDA, "cuTensorMapEncodeTiled failed (%s)", what);
    if (r) return cuda_ok(cudaGetLastError(), what);
    return FT_OK;
}

// The experts on MXFP4 activations.  The tokens' codes take the front of the workspace's x_sorted
// region and h's the front of its h region (17/32 of a byte per element against two).
static ft_status run_experts_mx4(const ft_moe_shape* s, int T, const ft_moe_weights* w, const uint16_t* x,
                                 const int32_t* offsets, const int32_t* inv_pos, uint16_t* o_sorted, const WsLayout& L,
                                 void* ws, cudaStream_t st) {
    const int H = s->hidden, F = s->ffn, E = s->num_experts, S = s->num_shared;
    uint8_t* xq = ws_at<uint8_t>(ws, L.x_sorted);
    uint8_t* xs = xq + size_t(L.R) * (H / 2);
    uint8_t* hq = ws_at<uint8_t>(ws, L.h);
    uint8_t* hs = hq + size_t(L.R) * (F / 2);
    ft_status r = cuda_ok(launch_mx4_sorted_tokens(T, H, s->top_k, S, x, inv_pos, xq, xs, st), "token quantisation launch");
    if (r) return r;
    Mx4Launch g{};
    g.G = E + S; g.E = E; g.R = L.R;
    g.offsets = offsets;
    g.err = ws_at<uint32_t>(ws, L.err);
    g.early = 1;          // each product overlaps its start (tile list, first weights) with the kernel before it
    g.swiglu = 1; g.N = F; g.K = H;
    g.a = xq; g.as = xs;
    g.w = static_cast<const uint8_t*>(w->w13); g.ws = w->w13_scale;
    g.sw = static_cast<const uint8_t*>(w->shared_w13); g.sws = w->shared_w13_scale;
    g.hq = hq; g.hs = hs;
    if ((r = product_status(launch_mx4_product(g, st), "gate/up MXFP4 product launch"))) return r;
    g.swiglu = 0; g.N = H; g.K = F;
    g.a = hq; g.as = hs;
    g.w = static_cast<const uint8_t*>(w->w2); g.ws = w->w2_scale;
    g.sw = static_cast<const uint8_t*>(w->shared_w2); g.sws = w->shared_w2_scale;
    g.out = o_sorted;
    return product_status(launch_mx4_product(g, st), "down MXFP4 product launch");
}

static ft_status check_mx4_weights(const ft_moe_shape* s, const ft_moe_weights* w) {
    if (s->wdtype != FT_W_MXFP4) return fail(FT_ERR_UNSUPPORTED, "MXFP4 activations need MXFP4 weights (wdtype FT_W_MXFP4)");
    ft_status r = check_weights(s, w, true);
    if (r) return r;
    if (s->num_shared && (!al(w->shared_w13_scale, 2) || !al(w->shared_w2_scale, 2)))
        return fail(FT_ERR_INVALID_ARG, "shared MXFP4 scales must be 2-byte aligned");
    return FT_OK;
}

}  // namespace ftmoe

using namespace ftmoe;

extern "C" {

ft_status ft_mx4_quantize(int64_t rows, int32_t cols, int32_t dtype, const void* x, int64_t x_stride, uint8_t* codes,
                          uint8_t* scales, void* values, void* stream) {
    FT_TRACE("ft_mx4_quantize");
    if (rows < 0 || cols <= 0) return fail(FT_ERR_INVALID_ARG, "need rows >= 0 and cols > 0 (rows=%lld cols=%d)", (long long)rows, cols);
    if (cols % 32) return fail(FT_ERR_UNSUPPORTED, "cols %d: a row must be whole 32-element blocks", cols);
    if (dtype != FT_T_BF16 && dtype != FT_T_FP16 && dtype != FT_T_FP32) return fail(FT_ERR_INVALID_ARG, "unknown element type %d", dtype);
    if (rows == 0) return FT_OK;
    if (!x || !codes || !scales) return fail(FT_ERR_INVALID_ARG, "NULL x, codes or scales");
    const size_t es = dtype == FT_T_FP32 ? 4 : 2;
    if (!al(x, es)) return fail(FT_ERR_INVALID_ARG, "x must be aligned to its elements");
    if (!al(codes, 16) || (values && !al(values, 16))) return fail(FT_ERR_INVALID_ARG, "codes and values must be 16-byte aligned");
    if (rows > 1 && x_stride < cols) return fail(FT_ERR_INVALID_ARG, "x_stride %lld < cols %d", (long long)x_stride, cols);
    if (rows > (int64_t(1) << 40) / cols) return fail(FT_ERR_UNSUPPORTED, "more than 2^40 elements");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    ft_status s = cuda_state();
    if (s) return s;
    return cuda_ok(launch_mx4_quantize(rows, cols, dtype, x, rows > 1 ? x_stride : cols, codes, scales, values, st), "quantize launch");
}

static ft_status check_product(int32_t groups, int32_t rows, int32_t n, int32_t k) {
    if (groups <= 0 || rows < 0 || n <= 0 || k <= 0)
        return fail(FT_ERR_INVALID_ARG, "need groups, n, k > 0 and rows >= 0 (groups=%d rows=%d n=%d k=%d)", groups, rows, n, k);
    if (groups > kMaxExperts) return fail(FT_ERR_UNSUPPORTED, "groups %d > %d", groups, kMaxExperts);
    if (k % 64 || k > 16384) return fail(FT_ERR_UNSUPPORTED, "k %d: need k %% 64 == 0, k <= 16384", k);
    if (n % 8) return fail(FT_ERR_UNSUPPORTED, "n %d: need n %% 8 == 0", n);
    if ((int64_t(rows) / 32 + groups + 1) * ((n + 127) / 128) > 0x7FFFFFFFll || n > (1 << 22))
        return fail(FT_ERR_UNSUPPORTED, "rows %d x n %d is too large for one call", rows, n);
    return FT_OK;
}

size_t ft_mx4_product_workspace_bytes(int32_t groups, int32_t rows, int32_t n, int32_t k) {
    return check_product(groups, rows, n, k) == FT_OK ? kWsHeaderBytes : 0;
}

ft_status ft_mx4_product(int32_t groups, int32_t rows, int32_t n, int32_t k, const int32_t* offsets, const uint8_t* a_codes,
                         const uint8_t* a_scales, const uint8_t* w_codes, const uint8_t* w_scales, void* out, void* ws,
                         size_t ws_bytes, void* stream) {
    FT_TRACE("ft_mx4_product");
    ft_status s = check_product(groups, rows, n, k);
    if (s) return s;
    if (rows == 0) return FT_OK;
    if (!offsets || !a_codes || !a_scales || !w_codes || !w_scales || !out) return fail(FT_ERR_INVALID_ARG, "NULL pointer");
    if (!al(a_codes, 16) || !al(w_codes, 16) || !al(out, 16)) return fail(FT_ERR_INVALID_ARG, "codes and out must be 16-byte aligned");
    if (!al(a_scales, 2) || !al(w_scales, 2)) return fail(FT_ERR_INVALID_ARG, "scales must be 2-byte aligned");
    if (!ws || !al(ws, 256)) return fail(FT_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
    const size_t need = ft_mx4_product_workspace_bytes(groups, rows, n, k);
    if (ws_bytes < need) return fail(FT_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((s = cuda_state())) return s;
    Mx4Launch g{};
    g.G = groups; g.E = groups; g.R = rows; g.N = n; g.K = k;
    g.offsets = offsets;
    g.a = a_codes; g.as = a_scales; g.w = w_codes; g.ws = w_scales;
    g.out = static_cast<uint16_t*>(out);
    g.err = static_cast<uint32_t*>(ws);
    return product_status(launch_mx4_product(g, st), "MXFP4 product launch");
}

ft_status ft_moe_experts_mx4(const ft_moe_shape* shape, int32_t T, const ft_moe_weights* weights, const void* x,
                             const int32_t* offsets, const int32_t* inv_pos, void* o_sorted, void* ws, size_t ws_bytes,
                             void* stream) {
    FT_TRACE("ft_moe_experts_mx4");
    int64_t rows = 0;
    ft_status s = check_layer(shape, T, &rows);
    if (s) return s;
    if (T == 0) return FT_OK;
    if ((s = check_mx4_weights(shape, weights))) return s;
    if (!x || !offsets || !inv_pos || !o_sorted) return fail(FT_ERR_INVALID_ARG, "NULL x, permutation or output pointer");
    if (!al(x, 16) || !al(o_sorted, 16)) return fail(FT_ERR_INVALID_ARG, "x and o_sorted must be 16-byte aligned");
    WsLayout L;
    if ((s = check_ws(shape, T, ws, ws_bytes, &L))) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((s = cuda_state())) return s;
    return run_experts_mx4(shape, T, weights, static_cast<const uint16_t*>(x), offsets, inv_pos,
                           static_cast<uint16_t*>(o_sorted), L, ws, st);
}

ft_status ft_moe_layer_forward_mx4(const ft_moe_shape* shape, int32_t T, const void* x, const float* w_router,
                                   const float* bias, const ft_moe_weights* weights, void* y, int32_t* topk_idx_out,
                                   float* logits_out, void* ws, size_t ws_bytes, void* stream) {
    FT_TRACE("ft_moe_layer_forward_mx4");
    int64_t rows = 0;
    ft_status s = check_layer(shape, T, &rows);
    if (s) return s;
    if (T == 0) return FT_OK;
    if (!x || !w_router || !y) return fail(FT_ERR_INVALID_ARG, "NULL x, w_router or y");
    if (!al(x, 16) || !al(w_router, 16) || !al(y, 16)) return fail(FT_ERR_INVALID_ARG, "x, w_router, y must be 16-byte aligned");
    if ((s = check_mx4_weights(shape, weights))) return s;
    WsLayout L;
    if ((s = check_ws(shape, T, ws, ws_bytes, &L))) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((s = cuda_state())) return s;
    const int H = shape->hidden, E = shape->num_experts, k = shape->top_k, S = shape->num_shared;
    uint32_t* err = ws_at<uint32_t>(ws, L.err);
    int32_t* idx = topk_idx_out ? topk_idx_out : ws_at<int32_t>(ws, L.topk_idx);
    float* gw = ws_at<float>(ws, L.topk_w);
    float* lg = logits_out ? logits_out : ws_at<float>(ws, L.logits);
    int32_t* inv_pos = ws_at<int32_t>(ws, L.inv_pos);
    PermOut po{ws_at<int32_t>(ws, L.offsets), ws_at<int32_t>(ws, L.sorted_flat), inv_pos, ws_at<int32_t>(ws, L.sched), err,
               err + kWsReady};
    const uint16_t* xb = static_cast<const uint16_t*>(x);
    const bool fused = T <= kSmallRoute;      // the router's last CTA sorts small batches itself
    if ((s = cuda_ok(launch_route(T, H, E, k, S, xb, w_router, bias, idx, gw, lg, err, ws_at<uint16_t>(ws, L.wr_planes),
                                  ws_at<float>(ws, L.route_part), fused ? &po : nullptr, st), "route launch")))
        return s;
    if (!fused && (s = cuda_ok(launch_permute(T, k, E, S, H, idx, nullptr, nullptr, ws_at<int32_t>(ws, L.chunk_cnt),
                                              ws_at<int32_t>(ws, L.chunk_base), ws_at<int32_t>(ws, L.local_rank), po, st),
                               "permute launch")))
        return s;
    uint16_t* os = ws_at<uint16_t>(ws, L.o_sorted);
    if ((s = run_experts_mx4(shape, T, weights, xb, po.offsets, inv_pos, os, L, ws, st))) return s;
    return cuda_ok(launch_combine_dependent(T, H, k, S, L.R, os, inv_pos, gw, static_cast<uint16_t*>(y), st), "combine launch");
}

ft_status ft_moe_combine_backward(const ft_moe_shape* shape, int32_t T, const void* dy, const void* o_sorted,
                                  const int32_t* inv_pos, const float* topk_w, void* d_o_sorted, float* d_topk_w,
                                  void* stream) {
    FT_TRACE("ft_moe_combine_backward");
    int64_t rows = 0;
    ft_status s = check_layer(shape, T, &rows);
    if (s) return s;
    if (!d_o_sorted && !d_topk_w) return fail(FT_ERR_INVALID_ARG, "neither d_o_sorted nor d_topk_w is asked for");
    if (T == 0) return FT_OK;
    if (!dy || !inv_pos || !topk_w || (d_topk_w && !o_sorted)) return fail(FT_ERR_INVALID_ARG, "NULL pointer");
    if (!al(dy, 16) || !al(o_sorted, 16) || !al(d_o_sorted, 16))
        return fail(FT_ERR_INVALID_ARG, "dy, o_sorted and d_o_sorted must be 16-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((s = cuda_state())) return s;
    return cuda_ok(launch_combine_backward(T, shape->hidden, shape->top_k, shape->num_shared, int(rows),
                                           static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(o_sorted), inv_pos,
                                           topk_w, static_cast<uint16_t*>(d_o_sorted), d_topk_w, st),
                   "combine backward launch");
}

ft_status ft_moe_permute_backward(const ft_moe_shape* shape, int32_t T, const void* dx_sorted, const int32_t* inv_pos,
                                  const int32_t* topk_idx, const float* dlogits, const float* w_router, void* dx,
                                  void* stream) {
    FT_TRACE("ft_moe_permute_backward");
    int64_t rows = 0;
    ft_status s = check_layer(shape, T, &rows);
    if (s) return s;
    const int given = (topk_idx != nullptr) + (dlogits != nullptr) + (w_router != nullptr);
    if (given != 0 && given != 3)
        return fail(FT_ERR_INVALID_ARG, "the router's part needs topk_idx, dlogits and w_router together");
    if (T == 0) return FT_OK;
    if (!dx_sorted || !inv_pos || !dx) return fail(FT_ERR_INVALID_ARG, "NULL pointer");
    if (!al(dx_sorted, 16) || !al(dx, 16) || !al(w_router, 16))
        return fail(FT_ERR_INVALID_ARG, "dx_sorted, dx and w_router must be 16-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((s = cuda_state())) return s;
    return cuda_ok(launch_permute_backward(T, shape->hidden, shape->top_k, shape->num_shared, shape->num_experts, int(rows),
                                           static_cast<const uint16_t*>(dx_sorted), inv_pos, topk_idx, dlogits, w_router,
                                           static_cast<uint16_t*>(dx), st),
                   "permute backward launch");
}

ft_status ft_moe_route_backward(const ft_moe_shape* shape, int32_t T, const void* x, const int32_t* topk_idx,
                                const float* topk_w, const float* d_topk_w, const int32_t* offsets,
                                const int32_t* sorted_flat, float* dlogits, float* dw_router, float* dbias, void* ws,
                                size_t ws_bytes, void* stream) {
    FT_TRACE("ft_moe_route_backward");
    int64_t rows = 0;
    ft_status s = check_layer(shape, T, &rows);
    if (s) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool sums = dw_router || dbias;
    if (T == 0) {                              // the sums over no pairs are zeros
        if (!sums) return FT_OK;
        if ((s = cuda_state())) return s;
        if (dw_router && (s = cuda_ok(cudaMemsetAsync(dw_router, 0, sizeof(float) * size_t(shape->num_experts) * shape->hidden, st), "zero dw_router")))
            return s;
        return dbias ? cuda_ok(cudaMemsetAsync(dbias, 0, sizeof(float) * size_t(shape->num_experts), st), "zero dbias") : FT_OK;
    }
    if (!topk_w || !d_topk_w || !dlogits) return fail(FT_ERR_INVALID_ARG, "NULL topk_w, d_topk_w or dlogits");
    if (sums && (!topk_idx || !offsets || !sorted_flat)) return fail(FT_ERR_INVALID_ARG, "dw_router and dbias need topk_idx, offsets and sorted_flat");
    if (dw_router && !x) return fail(FT_ERR_INVALID_ARG, "dw_router needs x");
    if (!al(x, 16) || !al(dw_router, 16)) return fail(FT_ERR_INVALID_ARG, "x and dw_router must be 16-byte aligned");
    WsLayout L;
    if ((s = check_ws(shape, T, ws, ws_bytes, &L))) return s;
    // the partial sums take the row regions (x_sorted, h, o_sorted: 4 H + 2 F bytes per row)
    if (route_backward_part_bytes(T, shape->hidden, shape->top_k) > L.total - L.x_sorted)
        return fail(FT_ERR_WORKSPACE, "partial sums exceed the workspace's row regions");
    if ((s = cuda_state())) return s;
    return cuda_ok(launch_route_backward(T, shape->hidden, shape->top_k, shape->num_experts, static_cast<const uint16_t*>(x),
                                         topk_idx, topk_w, d_topk_w, offsets, sorted_flat, dlogits, dw_router, dbias,
                                         ws_at<uint8_t>(ws, L.x_sorted), st),
                   "route backward launch");
}

}  // extern "C"
