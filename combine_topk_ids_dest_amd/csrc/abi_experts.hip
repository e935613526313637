// C ABI of the router's choice and of the products: argument checks and the
// launch. Every check runs before anything is enqueued.
#include <limits.h>

#include "experts.h"

using namespace moe_ep;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_EP_OK : MOE_EP_EHIP; }

// Bytes of an element of the output, 0 for a type that the call lacks.
inline int out_bytes(int32_t dtype, bool fp8) {
    if (dtype == MOE_EP_BF16) return 2;
    if (dtype == MOE_EP_F32) return 4;
    return fp8 && dtype == MOE_EP_E4M3 ? 1 : 0;
}

inline int64_t scale_pitch(int64_t columns) { return (columns / kScaleBlock + 3) / 4 * 4; }

// stride >= rows * width without forming the product, and small enough that
// `blocks` of `bytes`-byte elements stay addressable.
inline bool covers(int64_t stride, int64_t rows, int64_t width, int64_t blocks, int64_t bytes) {
    if (stride < 0 || stride > INT64_MAX / bytes / (blocks > 0 ? blocks : 1)) return false;
    return rows <= 0 || stride / width >= rows;
}

// Sizes that the calls share; nw = rows of w.
int check_sizes(int32_t groups, int64_t rows, int64_t H, int64_t N, int32_t act, int64_t w_row,
                int64_t* nw) {
    // sums like rows + 255 (runs of rows, and where they end) stay below 2^31
    if (groups <= 0 || groups > MOE_EP_MAX_LOCAL_EXPERTS || rows < 0 || rows > INT_MAX - 255 ||
        H <= 0 || H > MOE_EP_MAX_WIDTH || N <= 0 || N > MOE_EP_MAX_WIDTH)
        return MOE_EP_EINVAL;
    if (act < MOE_EP_ACT_NONE || act > MOE_EP_ACT_SILU_GATED) return MOE_EP_EINVAL;
    *nw = act == MOE_EP_ACT_SILU_GATED ? 2 * N : N;
    if (w_row <= 0 || *nw > INT_MAX / w_row) return MOE_EP_EINVAL;
    // tile numbers and the steps over them stay below 2^31
    if ((int64_t)groups * ((rows + 15) / 16) > (INT_MAX / 2) / ((N + 7) / 8)) return MOE_EP_EINVAL;
    return MOE_EP_OK;
}

int expert_matmul(MatmulArgs a, int64_t rows, int64_t H, int64_t N, const float* x_scale,
                  int64_t x_scale_stride, const float* w_scale, int64_t w_scale_stride,
                  float* out_scale, int64_t out_scale_stride, void* stream) {
    const int eb = a.fp8 ? 1 : 2;
    if (H <= 0 || H > MOE_EP_MAX_WIDTH) return MOE_EP_EINVAL;
    int64_t nw;
    const int rc = check_sizes(a.groups, rows, H, N, a.act, H * eb, &nw);
    if (rc) return rc;
    const int ob = out_bytes(a.out_dtype, a.fp8);
    if (ob == 0) return MOE_EP_EDTYPE;
    const bool e4m3 = a.out_dtype == MOE_EP_E4M3;
    if (a.fp8 && (H % kScaleBlock || (e4m3 && N % kScaleBlock))) return MOE_EP_EINVAL;
    if (e4m3 != (out_scale != nullptr)) return MOE_EP_EINVAL;
    if (!covers(a.x_stride, rows, H, a.groups, eb) || !covers(a.w_stride, nw, H, a.groups, eb) ||
        !covers(a.out_stride, rows, N, a.groups, ob) ||
        (a.bias && !covers(a.bias_stride, 1, nw, a.groups, 4)))
        return MOE_EP_EINVAL;
    if (a.fp8) {
        const int64_t per = (N + kScaleBlock - 1) / kScaleBlock;
        if (!covers(x_scale_stride, rows, scale_pitch(H), a.groups, 4) ||
            !covers(w_scale_stride, nw / N * per, H / kScaleBlock, a.groups, 4) ||
            (e4m3 && !covers(out_scale_stride, rows, scale_pitch(N), a.groups, 4)))
            return MOE_EP_EINVAL;
    }
    if (!a.counts) return MOE_EP_EINVAL;
    if (rows > 0 && (!a.x || !a.w || !a.out || (a.fp8 && (!x_scale || !w_scale))))
        return MOE_EP_EINVAL;
    if (H * eb % 16 || N * ob % 16 || a.x_stride * eb % 16 || a.w_stride * eb % 16 ||
        a.out_stride * ob % 16 || !aligned16(a.x) || !aligned16(a.w) || !aligned16(a.out) ||
        !aligned16(a.bias) || (a.bias && (N * 4 % 16 || a.bias_stride * 4 % 16)))
        return MOE_EP_EALIGN;
    if (a.fp8 && (!aligned16(x_scale) || !aligned16(w_scale) || !aligned16(out_scale) ||
                  x_scale_stride % 4 || (e4m3 && out_scale_stride % 4)))
        return MOE_EP_EALIGN;
    if (rows == 0) return MOE_EP_OK;
    a.x_row = a.w_row = H * eb;
    a.x_stride *= eb;
    a.w_stride *= eb;
    a.out_row = N * ob;
    a.out_stride *= ob;
    a.rows = (int32_t)rows;
    a.N = (int32_t)N;
    a.row_bytes = (int32_t)(H * eb);
    if (a.fp8) {
        a.xs = x_scale;
        a.xs_stride = x_scale_stride;
        a.xs_pitch = scale_pitch(H);
        a.ws = w_scale;
        a.ws_stride = w_scale_stride;
        a.os = out_scale;
        a.os_stride = out_scale_stride;
        a.os_pitch = scale_pitch(N);
    }
    return hip_status(launch_matmul(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int moe_ep_route_topk(const void* logits, int64_t logits_stride, int32_t dtype,
                      const float* bias, int64_t T, int32_t E, int32_t K, int32_t score,
                      int32_t n_group, int32_t topk_group, int32_t renormalize, float scale,
                      int32_t* topk_ids, float* topk_weights, void* stream) {
    if (T < 0 || E <= 0 || E > MOE_EP_MAX_ROUTE_EXPERTS || K <= 0 || K > MOE_EP_MAX_SLOTS || K > E)
        return MOE_EP_EINVAL;
    if (score != MOE_EP_SOFTMAX && score != MOE_EP_SIGMOID) return MOE_EP_EINVAL;
    if (n_group <= 0 || n_group > 64 || E % n_group || topk_group <= 0 || topk_group > n_group ||
        K > topk_group * (E / n_group))
        return MOE_EP_EINVAL;
    if (dtype != MOE_EP_BF16 && dtype != MOE_EP_F32) return MOE_EP_EDTYPE;
    const int eb = dtype == MOE_EP_BF16 ? 2 : 4;
    if (T > INT_MAX / K) return MOE_EP_EINVAL;
    if (logits_stride < E || logits_stride > INT64_MAX / 4 / (T > 0 ? T : 1)) return MOE_EP_EINVAL;
    if (T > 0 && (!logits || !topk_ids || !topk_weights)) return MOE_EP_EINVAL;
    if (reinterpret_cast<uintptr_t>(logits) % eb || reinterpret_cast<uintptr_t>(bias) % 4 ||
        reinterpret_cast<uintptr_t>(topk_ids) % 4 || reinterpret_cast<uintptr_t>(topk_weights) % 4)
        return MOE_EP_EALIGN;
    if (T == 0) return MOE_EP_OK;
    RouteArgs a = {};
    a.logits = static_cast<const uint8_t*>(logits);
    a.logits_stride = logits_stride * eb;
    a.bf16 = dtype == MOE_EP_BF16;
    a.bias = bias;
    a.T = T;
    a.E = E;
    a.K = K;
    a.score = score;
    a.n_group = n_group;
    a.topk_group = topk_group;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    a.ids = topk_ids;
    a.weights = topk_weights;
    return hip_status(launch_route_topk(a, static_cast<hipStream_t>(stream)));
}

int moe_ep_expert_matmul(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                         const float* bias, int64_t bias_stride,
                         const int32_t* expert_num_tokens, int32_t e_local, int64_t rows,
                         int64_t H, int64_t N, int32_t act, void* out, int64_t out_stride,
                         int32_t out_dtype, void* stream) {
    MatmulArgs a = {};
    a.x = static_cast<const uint8_t*>(x);
    a.x_stride = x_stride;
    a.w = static_cast<const uint8_t*>(w);
    a.w_stride = w_stride;
    a.bias = bias;
    a.bias_stride = bias_stride;
    a.counts = expert_num_tokens;
    a.groups = e_local;
    a.act = act;
    a.out = static_cast<uint8_t*>(out);
    a.out_stride = out_stride;
    a.out_dtype = out_dtype;
    return expert_matmul(a, rows, H, N, nullptr, 0, nullptr, 0, nullptr, 0, stream);
}

int moe_ep_expert_matmul_fp8(const void* x, int64_t x_stride, const float* x_scale,
                             int64_t x_scale_stride, const void* w, int64_t w_stride,
                             const float* w_scale, int64_t w_scale_stride, const float* bias,
                             int64_t bias_stride, const int32_t* expert_num_tokens,
                             int32_t e_local, int64_t rows, int64_t H, int64_t N, int32_t act,
                             void* out, int64_t out_stride, int32_t out_dtype,
                             float* out_scale, int64_t out_scale_stride, void* stream) {
    MatmulArgs a = {};
    a.fp8 = true;
    a.x = static_cast<const uint8_t*>(x);
    a.x_stride = x_stride;
    a.w = static_cast<const uint8_t*>(w);
    a.w_stride = w_stride;
    a.bias = bias;
    a.bias_stride = bias_stride;
    a.counts = expert_num_tokens;
    a.groups = e_local;
    a.act = act;
    a.out = static_cast<uint8_t*>(out);
    a.out_stride = out_stride;
    a.out_dtype = out_dtype;
    return expert_matmul(a, rows, H, N, x_scale, x_scale_stride, w_scale, w_scale_stride,
                         out_scale, out_scale_stride, stream);
}

int moe_ep_matmul(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                  const float* bias, int64_t T, int64_t H, int64_t N, int32_t act,
                  const void* residual, int64_t residual_stride, void* out, int64_t out_stride,
                  int32_t out_dtype, void* stream) {
    if (w_stride <= 0 || w_stride >= (1 << 30)) return MOE_EP_EINVAL;
    int64_t nw;
    const int rc = check_sizes(1, T, H, N, act, w_stride * 2, &nw);
    if (rc) return rc;
    const int ob = out_bytes(out_dtype, false);
    if (ob == 0) return MOE_EP_EDTYPE;
    // a tile's rows are addressed by 32-bit offsets
    const int64_t most = 1 << 23;
    if (x_stride < H || x_stride >= most / 2 || w_stride < H || out_stride < N ||
        out_stride >= most / ob)
        return MOE_EP_EINVAL;
    if (residual && (residual_stride < N || residual_stride >= most / ob)) return MOE_EP_EINVAL;
    if (residual == out && residual && residual_stride != out_stride) return MOE_EP_EINVAL;
    if (T > 0 && (!x || !w || !out)) return MOE_EP_EINVAL;
    if (H * 2 % 16 || N * ob % 16 || x_stride * 2 % 16 || w_stride * 2 % 16 ||
        out_stride * ob % 16 || !aligned16(x) || !aligned16(w) || !aligned16(out) ||
        !aligned16(bias) || !aligned16(residual) || (residual && residual_stride * ob % 16))
        return MOE_EP_EALIGN;
    if (T == 0) return MOE_EP_OK;
    MatmulArgs a = {};
    a.x = static_cast<const uint8_t*>(x);
    a.x_row = x_stride * 2;
    a.w = static_cast<const uint8_t*>(w);
    a.w_row = w_stride * 2;
    a.bias = bias;
    a.res = static_cast<const uint8_t*>(residual);
    a.res_row = residual_stride * ob;
    a.out = static_cast<uint8_t*>(out);
    a.out_row = out_stride * ob;
    a.groups = 1;
    a.rows = (int32_t)T;
    a.N = (int32_t)N;
    a.row_bytes = (int32_t)(H * 2);
    a.act = act;
    a.out_dtype = out_dtype;
    return hip_status(launch_matmul(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
