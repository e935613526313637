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

// The part of the 4-bit products' arguments that does not go by their shape.
int check_w4(const W4Args& a, int64_t H, int64_t N, int64_t rows, int ob) {
    if (a.group != 16 && a.group != 32) return MOE_EP_EINVAL;
    if (ob == 0) return MOE_EP_EDTYPE;
    if (rows > 0 && (!a.m.x || !a.m.w || !a.s || !a.m.out)) return MOE_EP_EINVAL;
    if (H % 32 || N * ob % 16 || !aligned16(a.m.x) || !aligned16(a.m.w) || !aligned16(a.s) ||
        !aligned16(a.m.out) || !aligned16(a.m.bias) || (a.m.bias && N * 4 % 16) ||
        reinterpret_cast<uintptr_t>(a.whole) % 4)
        return MOE_EP_EALIGN;
    return MOE_EP_OK;
}

// Bytes of a row of 4-bit weights' scales.
inline int64_t w4_scale_row(int64_t H, int32_t group) { return (H / group + 15) / 16 * 16; }

// Tokens of a block of the balance loss's sums, 0: few enough tokens for a block
// per sequence, which ends the call in one launch. Calls one by one (one sequence,
// 256 experts, softmax): 64 tokens 9.1 us, with tiles and the join of them 12.2; 128
// tokens 10.5 and 12.4, 256 tokens 16.6 and 12.2. Replayed from a graph, without a
// second launch's time on the host: 64 tokens 7.9 and 9.7, 128 tokens 10.9 and 9.6
// (8 experts 8.8 and 7.5, 1024 experts 19.4 and 14.3; in 8 sequences, which are as
// many blocks, 7.5 and 16.8).
// At most 4096, so that a wave adds at most 256 scores in fp32: with 2^26 tokens
// alike in 256 tiles a mean score was 2.4e-4 off.
inline int64_t balance_tile(int64_t T) {
    if (T <= 128) return 0;
    const int64_t per = (T + 255) / 256;
    return per < 32 ? 32 : per > 4096 ? 4096 : per;
}

// Sizes of the balance loss; its slots of sums and their bytes.
int check_balance(int64_t T, int32_t E, int32_t S, int64_t* slots, size_t* bytes) {
    if (T < 0 || T > INT_MAX || E <= 0 || E > MOE_EP_MAX_ROUTE_EXPERTS || S <= 0 ||
        S > INT_MAX / 2 / E)
        return MOE_EP_EINVAL;
    const int64_t tile = balance_tile(T);
    *slots = tile ? (T + tile - 1) / tile + S : 0;
    // the sums, per sequence the parts of its loss (16 bytes per 64 experts) and a ticket
    *bytes = tile ? ((size_t)S * (((size_t)E + 63) / 64 * 16 + 4) +
                     (size_t)*slots * ((size_t)E * 8 + 4) + 15) / 16 * 16
                  : 0;
    return MOE_EP_OK;
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

int moe_ep_expert_matmul_w4(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                            const void* w_scale, int64_t w_scale_stride, int32_t group,
                            const float* w_global, const float* bias, int64_t bias_stride,
                            const int32_t* expert_num_tokens, int32_t e_local, int64_t rows,
                            int64_t H, int64_t N, int32_t act, void* out, int64_t out_stride,
                            int32_t out_dtype, void* stream) {
    W4Args a = {};
    MatmulArgs& m = a.m;
    a.s = static_cast<const uint8_t*>(w_scale);
    a.group = group;
    a.whole = w_global;
    m.x = static_cast<const uint8_t*>(x);
    m.w = static_cast<const uint8_t*>(w);
    m.out = static_cast<uint8_t*>(out);
    m.bias = bias;
    m.bias_stride = bias_stride;
    m.counts = expert_num_tokens;
    m.groups = e_local;
    m.act = act;
    m.out_dtype = out_dtype;
    if (H <= 0 || H > MOE_EP_MAX_WIDTH) return MOE_EP_EINVAL;
    int64_t nw;
    int rc = check_sizes(e_local, rows, H, N, act, H * 2, &nw);
    if (rc) return rc;
    const int ob = out_bytes(out_dtype, false);
    rc = check_w4(a, H, N, rows, ob);
    if (rc && rc != MOE_EP_EALIGN) return rc;
    const int64_t s_row = w4_scale_row(H, group);
    if (!covers(x_stride, rows, H, e_local, 2) || !covers(w_stride, nw, (H + 1) / 2, e_local, 1) ||
        !covers(w_scale_stride, nw, s_row, e_local, 1) ||
        !covers(out_stride, rows, N, e_local, ob) ||
        (bias && !covers(bias_stride, 1, nw, e_local, 4)) || !expert_num_tokens)
        return MOE_EP_EINVAL;
    if (rc || x_stride * 2 % 16 || w_stride % 16 || w_scale_stride % 16 || out_stride * ob % 16 ||
        (bias && bias_stride * 4 % 16))
        return MOE_EP_EALIGN;
    if (rows == 0) return MOE_EP_OK;
    m.x_stride = x_stride * 2;
    m.x_row = H * 2;
    m.w_stride = w_stride;
    m.w_row = H / 2;
    a.s_stride = w_scale_stride;
    a.s_row = s_row;
    m.out_stride = out_stride * ob;
    m.out_row = N * ob;
    m.rows = (int32_t)rows;
    m.N = (int32_t)N;
    m.row_bytes = (int32_t)(H * 2);
    return hip_status(launch_matmul_w4(a, static_cast<hipStream_t>(stream)));
}

int moe_ep_matmul_w4(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                     const void* w_scale, int64_t w_scale_stride, int32_t group,
                     const float* w_global, const float* bias, int64_t T, int64_t H, int64_t N,
                     int32_t act, const void* residual, int64_t residual_stride, void* out,
                     int64_t out_stride, int32_t out_dtype, void* stream) {
    // a row of codes and of scales, and all of their rows, by 32-bit offsets
    if (w_stride <= 0 || w_stride >= (1 << 30) || w_scale_stride <= 0 ||
        w_scale_stride >= (1 << 30))
        return MOE_EP_EINVAL;
    int64_t nw;
    int rc = check_sizes(1, T, H, N, act, w_stride > w_scale_stride ? w_stride : w_scale_stride,
                         &nw);
    if (rc) return rc;
    if (H * 2 > INT_MAX / nw) return MOE_EP_EINVAL;
    W4Args a = {};
    MatmulArgs& m = a.m;
    a.s = static_cast<const uint8_t*>(w_scale);
    a.s_row = w_scale_stride;
    a.group = group;
    a.whole = w_global;
    m.x = static_cast<const uint8_t*>(x);
    m.w = static_cast<const uint8_t*>(w);
    m.bias = bias;
    m.res = static_cast<const uint8_t*>(residual);
    m.out = static_cast<uint8_t*>(out);
    m.groups = 1;
    m.act = act;
    m.out_dtype = out_dtype;
    const int ob = out_bytes(out_dtype, false);
    rc = check_w4(a, H, N, T, ob);
    if (rc && rc != MOE_EP_EALIGN) return rc;
    // a tile's rows are addressed by 32-bit offsets
    const int64_t most = 1 << 23;
    if (x_stride < H || x_stride >= most / 2 || w_stride < H / 2 ||
        w_scale_stride < H / group || out_stride < N || out_stride >= most / ob)
        return MOE_EP_EINVAL;
    if (residual && (residual_stride < N || residual_stride >= most / ob)) return MOE_EP_EINVAL;
    if (residual == out && residual && residual_stride != out_stride) return MOE_EP_EINVAL;
    if (rc || x_stride * 2 % 16 || w_stride % 16 || w_scale_stride % 16 || out_stride * ob % 16 ||
        !aligned16(residual) || (residual && residual_stride * ob % 16))
        return MOE_EP_EALIGN;
    if (T == 0) return MOE_EP_OK;
    m.x_row = x_stride * 2;
    m.w_row = w_stride;
    m.res_row = residual_stride * ob;
    m.out_row = out_stride * ob;
    m.rows = (int32_t)T;
    m.N = (int32_t)N;
    m.row_bytes = (int32_t)(H * 2);
    return hip_status(launch_matmul_w4(a, static_cast<hipStream_t>(stream)));
}

int moe_ep_balance_workspace_bytes(int64_t T, int32_t E, int32_t S, size_t* bytes) {
    if (!bytes) return MOE_EP_EINVAL;
    int64_t slots;
    return check_balance(T, E, S, &slots, bytes);
}

int moe_ep_balance_loss(const void* logits, int64_t logits_stride, int32_t dtype,
                        const int32_t* topk_ids, int64_t T, int32_t E, int32_t K, int32_t score,
                        const int32_t* seq_start, int32_t S, int32_t* counts, int32_t* tokens,
                        float* mean_score, float* loss, void* workspace, size_t workspace_bytes,
                        void* stream) {
    int64_t slots;
    size_t need;
    const int rc = check_balance(T, E, S, &slots, &need);
    if (rc) return rc;
    if (K <= 0 || K > MOE_EP_MAX_SLOTS || T > INT_MAX / K) return MOE_EP_EINVAL;
    if (score != MOE_EP_SOFTMAX && score != MOE_EP_SIGMOID) return MOE_EP_EINVAL;
    if (!seq_start && S != 1) return MOE_EP_EINVAL;
    if (dtype != MOE_EP_BF16 && dtype != MOE_EP_F32) return MOE_EP_EDTYPE;
    const int eb = dtype == MOE_EP_BF16 ? 2 : 4;
    if (logits_stride < E || logits_stride > INT64_MAX / 4 / (T > 0 ? T : 1)) return MOE_EP_EINVAL;
    if ((T > 0 && (!logits || !topk_ids)) || !counts || !tokens || !mean_score || !loss)
        return MOE_EP_EINVAL;
    if (reinterpret_cast<uintptr_t>(logits) % eb || reinterpret_cast<uintptr_t>(topk_ids) % 4 ||
        reinterpret_cast<uintptr_t>(seq_start) % 4 || reinterpret_cast<uintptr_t>(counts) % 4 ||
        reinterpret_cast<uintptr_t>(tokens) % 4 || reinterpret_cast<uintptr_t>(mean_score) % 4 ||
        reinterpret_cast<uintptr_t>(loss) % 4 || (need && !aligned16(workspace)))
        return MOE_EP_EALIGN;
    if (need && (!workspace || workspace_bytes < need)) return MOE_EP_EWORKSPACE;
    BalanceArgs a = {};
    a.logits = static_cast<const uint8_t*>(logits);
    a.logits_stride = logits_stride * eb;
    a.bf16 = dtype == MOE_EP_BF16;
    a.ids = topk_ids;
    a.T = T;
    a.E = E;
    a.K = K;
    a.score = score;
    a.start = seq_start;
    a.S = S;
    a.counts = counts;
    a.mean = mean_score;
    a.tokens = tokens;
    a.loss = loss;
    if (need) {
        a.tile = balance_tile(T);
        a.part = static_cast<double*>(workspace);
        a.slot_count = reinterpret_cast<int32_t*>(a.part + (int64_t)S * ((E + 63) / 64) * 2);
        a.slot_score = reinterpret_cast<float*>(a.slot_count + slots * E);
        a.slot_tokens = reinterpret_cast<int32_t*>(a.slot_score + slots * E);
        a.ticket = a.slot_tokens + slots;
    }
    return hip_status(launch_balance(a, static_cast<hipStream_t>(stream)));
}

int moe_ep_route_backward(const void* logits, int64_t logits_stride, int32_t dtype,
                          const int32_t* topk_ids, int64_t T, int32_t E, int32_t K, int32_t score,
                          int32_t renormalize, float scale, const float* grad_weights,
                          const int32_t* seq_start, int32_t S, const int32_t* counts,
                          const int32_t* tokens, const float* grad_loss, void* grad_logits,
                          int64_t grad_stride, int32_t grad_dtype, void* stream) {
    if (T < 0 || E <= 0 || E > MOE_EP_MAX_ROUTE_EXPERTS || K <= 0 || K > MOE_EP_MAX_SLOTS ||
        T > INT_MAX / K)
        return MOE_EP_EINVAL;
    if (score != MOE_EP_SOFTMAX && score != MOE_EP_SIGMOID) return MOE_EP_EINVAL;
    if (dtype != MOE_EP_BF16 && dtype != MOE_EP_F32) return MOE_EP_EDTYPE;
    if (grad_dtype != MOE_EP_BF16 && grad_dtype != MOE_EP_F32) return MOE_EP_EDTYPE;
    const int eb = dtype == MOE_EP_BF16 ? 2 : 4, gb = grad_dtype == MOE_EP_BF16 ? 2 : 4;
    const int64_t most = INT64_MAX / 4 / (T > 0 ? T : 1);
    if (logits_stride < E || logits_stride > most || grad_stride < E || grad_stride > most)
        return MOE_EP_EINVAL;
    if (grad_logits == logits && logits && (grad_stride != logits_stride || grad_dtype != dtype))
        return MOE_EP_EINVAL;
    if (!grad_weights && !grad_loss) return MOE_EP_EINVAL;
    if (grad_loss &&
        (!counts || !tokens || S <= 0 || S > INT_MAX / 2 / E || (!seq_start && S != 1)))
        return MOE_EP_EINVAL;
    if (T > 0 && (!logits || !topk_ids || !grad_logits)) return MOE_EP_EINVAL;
    if (reinterpret_cast<uintptr_t>(logits) % eb || reinterpret_cast<uintptr_t>(grad_logits) % gb ||
        reinterpret_cast<uintptr_t>(topk_ids) % 4 ||
        reinterpret_cast<uintptr_t>(grad_weights) % 4 ||
        reinterpret_cast<uintptr_t>(seq_start) % 4 || reinterpret_cast<uintptr_t>(counts) % 4 ||
        reinterpret_cast<uintptr_t>(tokens) % 4 || reinterpret_cast<uintptr_t>(grad_loss) % 4)
        return MOE_EP_EALIGN;
    if (T == 0) return MOE_EP_OK;
    RouteGradArgs a = {};
    a.logits = static_cast<const uint8_t*>(logits);
    a.logits_stride = logits_stride * eb;
    a.bf16 = dtype == MOE_EP_BF16;
    a.ids = topk_ids;
    a.T = T;
    a.E = E;
    a.K = K;
    a.score = score;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    a.grad_weights = grad_weights;
    a.grad_loss = grad_loss;
    a.start = seq_start;
    a.S = S;
    a.counts = counts;
    a.tokens = tokens;
    a.grad = static_cast<uint8_t*>(grad_logits);
    a.grad_stride = grad_stride * gb;
    a.grad_bf16 = grad_dtype == MOE_EP_BF16;
    // blocks of four waves: a token each where there are few, up to eight
    const int64_t per = (T + 2047) / 2048;
    a.tile = per <= 4 ? 4 : per >= 32 ? 32 : (per + 3) / 4 * 4;
    // (a grid has fewer than 2^32 threads)
    if (T >> 20 > 31) a.tile = ((T >> 20) + 32) / 32 * 32;
    return hip_status(launch_route_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
