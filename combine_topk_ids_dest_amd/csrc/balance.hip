// A router's training terms: per-expert counts, mean scores and the balance
// loss of sequences of tokens, and the gradient of the logits.
//
//   q[t,e]  softmax(x)[e], or sigmoid(x[e]) / sum_j sigmoid(x[j])
//   c[e]    picks of e, n tokens that have a pick; P[e] = sum_t q[t,e] / n
//   loss    E * sum_e (c[e] / sum c) P[e]; c is a constant to its gradient:
//   dx[t,e] = q[t,e] (a[e] - sum_j q[t,j] a[j]), a[e] = g E c[e] / (sum c * n),
//             for sigmoid scores times 1 - sigmoid(x[e])
//
// A wave has one token at a time, lane l the experts l, l + 64, ... Exponentials
// and sums over a token's experts are fp32 (a result is used once, in fp32: no
// choice hangs on its last bit); sums over tokens are fp32 within a block's
// tokens and fp64 over blocks, always in the same order. Counts are integers.
#include <type_traits>

#include "experts.h"

namespace moe_ep {
namespace {

constexpr int kTokenWaves = 16;                  // of a block of the sums
constexpr int kTokenThreads = kTokenWaves * 64;
constexpr int kGradWaves = 4;

// v of the lane that CTRL names (`none` where there is none, or in the rows
// that ROWS leaves out).
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float v, float none) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        (int)__float_as_uint(none), (int)__float_as_uint(v), CTRL, ROWS, 0xF, false));
}

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

// Rows of 16 lanes by shifts of 1, 2, 4, 8, then row 0 into 1 and 2 into 3,
// then rows 0-1 into 2-3: lane 63 has the whole, which every lane gets.
__device__ __forceinline__ float wave_sum(float v) {
    v += moved<0x111, 0xF>(v, 0.f);
    v += moved<0x112, 0xF>(v, 0.f);
    v += moved<0x114, 0xF>(v, 0.f);
    v += moved<0x118, 0xF>(v, 0.f);
    v += moved<0x142, 0xA>(v, 0.f);
    v += moved<0x143, 0xC>(v, 0.f);
    return lane_value(v, 63);
}

__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, moved<0x111, 0xF>(v, v));
    v = fmaxf(v, moved<0x112, 0xF>(v, v));
    v = fmaxf(v, moved<0x114, 0xF>(v, v));
    v = fmaxf(v, moved<0x118, 0xF>(v, v));
    v = fmaxf(v, moved<0x142, 0xA>(v, v));
    v = fmaxf(v, moved<0x143, 0xC>(v, v));
    return lane_value(v, 63);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
    return v;
}

__device__ __forceinline__ float load_logit(const uint8_t* row, bool bf16, int e) {
    return bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << 16)
                : reinterpret_cast<const float*>(row)[e];
}

// A logit of -inf or NaN belongs to no expert; +inf counts as the largest fp32.
__device__ __forceinline__ bool is_live(float x) { return x > -__builtin_huge_valf(); }
__device__ __forceinline__ float finite(float x) { return x < 3.402823466e38f ? x : 3.402823466e38f; }

// Where sequence s of T tokens begins and ends.
struct Span {
    int64_t lo, hi;
};

__device__ __forceinline__ Span span_of(const int32_t* start, int64_t T, int s) {
    Span r = {0, T};
    if (start) {
        const int64_t lo = start[s], hi = start[s + 1];
        r.lo = lo < 0 ? 0 : lo > T ? T : lo;
        r.hi = hi < r.lo ? r.lo : hi > T ? T : hi;
    }
    return r;
}

// The first sequence that ends behind token t (S: none).
__device__ __forceinline__ int first_behind(const int32_t* start, int S, int64_t T, int64_t t) {
    if (!start) return 0;
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (start[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// A token's scores q, and for sigmoid scores rest = 1 - sigmoid(x). x: the
// lane's logits (-inf or NaN: 0). Sigmoid scores are taken times e^-m with
// m = min(0, the largest logit), so that a token of far negative logits has
// scores too.
template <int V, bool SIGMOID>
__device__ __forceinline__ void scores(const float (&x)[V], float (&q)[V], float (&rest)[V],
                                       float& top, float& inv) {
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (is_live(x[i])) m = fmaxf(m, finite(x[i]));
    m = wave_max(m);
    if (SIGMOID) m = fminf(m, 0.f);
    const float em = SIGMOID ? expf(m) : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float v = finite(x[i]);
        if (SIGMOID) {
            const float z = expf(v > 0.f ? -v : v - m);
            const float d = 1.f + (v > 0.f ? z : z * em);
            q[i] = (v > 0.f ? 1.f : z) / d;
            rest[i] = (v > 0.f ? z : 1.f) / d;
        } else {
            q[i] = expf(v - m);
            rest[i] = 1.f;
        }
        if (!is_live(x[i])) q[i] = 0.f;
        sum += q[i];
    }
    sum = wave_sum(sum);
    top = m;
    inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] *= inv;
}

// Sums over a block of a per-thread value pair.
__device__ __forceinline__ void block_sums(double& a, double& b, double* lds) {
    a = wave_sum(a);
    b = wave_sum(b);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        lds[2 * (threadIdx.x >> 6)] = a;
        lds[2 * (threadIdx.x >> 6) + 1] = b;
    }
    __syncthreads();
    a = b = 0.0;
    for (int w = 0; w < (int)blockDim.x / 64; ++w) {
        a += lds[2 * w];
        b += lds[2 * w + 1];
    }
}

// Counts, mean scores and the loss of one sequence from its sums: thread e of
// the first E has expert e's.
__device__ __forceinline__ void finish_sequence(const BalanceArgs& a, int s, int64_t count,
                                                double score, int64_t tokens, double* lds) {
    const int e = threadIdx.x;
    double mean = 0.0;
    if (e < a.E) {
        mean = tokens > 0 ? score / (double)tokens : 0.0;
        a.counts[(int64_t)s * a.E + e] = (int32_t)count;
        a.mean[(int64_t)s * a.E + e] = (float)mean;
    }
    double picks = e < a.E ? (double)count : 0.0, both = e < a.E ? (double)count * mean : 0.0;
    block_sums(picks, both, lds);
    if (threadIdx.x == 0) {
        a.tokens[s] = (int32_t)tokens;
        a.loss[s] = (float)(picks > 0.0 ? (double)a.E * both / picks : 0.0);
    }
}

// Sums over tokens. With TILES a block has the tokens of one tile and leaves a
// sum for each sequence s in it in slot tile + s: along the tokens either the
// tile or the sequence grows from one to the next, so no two share a slot.
// Without, a block has a whole sequence and finishes it.
template <int V, bool SIGMOID, bool TILES>
__global__ __launch_bounds__(kTokenThreads) void balance_kernel(const BalanceArgs a) {
    extern __shared__ __align__(16) uint8_t lds[];
    float* const part = reinterpret_cast<float*>(lds);                   // [waves / 2][E]
    int32_t* const hist = reinterpret_cast<int32_t*>(part + kTokenWaves / 2 * a.E);   // [E]
    __shared__ int32_t counted[kTokenWaves];
    __shared__ double sums[2 * kTokenWaves];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int64_t t0 = TILES ? (int64_t)blockIdx.x * a.tile : 0;
    const int64_t t1 = TILES ? (t0 + a.tile < a.T ? t0 + a.tile : a.T) : a.T;
    for (int s = TILES ? first_behind(a.start, a.S, a.T, t0) : (int)blockIdx.x;;
         ++s) {
        if (s >= a.S) break;
        const Span span = span_of(a.start, a.T, s);
        if (TILES && span.lo >= t1) break;
        const int64_t lo = span.lo > t0 ? span.lo : t0, hi = span.hi < t1 ? span.hi : t1;
        if (TILES && hi <= lo) continue;
        for (int e = threadIdx.x; e < a.E; e += kTokenThreads) hist[e] = 0;
        __syncthreads();
        float acc[V] = {};
        int32_t tokens = 0;
        for (int64_t t = lo + wave; t < hi; t += kTokenWaves) {
            const int32_t id = lane < a.K ? a.ids[t * a.K + lane] : -1;
            const uint8_t* row = a.logits + t * a.logits_stride;
            float x[V], q[V], rest[V], top, inv;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 64 * i;
                x[i] = e < a.E ? load_logit(row, a.bf16, e) : -__builtin_huge_valf();
            }
            const bool pick = id >= 0 && id < a.E;
            if (!__ballot(pick)) continue;       // a padding token
            ++tokens;
            if (pick) atomicAdd(&hist[id], 1);
            scores<V, SIGMOID>(x, q, rest, top, inv);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += q[i];
        }
        // the upper half of the waves first, then both (LDS holds half of them)
        if (lane == 0) counted[wave] = tokens;
        float* const mine = part + wave % (kTokenWaves / 2) * a.E;
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            if (wave / (kTokenWaves / 2) == half)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (lane + 64 * i < a.E)
                        mine[lane + 64 * i] = half ? acc[i] : acc[i] + mine[lane + 64 * i];
            __syncthreads();
        }
        const int e = threadIdx.x;
        float score = 0.f;
        int32_t all = 0;
        if (e < a.E)
            for (int w = 0; w < kTokenWaves / 2; ++w) score += part[w * a.E + e];
        for (int w = 0; w < kTokenWaves; ++w) all += counted[w];
        const int32_t count = e < a.E ? hist[e] : 0;
        if (!TILES) {
            finish_sequence(a, s, count, (double)score, all, sums);
            break;
        }
        const int64_t slot = (int64_t)blockIdx.x + s;
        if (e < a.E) {
            a.slot_count[slot * a.E + e] = count;
            a.slot_score[slot * a.E + e] = score;
        }
        if (e == 0) a.slot_tokens[slot] = all;
        __syncthreads();                         // hist and part are written again
    }
}

// One block per sequence: its tiles' sums, in tile order.
__global__ __launch_bounds__(kTokenThreads) void balance_join_kernel(const BalanceArgs a) {
    __shared__ double sums[2 * kTokenWaves];
    const int s = blockIdx.x;
    const Span span = span_of(a.start, a.T, s);
    int64_t count = 0, tokens = 0;
    double score = 0.0;
    if (span.hi > span.lo) {
        const int64_t first = span.lo / a.tile, last = (span.hi - 1) / a.tile;
        for (int64_t b = first; b <= last; ++b) {
            const int64_t slot = b + s;
            tokens += a.slot_tokens[slot];
            if ((int)threadIdx.x < a.E) {
                count += a.slot_count[slot * a.E + threadIdx.x];
                score += (double)a.slot_score[slot * a.E + threadIdx.x];
            }
        }
    }
    finish_sequence(a, s, count, score, tokens, sums);
}

// The gradient of the logits. Through the picks' weights w = scale * p[pick]
// (renormalize: / the picks' sum) with g their gradient:
//   softmax, renormalised    dx[pick] += w (g - sum g w / scale)
//   softmax                  dx[e]    += sum over picks of e of w g - p[e] sum w g
//   sigmoid                  the first form (plain: w g) times 1 - sigmoid(x[pick])
// The picks' part, one exponential a token, is fp64: g - sum g w cancels.
template <int V, bool SIGMOID>
__global__ __launch_bounds__(kGradWaves * 64) void route_backward_kernel(const RouteGradArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    float each[V] = {};                          // a[e] of the sequence at hand
    int s = -1, at_s = -1;
    Span span = {0, 0};                          // of sequence s
    const int64_t t0 = (int64_t)blockIdx.x * a.tile;
    const int64_t t1 = t0 + a.tile < a.T ? t0 + a.tile : a.T;
    for (int64_t t = t0 + wave; t < t1; t += kGradWaves) {
        const int32_t id = lane < a.K ? a.ids[t * a.K + lane] : -1;
        const uint8_t* row = a.logits + t * a.logits_stride;
        float x[V], q[V], rest[V], top, inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            x[i] = e < a.E ? load_logit(row, a.bf16, e) : -__builtin_huge_valf();
        }
        const bool pick = id >= 0 && id < a.E;
        const bool counted = __ballot(pick) != 0;
        float xp = -__builtin_huge_valf();
        if (pick) xp = load_logit(row, a.bf16, id);
        float g = 0.f;
        if (pick && a.grad_weights) g = a.grad_weights[t * a.K + lane];
        scores<V, SIGMOID>(x, q, rest, top, inv);

        float dx[V] = {};
        float through = 0.f;                     // sum_j q[j] (what reaches q[j])
        bool aux = false;
        if (a.grad_loss && counted) {
            if (s < 0 || span.hi <= t) {
                if (s < a.S) s = s < 0 ? first_behind(a.start, a.S, a.T, t) : s + 1;
                for (; s < a.S && (span = span_of(a.start, a.T, s)).hi <= t; ++s) {}
            }
            aux = s < a.S && span.lo <= t;
        }
        if (aux) {
            if (at_s != s) {
                const int32_t* c = a.counts + (int64_t)s * a.E;
                float n[V], picks = 0.f;
                int64_t all = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = lane + 64 * i;
                    const int32_t v = e < a.E ? c[e] : 0;
                    n[i] = (float)v;
                    all += v;
                }
                picks = (float)wave_sum((double)all);
                const int32_t tokens = a.tokens[s];
                const float f = picks > 0.f && tokens > 0
                                    ? a.grad_loss[s] * (float)a.E / picks / (float)tokens
                                    : 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) each[i] = f * n[i];
                at_s = s;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) through += q[i] * each[i];
            through = wave_sum(through);
        }
        float back = 0.f;                        // lane k: what reaches the logit of pick k
        if (a.grad_weights && counted) {
            const bool live = pick && is_live(xp);
            const double v = (double)finite(xp);
            double w = 0.0, left = 1.0;
            if (SIGMOID) {
                const double z = live ? exp(-fabs(v)) : 0.0;
                w = live ? (v >= 0.0 ? 1.0 : z) / (1.0 + z) : 0.0;
                left = (v >= 0.0 ? z : 1.0) / (1.0 + z);
            } else if (live) {
                w = exp(v - (double)top);        // times 1 / sum, left out of a ratio
            }
            double gw = (double)g;
            if (a.renormalize) {
                const double all = wave_sum(w);
                w = all > 0.0 ? w / all : 0.0;
                gw -= wave_sum(live ? gw * w : 0.0);
            } else if (!SIGMOID) {
                w *= (double)inv;
            }
            back = live ? (float)((double)a.scale * w * gw * left) : 0.f;
            if (!SIGMOID && !a.renormalize) through += wave_sum(back);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            dx[i] = q[i] != 0.f ? q[i] * ((aux ? each[i] : 0.f) - through) * rest[i] : 0.f;
        if (a.grad_weights && counted)
            for (int k = 0; k < a.K; ++k) {
                const int e = __builtin_amdgcn_readlane(pick ? id : -1, k);
                if (e < 0) continue;
                const float v = lane_value(back, k);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e >> 6 == i && (e & 63) == lane) dx[i] += v;
            }
        uint8_t* out = a.grad + t * a.grad_stride;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            if (e >= a.E) continue;
            if (a.grad_bf16)
                reinterpret_cast<uint16_t*>(out)[e] = (uint16_t)to_bf16_rne(dx[i]);
            else
                reinterpret_cast<float*>(out)[e] = dx[i];
        }
    }
}

template <class F>
hipError_t by_width(int E, F&& f) {
    if (E <= 64) f(std::integral_constant<int, 1>{});
    else if (E <= 128) f(std::integral_constant<int, 2>{});
    else if (E <= 256) f(std::integral_constant<int, 4>{});
    else if (E <= 512) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
    return hipGetLastError();
}

}  // namespace

hipError_t launch_balance(const BalanceArgs& a, hipStream_t st) {
    const size_t lds = (size_t)(kTokenWaves / 2 + 1) * a.E * 4;
    const bool tiles = a.slot_count != nullptr;
    const unsigned grid = tiles ? (unsigned)((a.T + a.tile - 1) / a.tile) : (unsigned)a.S;
    const hipError_t rc = by_width(a.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        auto run = [&](auto sigmoid) {
            constexpr bool SG = decltype(sigmoid)::value;
            if (tiles)
                balance_kernel<V, SG, true><<<grid, kTokenThreads, lds, st>>>(a);
            else
                balance_kernel<V, SG, false><<<grid, kTokenThreads, lds, st>>>(a);
        };
        if (a.score == MOE_EP_SIGMOID) run(std::true_type{});
        else run(std::false_type{});
    });
    if (rc != hipSuccess || !tiles) return rc;
    balance_join_kernel<<<(unsigned)a.S, kTokenThreads, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteGradArgs& a, hipStream_t st) {
    const unsigned grid = (unsigned)((a.T + a.tile - 1) / a.tile);
    return by_width(a.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (a.score == MOE_EP_SIGMOID)
            route_backward_kernel<V, true><<<grid, kGradWaves * 64, 0, st>>>(a);
        else
            route_backward_kernel<V, false><<<grid, kGradWaves * 64, 0, st>>>(a);
    });
}

}  // namespace moe_ep
