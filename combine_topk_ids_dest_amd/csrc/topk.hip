// The router's choice: scores of a token's logits, the experts it goes to and
// their weights, in the layout the pack takes (topk_ids, topk_weights).
//
// A wave has one token; lane l holds the experts l, l + 64, ... Scores are
// computed in fp64 and rounded once to fp32 (a softmax's sum too), so which
// expert wins at a near tie is a property of the logits, not of an
// exponential's last bit. The choice is K rounds of a maximum over the wave
// on 64-bit keys: the value in an order-preserving integer form above, the
// inverted expert index below, so equal values go to the lower index.
//
// Bound by latency at decode sizes (one wave per token, K dependent rounds
// of six lane exchanges) and by the logits' bytes only far above them.
#include "experts.h"

namespace moe_ep {
namespace {

constexpr int kRouteWaves = 4;
constexpr uint64_t kNone = 0;   // key of an expert that cannot be picked

// Order-preserving map of a finite or infinite fp32 value to uint32, larger
// for larger values, never 0. -0.0 and +0.0 are one value.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t k) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)k, off, 64);
        k = o > k ? o : k;
    }
    return k;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// V: experts per lane, E <= 64 * V.
template <int V>
__global__ __launch_bounds__(kRouteWaves * 64) void route_topk_kernel(const RouteArgs a) {
    // the groups' share: choice values of a wave's token, one group apart by
    // an odd pitch so that lanes walking different groups meet in no bank
    extern __shared__ float choice_lds[];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T) return;   // waves are independent: there is no block barrier

    float x[V];
    const uint8_t* row = a.logits + t * a.logits_stride;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        x[i] = __uint_as_float(0xFF800000u);
        if (e < a.E)
            x[i] = a.bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << 16)
                          : reinterpret_cast<const float*>(row)[e];
    }
    float b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        b[i] = a.bias && e < a.E ? a.bias[e] : 0.0f;
    }
    bool live[V];
    float m = -__builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        live[i] = x[i] > -__builtin_huge_valf();        // false for NaN and -inf
        x[i] = x[i] < 3.402823466e38f ? x[i] : 3.402823466e38f;   // +inf counts as the largest
        if (live[i]) m = fmaxf(m, x[i]);
    }
    double p[V];
    if (a.score == MOE_EP_SOFTMAX) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = live[i] ? exp((double)x[i] - (double)m) : 0.0;
            sum += p[i];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = live[i] ? p[i] / sum : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = live[i] ? 1.0 / (1.0 + exp(-(double)x[i])) : 0.0;
    }
    uint64_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float c = (float)p[i] + b[i];
        key[i] = live[i] && c > -__builtin_huge_valf()
                     ? ((uint64_t)ordered(c) << 32) | (uint32_t)~(lane + 64 * i)
                     : kNone;
    }

    if (a.n_group > 1) {
        const int per = a.E / a.n_group;
        const int pitch = per | 1;
        float* c = choice_lds + (size_t)wave * a.n_group * pitch;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            if (e < a.E)
                c[e / per * pitch + e % per] =
                    key[i] != kNone ? (float)p[i] + b[i] : -__builtin_huge_valf();
        }
        // one wave, one instruction stream: the writes above precede the
        // reads below in program order and LDS serves a wave in order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        uint64_t g = kNone;
        if (lane < a.n_group) {
            float hi = -__builtin_huge_valf(), lo = hi;
            for (int j = 0; j < per; ++j) {
                const float v = c[lane * pitch + j];
                lo = fmaxf(lo, fminf(hi, v));
                hi = fmaxf(hi, v);
            }
            // with a selection bias a group's value is the sum of its two
            // best; one that has a single expert left has that one's value
            const float v = a.bias && lo > -__builtin_huge_valf() ? hi + lo : hi;
            if (hi > -__builtin_huge_valf())
                g = ((uint64_t)ordered(v) << 32) | (uint32_t)~lane;
        }
        uint64_t kept = 0;
        for (int r = 0; r < a.topk_group; ++r) {
            const uint64_t best = wave_max(g);
            if (best == kNone) break;
            const int w = (int)~(uint32_t)best;
            kept |= 1ull << w;
            if (lane == w) g = kNone;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            if (e < a.E && !((kept >> (e / per)) & 1)) key[i] = kNone;
        }
    }

    // lane k keeps pick k
    int32_t my_id = -1;
    double my_p = 0.0, total = 0.0;
    for (int k = 0; k < a.K; ++k) {
        uint64_t best = key[0];
        double bp = p[0];
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (key[i] > best) { best = key[i]; bp = p[i]; }
        const uint64_t win = wave_max(best);
        if (win == kNone) break;                 // uniform: nothing is left
        const int id = (int)~(uint32_t)win;
        const double wp = __shfl(bp, id & 63, 64);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] == win) key[i] = kNone;   // keys are unique
        if (lane == k) { my_id = id; my_p = wp; }
        total += wp;
    }
    if (lane < a.K) {
        double w = my_p;
        if (a.renormalize) w = total > 0.0 ? w / total : 0.0;
        a.ids[t * a.K + lane] = my_id;
        a.weights[t * a.K + lane] = (float)(w * (double)a.scale);
    }
}

}  // namespace

hipError_t launch_route_topk(const RouteArgs& a, hipStream_t stream) {
    const unsigned grid = (unsigned)((a.T + kRouteWaves - 1) / kRouteWaves);
    const int per = a.n_group > 1 ? a.E / a.n_group : 0;
    const size_t lds =
        a.n_group > 1 ? (size_t)kRouteWaves * a.n_group * (per | 1) * sizeof(float) : 0;
    const dim3 blk(kRouteWaves * 64);
    if (a.E <= 64)
        route_topk_kernel<1><<<grid, blk, lds, stream>>>(a);
    else if (a.E <= 256)
        route_topk_kernel<4><<<grid, blk, lds, stream>>>(a);
    else
        route_topk_kernel<16><<<grid, blk, lds, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe_ep
