// The router's choice: scores of a token's logits, the experts it goes to and
// their weights, in the layout the pack takes (topk_ids, topk_weights).
//
// A wave has one token; lane l holds the experts l, l + 64, ... Scores are
// computed in fp64 and rounded once to fp32 (a softmax's sum too), so which
// expert wins at a near tie is a property of the logits, not of an
// exponential's last bit. The choice is K rounds of a maximum over the wave,
// on the values in an order-preserving integer form; among equal values the
// lowest set bit of the lowest expert range that holds one is the lowest index.
//
// Bound by the dependent steps of a wave at decode sizes (maxima and sums run
// over lanes by DPP moves, a few cycles a step, not through LDS: ten 64-bit
// maxima by lane exchanges took 4 us of 10) and by the fp64 instructions at
// prefill.
#include "experts.h"

namespace moe_ep {
namespace {

constexpr int kRouteWaves = 4;
constexpr uint32_t kNone = 0;   // key of an expert that cannot be picked

// Order-preserving map of a finite or infinite fp32 value to uint32, larger
// for larger values, never 0. -0.0 and +0.0 are one value.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One step of a reduction over the wave: v of the lane that CTRL names (0
// where there is none, or in the rows that ROWS leaves out).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL, ROWS>((uint32_t)u) |
                                          (uint64_t)dpp<CTRL, ROWS>((uint32_t)(u >> 32)) << 32);
}

// Rows of 16 lanes by shifts of 1, 2, 4, 8, then row 0 into 1 and 2 into 3,
// then rows 0-1 into 2-3: lane 63 has the whole.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp<0x111, 0xF>(v));
    v = max(v, dpp<0x112, 0xF>(v));
    v = max(v, dpp<0x114, 0xF>(v));
    v = max(v, dpp<0x118, 0xF>(v));
    v = max(v, dpp<0x142, 0xA>(v));
    v = max(v, dpp<0x143, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ double wave_sum(double v) {
    v += dpp<0x111, 0xF>(v);
    v += dpp<0x112, 0xF>(v);
    v += dpp<0x114, 0xF>(v);
    v += dpp<0x118, 0xF>(v);
    v += dpp<0x142, 0xA>(v);
    v += dpp<0x143, 0xC>(v);
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(
        double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63) |
                    (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63) << 32);
}

__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(
        double,
        (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane) |
            (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane) << 32);
}

// V: experts per lane, E <= 64 * V.
template <int V>
__global__ __launch_bounds__(kRouteWaves * 64) void route_topk_kernel(const RouteArgs a) {
    // the groups' share: choice values of a wave's token, groups an odd pitch
    // apart so that lanes walking different groups meet in few banks
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
        const uint32_t top = wave_max(ordered(m));
        m = __uint_as_float(top & 0x80000000u ? top & 0x7FFFFFFFu : ~top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = live[i] ? exp((double)x[i] - (double)m) : 0.0;
            sum += p[i];
        }
        const double part = 1.0 / wave_sum(sum);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = live[i] ? p[i] * part : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = live[i] ? 1.0 / (1.0 + exp(-(double)x[i])) : 0.0;
    }
    float c[V];
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        c[i] = (float)p[i] + b[i];
        key[i] = live[i] && c[i] > -__builtin_huge_valf() ? ordered(c[i]) : kNone;
    }

    if (a.n_group > 1) {
        const int per = a.E / a.n_group;
        const int pitch = per | 1;
        float* cl = choice_lds + (size_t)wave * a.n_group * pitch;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            if (e < a.E)
                cl[e / per * pitch + e % per] = key[i] != kNone ? c[i] : -__builtin_huge_valf();
        }
        // one wave, one instruction stream: the writes above precede the
        // reads below in program order and LDS serves a wave in order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // `parts` lanes to a group, each with every parts-th of its experts
        int parts = 1;
        while (parts * 2 * a.n_group <= 64) parts *= 2;
        const int grp = lane / parts;
        float hi = -__builtin_huge_valf(), lo = hi;
        if (grp < a.n_group)
            for (int j = lane % parts; j < per; j += parts) {
                const float v = cl[grp * pitch + j];
                lo = fmaxf(lo, fminf(hi, v));
                hi = fmaxf(hi, v);
            }
        for (int off = 1; off < parts; off *= 2) {
            const float h2 = __shfl_xor(hi, off, 64), l2 = __shfl_xor(lo, off, 64);
            lo = fmaxf(fminf(hi, h2), fmaxf(lo, l2));
            hi = fmaxf(hi, h2);
        }
        // with a selection bias a group's value is the sum of its two best;
        // one that has a single expert left has that one's value
        const float gv = a.bias && lo > -__builtin_huge_valf() ? hi + lo : hi;
        uint32_t g = grp < a.n_group && hi > -__builtin_huge_valf() ? ordered(gv) : kNone;
        uint64_t kept = 0;
        for (int r = 0; r < a.topk_group; ++r) {
            const uint32_t best = wave_max(g);
            if (best == kNone) break;
            const int w = __builtin_ctzll(__ballot(g == best)) / parts;
            kept |= 1ull << w;
            if (grp == w) g = kNone;
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
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) best = max(best, key[i]);
        best = wave_max(best);
        if (best == kNone) break;                // uniform: nothing is left
        int id = 0;
        double wp = 0.0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t at = __ballot(key[i] == best);
            if (at && !found) {
                const int l = __builtin_ctzll(at);
                found = true;
                id = 64 * i + l;
                wp = lane_of(p[i], l);
                if (lane == l) key[i] = kNone;
            }
        }
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
