// Products of bf16 rows with 4-bit weights, grouped by expert with ragged row
// counts or over all tokens of a rank:
//   out = act(f * sum_k x[k] * code(w[n][k]) * s[n][k / group] + bias) + residual
// An E2M1 code has two significant bits and an E4M3 scale four, so a weight,
// code times scale, is exact in bf16 (as is a code times a power of two): the
// weights are made there in registers and multiplied in the bf16 matrix cores,
// with fp32 sums of exact products. f, one factor for a matrix, is applied to
// the sum.
#include "product_tiles.h"

namespace moe_ep {
namespace {

// Eight codes (the first in the lowest bits) times their scale, as bf16.
template <int GROUP>
__device__ __forceinline__ u32x4 widen4(uint32_t c, float s) {
    u32x4 r;
    if constexpr (GROUP == 32) {
        // a power of two: the instruction's own scale
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
    } else {
        auto two = [s](auto v) {
            const float lo = v[0] * s, hi = v[1] * s;
            // exact in bf16: the upper halves
            return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
        };
        r[0] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0));
        r[1] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1));
        r[2] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2));
        r[3] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3));
    }
    return r;
}

// One value of the output from its sum (gated: of gate and up).
template <bool GATED>
__device__ __forceinline__ void finish_value(const W4Args& a, int g, int64_t row, int n, float v,
                                             float up) {
    const MatmulArgs& m = a.m;
    if (a.whole) {
        const float* f = a.whole + g * (GATED ? 2 : 1);
        v *= f[0];
        if (GATED) up *= f[1];
    }
    if (m.bias) {
        const float* b = m.bias + g * m.bias_stride + n;
        v += b[0];
        if (GATED) up += b[m.N];
    }
    v = GATED ? silu_gated(v, up) : apply_act(v, m.act);
    const bool f32 = m.out_dtype == MOE_EP_F32;
    if (m.res) {
        const uint8_t* p = m.res + row * m.res_row;
        v += f32 ? reinterpret_cast<const float*>(p)[n]
                 : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[n] << 16);
    }
    uint8_t* p = m.out + g * m.out_stride + row * m.out_row;
    if (f32) reinterpret_cast<float*>(p)[n] = v;
    else reinterpret_cast<uint16_t*>(p)[n] = (uint16_t)to_bf16_rne(v);
}

// ---------------------------------------------------------------------
// Tiles of 16 rows of x by 16 of w (gated: 8 gate rows and their 8 up rows).
// Four waves share out k in runs of 128 columns, a lane has 32 of them of a row
// of each operand.
// ---------------------------------------------------------------------
constexpr int kPlainWaves = 4;

template <int GROUP, bool GATED>
__global__ __launch_bounds__(kPlainWaves * 64) void w4_kernel(const W4Args a) {
    __shared__ float part[kPlainWaves][kSmall][kSmall + 1];
    const MatmulArgs& m = a.m;
    constexpr int BO = GATED ? kSmall / 2 : kSmall;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, q = lane >> 4;
    const int nt = (m.N + BO - 1) / BO;
    const int H = m.row_bytes / 2;
    const int rows0 = lane_rows(m, 0);
    int n[kKinds];
    count_runs(m, rows0, INT32_MAX, n);
    const int total = n[0] * nt;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const Place at = find_tile(m, rows0, INT32_MAX, 0, nt, t);
        const int mt = cut_rows(at.rows, INT32_MAX).runs;
        const int m0 = at.l % mt * kSmall, n0 = at.l / mt * BO;
        const int col = GATED ? n0 + (r & 7) : n0 + r;
        const int64_t row = GATED && r >= 8 ? (int64_t)m.N + col : col;
        const uint8_t* px = m.x + at.g * m.x_stride + (int64_t)(m0 + r) * m.x_row;
        const uint8_t* pw = m.w + at.g * m.w_stride + row * m.w_row;
        const uint8_t* ps = a.s + at.g * a.s_stride + row * a.s_row;
        const bool has_x = m0 + r < at.rows, has_w = col < m.N;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        for (int k0 = wave * 128; k0 < H; k0 += kPlainWaves * 128) {
            const int k = k0 + q * 32;
            u32x4 c = {0, 0, 0, 0}, x[4] = {};
            float s[2] = {0.f, 0.f};
            if (k < H && has_w) {
                c = *reinterpret_cast<const u32x4*>(pw + k / 2);
                if (GROUP == 16) {
                    s[0] = __builtin_amdgcn_cvt_f32_fp8((int)ps[k / 16], 0);
                    s[1] = __builtin_amdgcn_cvt_f32_fp8((int)ps[k / 16 + 1], 0);
                } else {
                    s[0] = s[1] = __uint_as_float((uint32_t)ps[k / 32] << 23);
                }
            }
            if (k < H && has_x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = *reinterpret_cast<const u32x4*>(px + k * 2 + i * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = mma_bf16(widen4<GROUP>(c[i], s[i / 2]), x[i], acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][r][q * 4 + i] = acc[i];
        __syncthreads();
        for (int i = threadIdx.x; i < kSmall * BO; i += kPlainWaves * 64) {
            const int o = i % BO, mr = i / BO;
            if (m0 + mr >= at.rows || n0 + o >= m.N) continue;
            float v = 0.f, up = 0.f;
            for (int w = 0; w < kPlainWaves; ++w) {
                v += part[w][mr][o];
                if (GATED) up += part[w][mr][o + 8];
            }
            finish_value<GATED>(a, at.g, m0 + mr, n0 + o, v, up);
        }
        __syncthreads();
    }
}

template <int GROUP>
hipError_t launch(const W4Args& a, hipStream_t st) {
    if (a.m.act == MOE_EP_ACT_SILU_GATED)
        w4_kernel<GROUP, true><<<2048, kPlainWaves * 64, 0, st>>>(a);
    else
        w4_kernel<GROUP, false><<<2048, kPlainWaves * 64, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul_w4(const W4Args& a, hipStream_t st) {
    return a.group == 16 ? launch<16>(a, st) : launch<32>(a, st);
}

}  // namespace moe_ep
