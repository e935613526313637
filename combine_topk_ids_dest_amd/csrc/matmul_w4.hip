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

// A scale from its code.
template <int GROUP>
__device__ __forceinline__ float scale_of(uint32_t code) {
    return GROUP == 16 ? __builtin_amdgcn_cvt_f32_fp8((int)code, 0) : __uint_as_float(code << 23);
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
                s[0] = scale_of<GROUP>(ps[k / GROUP]);
                s[1] = scale_of<GROUP>(ps[(k + 16) / GROUP]);
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

// ---------------------------------------------------------------------
// Big tiles: BM (32 to 256) rows of x by 256 rows of w, eight waves, WN of them
// side by side over the rows of w, each with its part of the sums in registers.
// A slab is 64 columns: 128 bytes of a row of x, 32 bytes of codes of a row of
// w. x goes from memory into LDS by slabs, codes by pairs of slabs (a row's 64
// bytes at a time), scales 16 bytes of a row at a time. Waves 0 to 3 load x,
// 4 to 7 codes and scales: a wave's loads complete in order, and x, which comes
// from nearer, would wait for weights that were asked for before it.
//
// Each wave widens the codes of its rows in registers (2 instructions a weight
// with E4M3 scales, half of one with powers of two), so LDS moves a quarter of
// the bytes that bf16 weights would.
//
// LDS: a lane takes 16 consecutive columns of a slab, q = lane / 16: 8 bytes of
// codes, chunks 2 q and 2 q + 1 of x. Row r of x holds chunk c at place
// c ^ place_x(r): 16-byte reads are served lanes 0-3, 12-15, 20-27 first and
// 4-11, 16-19, 28-31 next (then the same of the upper half), and both sets fall
// on all 64 banks. A pair's row of codes holds its chunk c at c ^ (r / 4 & 3).
// ---------------------------------------------------------------------
constexpr int kCols = 256;                       // rows of w of a tile
constexpr int kLds = 160 << 10;
constexpr int kPairCodes = kCols * 64;
constexpr int kScaleSet = kCols * 16;
constexpr int kScaleSets = 4;

template <int BM>
constexpr int kStagesX = BM > 224 ? 2 : BM > 160 ? 3 : 4;
template <int BM>
constexpr int kStagesW = BM == 224 ? 3 : BM > 128 ? 4 : BM == 128 ? 5 : 6;
template <int BM>
constexpr int kAcross = BM > 64 ? 4 : 8;         // waves over the rows of w

__device__ __forceinline__ int place_x(int r) {
    const int j = (r >> 2) & 3;                  // 0, 1, 2, 3 -> 0, 2, 3, 1
    return (r >> 1 & 1) | (j >> 1) << 1 | ((j >> 1) ^ (j & 1)) << 2;
}

template <int GROUP, bool GATED, int BM>
__device__ __forceinline__ void w4_tile(const W4Args& a, int g, int m0, int rows, int n0,
                                        uint8_t* lds) {
    constexpr int WN = kAcross<BM>;
    constexpr int JF = BM * WN / 128;             // fragments of x of a wave
    constexpr int FRAGS = 16 / WN;                // and of w
    constexpr int XS = kStagesX<BM>, WS = kStagesW<BM>;
    constexpr int SLAB_X = BM * kSlab;
    constexpr int FX = BM / 32;                   // loads of a wave per slab of x
    constexpr int AT_W = XS * SLAB_X, AT_S = AT_W + WS * kPairCodes;
    constexpr int SP = GROUP / 8;                 // pairs under 16 bytes of scales
    static_assert(AT_S + kScaleSets * kScaleSet <= kLds, "");
    static_assert((WS + SP - 2) / SP + 1 <= kScaleSets, "");
    const MatmulArgs& m = a.m;
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const bool is_x = wave < 4;
    const int H = m.row_bytes / 2;
    const int nslab = (H + 63) / 64;
    const int left = rows - m0 < BM ? rows - m0 : BM;
    const int nw = GATED ? 2 * m.N : m.N;
    const uint32_t lds0 = uniform((int)(uint32_t)(uintptr_t)(lds_byte*)lds);
    const i32x4 rx = row_rsrc4(m.x + g * m.x_stride + (int64_t)m0 * m.x_row,
                               (int64_t)(left - 1) * m.x_row + m.row_bytes);
    const i32x4 rw = row_rsrc4(m.w + g * m.w_stride, (int64_t)(nw - 1) * m.w_row + H / 2);
    const i32x4 rs = row_rsrc4(a.s + g * a.s_stride,
                               (int64_t)(nw - 1) * a.s_row + (H / GROUP + 15) / 16 * 16);

    // Load i of x fills rows (i * 4 + wave) * 8 .. + 7, of codes rows
    // (i * 4 + wave - 4) * 16 .. + 15 of the tile: one offset, and how many of
    // the loads have a row.
    uint32_t at, at_s = kOutside;
    int have, chunk;
    if (is_x) {
        const int r = wave * 8 + (lane >> 3);
        chunk = ((lane & 7) ^ place_x(r)) * 16;
        at = (uint32_t)r * (uint32_t)m.x_row + chunk;
        have = left > r ? (left - r + 31) / 32 : 0;
    } else {
        constexpr int STEP = GATED ? 32 : 64;
        const int r = (wave - 4) * 16 + (lane >> 2);
        int n;
        const int row = wrow<GATED, FRAGS>(r, n0, m.N, n);
        chunk = ((lane & 3) ^ ((r >> 2) & 3)) * 16;
        at = (uint32_t)row * (uint32_t)m.w_row + chunk;
        have = m.N > n ? (m.N - n + STEP - 1) / STEP : 0;
        const int srow = wrow<GATED, FRAGS>((wave - 4) * 64 + lane, n0, m.N, n);
        if (n < m.N) at_s = (uint32_t)srow * (uint32_t)a.s_row;
    }
    const uint32_t step = is_x ? 32u * (uint32_t)m.x_row
                               : (GATED ? 32u : 64u) * (uint32_t)m.w_row;
    auto fetch_x = [&](int s, int stage) {
        const bool in = s * kSlab + chunk < m.row_bytes;
        const uint32_t k = s < nslab ? s * kSlab : 0;
#pragma unroll
        for (int i = 0; i < FX; ++i)
            load_to_lds(rx, lds0 + stage * SLAB_X + (i * 4 + wave) * 1024,
                        in && i < have ? at + i * step : kOutside, k);
    };
    auto fetch_w = [&](int p, int stage) {
        const bool any = 2 * p < nslab;
        if (p % SP == 0)
            load_to_lds(rs, lds0 + AT_S + (p / SP) % kScaleSets * kScaleSet + (wave - 4) * 1024,
                        any ? at_s : kOutside, any ? p / SP * 16 : 0);
        const bool in = p * 64 + chunk < H / 2;
        const uint32_t k = any ? p * 64 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load_to_lds(rw, lds0 + AT_W + stage * kPairCodes + (i * 4 + wave - 4) * 1024,
                        in && i < have ? at + i * step : kOutside, k);
    };

    const int r = lane & 15, q = lane >> 4;
    const int rdx = (wm * (JF * 16) + r) * kSlab + ((2 * q) ^ place_x(r)) * 16;
    const int rdw = AT_W + (wn * (FRAGS * 16) + r) * 64 + (q & 1) * 8;
    const int swap = (r >> 2) & 3;
    const int rds = AT_S + (wn * (FRAGS * 16) + r) * 16 + (GROUP == 16 ? q : q >> 1);
    f32x4 acc[FRAGS][JF];
#pragma unroll
    for (int i = 0; i < FRAGS; ++i)
#pragma unroll
        for (int j = 0; j < JF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (is_x) {
#pragma unroll
        for (int v = 0; v < XS - 1; ++v) fetch_x(v, v);
    } else {
#pragma unroll
        for (int p = 0; p < WS - 1; ++p) fetch_w(p, p);
    }
    int ix = 0, iw = 0;                           // stages of slab s and of its pair
    for (int s = 0; s < nslab; ++s) {
        const int p = s >> 1;
        // Slab s (and its pair, with the scales asked for before it) has
        // arrived, slab s - 1 is read. Behind them are the loads of XS - 2
        // slabs, of WS - 2 pairs and now and then of scales.
        if (is_x) wait_and_barrier<(XS - 2) * FX>();
        else wait_and_barrier<(WS - 2) * 4>();
        if (is_x) fetch_x(s + XS - 1, ix == 0 ? XS - 1 : ix - 1);
        else if (!(s & 1)) fetch_w(p + WS - 1, iw == 0 ? WS - 1 : iw - 1);
        const uint8_t* px = lds + ix * SLAB_X;
        const uint8_t* pw = lds + iw * kPairCodes + ((((s & 1) * 2 + (q >> 1)) ^ swap) * 16);
        const uint8_t* ps = lds + (p / SP) % kScaleSets * kScaleSet + p % SP * (16 / SP) +
                            (s & 1) * (8 / SP);
        const bool in = s * 64 + q * 16 < H;      // what follows the last scale may be anything
        u32x2 c[FRAGS];
        uint32_t sc[FRAGS];
#pragma unroll
        for (int i = 0; i < FRAGS; ++i) {
            c[i] = *reinterpret_cast<const u32x2*>(pw + rdw + i * 16 * 64);
            sc[i] = ps[rds + i * 16 * 16];
        }
        u32x4 w[FRAGS][2];
#pragma unroll
        for (int i = 0; i < FRAGS; ++i) {
            const float f = in ? scale_of<GROUP>(sc[i]) : 0.f;
            w[i][0] = widen4<GROUP>(c[i][0], f);
            w[i][1] = widen4<GROUP>(c[i][1], f);
        }
#pragma unroll
        for (int j = 0; j < JF; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 x =
                    *reinterpret_cast<const u32x4*>(px + (rdx ^ (h * 16)) + j * 16 * kSlab);
#pragma unroll
                for (int i = 0; i < FRAGS; ++i) acc[i][j] = mma_bf16(w[i][h], x, acc[i][j]);
            }
        ix = ix + 1 < XS ? ix + 1 : 0;
        if (s & 1) iw = iw + 1 < WS ? iw + 1 : 0;
    }
    wait_and_barrier<0>();   // LDS is free for the next tile
    if (a.whole) {
        const float* f = a.whole + g * (GATED ? 2 : 1);
#pragma unroll
        for (int i = 0; i < FRAGS; ++i)
#pragma unroll
            for (int j = 0; j < JF; ++j) acc[i][j] *= f[GATED ? i & 1 : 0];
    }
    finish_tile<2, GATED, FRAGS, JF, WN>(m, g, m0, left, n0, acc, lds);
}

template <int GROUP, bool GATED>
__global__ __launch_bounds__(kThreads, 2) void w4_big_kernel(const W4Args a) {
    __shared__ __align__(1024) uint8_t lds[kLds];
    const MatmulArgs& m = a.m;
    constexpr int BB = GATED ? kCols / 2 : kCols;
    const int ntb = (m.N + BB - 1) / BB;
    const int rows0 = lane_rows(m, 0);
    int n[kKinds], total = 0;
    count_runs(m, rows0, 0, n);
#pragma unroll
    for (int k = 1; k < kKinds; ++k) {
        n[k] *= ntb;
        total += n[k];
    }
    const int parts = last_parts(total);
    for (int t0 = 0; t0 < total; t0 += kGrid) {
        const Turn turn = turn_of(blockIdx.x, t0, total, parts);
        if (turn.t < 0) break;
        int t = turn.t;
        int kind = kKinds - 1;
#pragma unroll
        for (int k = kKinds - 1; k > 1; --k)
            if (kind == k && t >= n[k]) {
                t -= n[k];
                --kind;
            }
        const Place at = find_tile(m, rows0, 0, kind, ntb, t);
        const int runs = cut_rows(at.rows, 0).runs;
        const Piece p = piece_of(at.l, at.rows, runs, kind, ntb, turn.sub, turn.cut);
        if (p.m0 >= p.end) continue;
        const int n0 = p.col * BB;
        auto run = [&](auto bm) {
            w4_tile<GROUP, GATED, decltype(bm)::value>(a, at.g, p.m0, p.end, n0, lds);
        };
        const int f = p.fragments;
        if (f == 8) run(std::integral_constant<int, 256>{});
        else if (f == 7) run(std::integral_constant<int, 224>{});
        else if (f == 6) run(std::integral_constant<int, 192>{});
        else if (f == 5) run(std::integral_constant<int, 160>{});
        else if (f > 2) run(std::integral_constant<int, 128>{});
        else if (f == 2) run(std::integral_constant<int, 64>{});
        else run(std::integral_constant<int, 32>{});
    }
}

template <int GROUP, bool GATED>
hipError_t launch(const W4Args& a, hipStream_t st) {
    if (a.m.rows <= kSmall)
        w4_kernel<GROUP, GATED><<<2048, kPlainWaves * 64, 0, st>>>(a);
    else
        w4_big_kernel<GROUP, GATED><<<kGrid, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul_w4(const W4Args& a, hipStream_t st) {
    const bool gated = a.m.act == MOE_EP_ACT_SILU_GATED;
    if (a.group == 16) return gated ? launch<16, true>(a, st) : launch<16, false>(a, st);
    return gated ? launch<32, true>(a, st) : launch<32, false>(a, st);
}

}  // namespace moe_ep
