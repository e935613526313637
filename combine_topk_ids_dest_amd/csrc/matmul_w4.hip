// Products of bf16 rows with 4-bit weights, grouped by expert with ragged row
// counts or over all tokens of a rank:
//   out = act(f * sum_k x[k] * code(w[n][k]) * s[n][k / group] + bias) + residual
// An E2M1 code has two significant bits and an E4M3 scale four, so a weight,
// code times scale, is exact in bf16 (as is a code times a power of two): the
// weights are made there in registers and multiplied in the bf16 matrix cores,
// with fp32 sums of exact products. f, one factor for a matrix, is applied to
// the sum. 32 experts of 15575 rows, 7168 -> 2 x 2048, E4M3: 917 us one after the
// other, 979 (919 to 1129) each by itself; 8 of 917 rows 82; 25 of one or two rows 88
// (4.7 TB/s); one token 9 (with 2048 -> 7168 and powers of two, 917 rows: 45 and 47).
#include "product_tiles.h"

namespace moe_ep {
namespace {

// Four codes, the low (HALF 0) or high ones of c, times their scale, as bf16.
template <int GROUP, int HALF>
__device__ __forceinline__ u32x2 widen_half(uint32_t c, float s) {
    if constexpr (GROUP == 32) {
        // a power of two: the instruction's own scale
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                                                      c, s, 2 * HALF)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                                                      c, s, 2 * HALF + 1))};
    } else {
        auto two = [s](auto v) {
            const float lo = v[0] * s, hi = v[1] * s;
            // exact in bf16: the upper halves
            return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
        };
        return u32x2{two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2 * HALF)),
                     two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2 * HALF + 1))};
    }
}

// Eight codes, the first in the lowest bits.
template <int GROUP>
__device__ __forceinline__ u32x4 widen4(uint32_t c, float s) {
    const u32x2 lo = widen_half<GROUP, 0>(c, s), hi = widen_half<GROUP, 1>(c, s);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// The lane, made anew for each tile: what is derived from it would otherwise be
// held in registers over all kinds of tiles, spilled, and loaded back in their
// loops, each time behind all loads in flight.
__device__ __forceinline__ int tile_lane() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
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
// Tiles of a few rows: up to 16 of x by 16 WN of w (gated: half gate rows, half
// up rows). Bound by the weights' bytes, so what counts is loads in flight. A
// wave has 16 rows of w and every WK-th block of 256 columns (WN WK = 8 waves:
// few rows of w leave CUs idle, so there the waves share out k and their sums
// are added through LDS, in wave order). Codes and scales go straight from
// memory into LDS of the wave's own, four steps of 256 columns always on their
// way, with no barrier between them; behind the last step of a tile come the
// first of the block's next tile.
//
// x is read by all waves: segments of 32 KB (2 to 16 rows of 8192 to 1024
// columns), the next one on its way while one is in use, a barrier between them.
//
// LDS: a wave's 128-byte row of codes holds chunk c at c ^ (r / 2 & 7), a
// 512-byte row of x chunk c at c ^ place_few(r): a lane takes chunks q and q + 4
// of the codes (q = lane / 16), so chunks 4 q + t and 16 + 4 q + t of x, and the
// sets of 16 lanes that a 16-byte read is served in (see the big tiles) meet on
// no bank.
// ---------------------------------------------------------------------
constexpr int kFewCols = 256;                    // columns of a step of a wave
constexpr int kFewStep = kSmall * kFewCols / 2 + 256;    // codes and scales of one
constexpr int kFewRing = 4;
constexpr int kSegment = 32 << 10;
constexpr int kFewX = kWaves * kFewRing * kFewStep;      // segments behind the rings,
constexpr int kFewPart = kFewX + 2 * kSegment;           // the waves' sums, twice
constexpr int kFewPitch = kSmall + 4;
constexpr int kFewSums = kWaves * kSmall * kFewPitch * 4;
constexpr int kFewZero = kFewPart + 2 * kFewSums;        // 512 bytes of zeros
constexpr int kFewLds = kFewZero + 512;
constexpr float kCodeUnit = 0x1p-7f;             // what a bare code of 1 is taken as
static_assert(kFewLds <= 160 << 10, "");

__device__ __forceinline__ int place_few(int r) {
    const int j = (r >> 2) & 3;                  // 0, 1, 2, 3 -> 0, 2, 3, 1
    return (r & 3) | (j >> 1) << 2 | ((j >> 1) ^ (j & 1)) << 3;
}

// What a wave needs to load a tile.
struct FewTile {
    i32x4 rx, rw, rs;
    uint32_t vw[2], vs;
    int g, m0, left, n0;
    int lx;                                      // x in 2^lx rows
    int lk, wk, nsteps;                          // 2^lk waves share out k, this one the wk-th
};

template <int GROUP, bool GATED>
__device__ __forceinline__ FewTile few_setup(const W4Args& a, int g, int m0, int rows, int n0,
                                             int lw) {
    const MatmulArgs& m = a.m;
    constexpr int BO = GATED ? kSmall / 2 : kSmall;
    const int lane = tile_lane();
    const int H = m.row_bytes / 2;
    const int nw = GATED ? 2 * m.N : m.N;
    const int wave = uniform(threadIdx.x >> 6), wn = wave & ((1 << lw) - 1);
    FewTile t;
    t.lk = 3 - lw;
    t.wk = wave >> lw;
    const int steps = (H + (kFewCols << t.lk) - 1) >> (8 + t.lk);
    t.nsteps = steps > kFewRing ? steps : kFewRing;
    t.g = g;
    t.m0 = m0;
    t.left = rows - m0 < kSmall ? rows - m0 : kSmall;
    t.n0 = n0;
    t.lx = t.left > 8 ? 4 : t.left > 4 ? 3 : t.left > 2 ? 2 : 1;
    t.rx = row_rsrc4(m.x + g * m.x_stride + (int64_t)m0 * m.x_row,
                     (int64_t)(t.left - 1) * m.x_row + m.row_bytes);
    t.rw = row_rsrc4(m.w + g * m.w_stride, (int64_t)(nw - 1) * m.w_row + H / 2);
    t.rs = row_rsrc4(a.s + g * a.s_stride,
                     (int64_t)(nw - 1) * a.s_row + (H / GROUP + 15) / 16 * 16);
    auto row = [&](int r, bool& in) {
        const int n = n0 + wn * BO + (GATED ? r & 7 : r);
        in = n < m.N;
        return GATED && r >= 8 ? (uint32_t)(m.N + n) : (uint32_t)n;
    };
    bool in;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = h * 8 + (lane >> 3);
        const uint32_t at = row(r, in) * (uint32_t)m.w_row;
        t.vw[h] = in ? at + ((lane & 7) ^ ((r >> 1) & 7)) * 16 : kOutside;
    }
    // E4M3: 16 bytes of a row to a lane; powers of two: 4 of 8
    const uint32_t at = row(GROUP == 16 ? lane & 15 : (lane >> 1) & 15, in) * (uint32_t)a.s_row;
    t.vs = in ? at + (GROUP == 16 ? 0 : (lane & 1) * 4) : kOutside;
    return t;
}

// Works through the block's tiles, number t of `total` at place(t): up to 16 rows
// each by WN = 8 / WK runs of 16 rows of w.
template <int GROUP, bool GATED, class Next>
__device__ __forceinline__ void few_tiles(const W4Args& a, uint8_t* lds, int total,
                                          const Next& place) {
    const MatmulArgs& m = a.m;
    const int lane = tile_lane();
    const int wave = uniform(threadIdx.x >> 6);
    const int H = m.row_bytes / 2;
    const uint32_t lds0 = uniform((int)(uint32_t)(uintptr_t)(lds_byte*)lds);
    const uint32_t ring = lds0 + wave * kFewRing * kFewStep;
    const uint8_t* mine = lds + wave * kFewRing * kFewStep;
    const int r = lane & 15, q = lane >> 4;

    auto tile_at = [&](int t0) {
        const int t = t0 < total ? tile_of(blockIdx.x, gridDim.x, total - t0) : -1;
        return t < 0 ? -1 : t + t0;
    };
    // Step i of a tile into place j of the wave's ring.
    auto fetch = [&](const FewTile& t, int i, int j) {
        const int k = ((i << t.lk) + t.wk) * kFewCols;
        const bool any = k < H;
        const uint32_t at = ring + j * kFewStep;
        if (lane < (GROUP == 16 ? 16 : 32)) {
            if (GROUP == 16)
                load_to_lds(uniform(t.rs), at + 2048, any ? t.vs : kOutside, any ? k / 16 : 0);
            else
                load4_to_lds(uniform(t.rs), at + 2048, any ? t.vs : kOutside, any ? k / 32 : 0);
        }
        // (codes behind a row's end meet x's zeros and a scale of zero)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            load_to_lds(uniform(t.rw), at + h * 1024, any ? t.vw[h] : kOutside, any ? k / 2 : 0);
    };
    // Segment n of a tile's x into buffer `to`: two rows of 256 columns a load
    // (none for rows and columns that no wave reads).
    auto fetch_x = [&](const FewTile& t, int n, int to) {
        const int pairs = t.lx - 1;              // 2^pairs pairs of rows
#pragma unroll 1
        for (int i = 0; i < kSegment / 1024 / kWaves; ++i) {
            const int load = i * kWaves + wave;
            const int k0 = (n << (14 - t.lx)) + (load >> pairs) * kFewCols;
            const int row0 = (load & ((1 << pairs) - 1)) * 2;
            if (k0 >= H || row0 >= t.left) continue;
            const int row = row0 + (lane >> 5);
            const int k = k0 + ((lane & 31) ^ place_few(row)) * 8;
            load_to_lds(uniform(t.rx), lds0 + kFewX + to * kSegment + load * 1024,
                        row < t.left && k < H ? (uint32_t)row * (uint32_t)m.x_row + k * 2 : kOutside,
                        0);
        }
    };
    auto finish = [&](const FewTile& t, int odd) {
        constexpr int BO = GATED ? kSmall / 2 : kSmall;
        const float* part = reinterpret_cast<const float*>(lds + kFewPart + odd * kFewSums);
        const int lw = 3 - t.lk, wide = BO << lw;
        for (int i = threadIdx.x; i < wide * t.left; i += kThreads) {
            const int o = i & (wide - 1), row = i / wide;
            const int n = t.n0 + o;
            if (n >= m.N) continue;
            float v = 0.f, up = 0.f;
            for (int w = o / BO; w < kWaves; w += 1 << lw) {
                const float* p = part + (w * kSmall + row) * kFewPitch + o % BO;
                v += p[0];
                if (GATED) up += p[8];
            }
            finish_value<GATED>(a, t.g, t.m0 + row, n, v, up);
        }
    };

    int t0 = 0, at = tile_at(0);
    if (at < 0) return;
    // (read behind the first segment's barrier)
    if (threadIdx.x < 128) reinterpret_cast<uint32_t*>(lds + kFewZero)[threadIdx.x] = 0;
    FewTile cur = place(at);
    // (rolled: at the start every line of code is a miss)
    fetch_x(cur, 0, 0);
#pragma unroll 1
    for (int j = 0; j < kFewRing; ++j) fetch(cur, j, j);
    FewTile old = cur;
    bool owed = false;                           // old's sums are still to be added up
    int odd = 0, to = 0, j = 0;
    int since = kFewRing;                        // steps asked for behind the next segment
    for (;;) {
        t0 += gridDim.x;
        at = tile_at(t0);
        FewTile nxt = cur;
        if (at >= 0) nxt = place(at);
        const int lk = cur.lk, wk = cur.wk, nsteps = cur.nsteps;
        const int lseg = 14 - cur.lx - 8 - lk;   // 2^lseg steps of a segment
        f32x4 acc = {0.f, 0.f, 0.f, 0.f}, acc2 = acc;
        // The steps of the tile. Up to four rows with E4M3 scales (SPLIT): products
        // of bare codes, each group's apart. x is the first operand, its row
        // 4 g + i row g of x in the columns of lane quarter i and zero in the
        // others, so that sum 4 g + i of a row of w is over one group of columns;
        // it is scaled and added. That takes an instruction a weight, weights
        // widened with their scales two. Codes are taken times 2^-7 and the scales
        // times 2^7: 16 products of a bare code, up to 6, with the largest bf16
        // would be past fp32's range where those of the weights are not.
        auto all_steps = [&](auto split) {
            constexpr bool SPLIT = decltype(split)::value;
            const int row = SPLIT ? r >> 2 : r & ((1 << cur.lx) - 1);
            const bool has = !SPLIT || (q == (r & 3) && row < cur.left);
            const uint32_t real = has ? ~0u : 0u;
            uint32_t from[4];                    // where the lane reads x, chunks 4 q + t
#pragma unroll
            for (int t = 0; t < 4; ++t)
                from[t] = has ? row * 512 + ((q * 4 + t) ^ place_few(row)) * 16
                              : kFewZero - kFewX;
            for (int i = 0; i < nsteps; ++i) {
                const int in_segment = i & ((1 << lseg) - 1);
                if (in_segment == 0) {
                    // the segment at hand has arrived: behind it are `since`
                    // steps of three loads
                    if (since >= 4) wait_and_barrier<3 * 4>();
                    else if (since >= 2) wait_and_barrier<3 * 2>();
                    else if (since == 1) wait_and_barrier<3>();
                    else wait_and_barrier<0>();
                    since = 0;
                    const int n = (i >> lseg) + 1;   // the next
                    if (n << lseg < nsteps) fetch_x(cur, n, to ^ 1);
                    else if (at >= 0) fetch_x(nxt, 0, to ^ 1);
                    if (owed) finish(old, odd ^ 1);
                    owed = false;
                    to ^= 1;
                }
                // the oldest step has arrived: behind it are three steps, or what
                // is left of the last tile
                const int behind = at >= 0 ? kFewRing - 1 : nsteps - 1 - i;
                static_assert(kFewRing == 4, "");
                if (behind >= 3) asm volatile("s_waitcnt vmcnt(9)" ::: "memory");
                else if (behind == 2) asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
                else if (behind == 1) asm volatile("s_waitcnt vmcnt(3)" ::: "memory");
                else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                const uint8_t* p = mine + j * kFewStep;
                const int k = ((i << lk) + wk) * kFewCols;
                u32x4 c[2], x[8];
                uint32_t sc[4];
                if (k < H) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        c[h] = *reinterpret_cast<const u32x4*>(p + r * 128 +
                                                               (((q + 4 * h) ^ (r >> 1)) & 7) * 16);
                        const uint8_t* ps = p + 2048 + r * (256 / GROUP) + h * (128 / GROUP);
                        if (SPLIT) {
                            const u32x2 v = *reinterpret_cast<const u32x2*>(ps);
                            sc[2 * h] = v[0];
                            sc[2 * h + 1] = v[1];
                        } else {
                            sc[2 * h] = GROUP == 32 ? ps[q]
                                                    : *reinterpret_cast<const uint16_t*>(ps + q * 2);
                        }
                    }
                    const uint32_t at_x = (uint32_t)((to ^ 1) * kSegment) +
                                          ((uint32_t)((in_segment << lk) + wk) << (9 + cur.lx));
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        x[t] = *reinterpret_cast<const u32x4*>(lds + kFewX + from[t & 3] +
                                                               (at_x & real) + (t >> 2) * 256);
                }
                // all of them on their way before the first is waited for; read, so
                // the codes' place can be filled again
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
                if (i + kFewRing < nsteps) {
                    fetch(cur, i + kFewRing, j);
                    ++since;
                } else if (at >= 0) {
                    fetch(nxt, i + kFewRing - nsteps, j);
                    ++since;
                }
                j = j + 1 < kFewRing ? j + 1 : 0;
                if (k >= H) continue;
                // what follows the last scale may be anything
                if constexpr (SPLIT) {
                    f32x4 d[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                        d[b] = mma_bf16(x[2 * b], widen4<32>(c[b >> 1][2 * b & 3], kCodeUnit), zero);
                    }
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        d[b] = mma_bf16(x[2 * b + 1],
                                        widen4<32>(c[b >> 1][(2 * b & 3) + 1], kCodeUnit), d[b]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int n = (H - k - h * 128) / 16;
                        const uint64_t mask = n >= 8 ? ~0ull : n > 0 ? (1ull << (8 * n)) - 1 : 0;
                        sc[2 * h] &= (uint32_t)mask;
                        sc[2 * h + 1] &= (uint32_t)(mask >> 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int v = (int)sc[2 * h + (e >> 1)];
                            // group 2 e + b of the half: byte 2 (e & 1) + b
                            const float f0 =
                                e & 1 ? __builtin_amdgcn_cvt_scalef32_f32_fp8(v, 1 / kCodeUnit, 2)
                                      : __builtin_amdgcn_cvt_scalef32_f32_fp8(v, 1 / kCodeUnit, 0);
                            const float f1 =
                                e & 1 ? __builtin_amdgcn_cvt_scalef32_f32_fp8(v, 1 / kCodeUnit, 3)
                                      : __builtin_amdgcn_cvt_scalef32_f32_fp8(v, 1 / kCodeUnit, 1);
                            acc[e] = __builtin_fmaf(d[2 * h][e], f0, acc[e]);
                            acc2[e] = __builtin_fmaf(d[2 * h + 1][e], f1, acc2[e]);
                        }
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool in = k + h * 128 + q * 32 < H;
                        const uint32_t v = in ? sc[2 * h] : 0;
                        const float s0 = GROUP == 16 ? __builtin_amdgcn_cvt_f32_fp8((int)v, 0)
                                                     : __uint_as_float(v << 23);
                        const float s1 = GROUP == 16 ? __builtin_amdgcn_cvt_f32_fp8((int)v, 1) : s0;
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const u32x4 w = widen4<GROUP>(c[h][t], t < 2 ? s0 : s1);
                            if (t & 1) acc2 = mma_bf16(w, x[4 * h + t], acc2);
                            else acc = mma_bf16(w, x[4 * h + t], acc);
                        }
                    }
                }
            }
        };
        const bool split = GROUP == 16 && cur.left <= 4;
        if constexpr (GROUP == 16) {
            if (split) all_steps(std::true_type{});
            else all_steps(std::false_type{});
        } else {
            all_steps(std::false_type{});
        }
        float* part = reinterpret_cast<float*>(lds + kFewPart + odd * kFewSums);
        acc += acc2;
        if (split) part[(wave * kSmall + q) * kFewPitch + r] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        else *reinterpret_cast<f32x4*>(part + (wave * kSmall + r) * kFewPitch + q * 4) = acc;
        old = cur;
        owed = true;
        odd ^= 1;
        if (at < 0) break;
        cur = nxt;
    }
    wait_and_barrier<0>();
    finish(old, odd ^ 1);
}

template <int GROUP, bool GATED>
__device__ __forceinline__ void few_rows(const W4Args& a, uint8_t* lds, int rows0, int small_to,
                                         int runs) {
    const MatmulArgs& m = a.m;
    constexpr int BO = GATED ? kSmall / 2 : kSmall;
    FewCut cut = a.cut;                          // over all tokens the host's
    if (m.counts) {
        bool wide = false;
        for (int g0 = 0; g0 < m.groups; g0 += 64) {
            const int rows = g0 ? lane_rows(m, g0) : rows0;
            wide |= __ballot(rows <= small_to && rows > 8) != 0;
        }
        cut = few_cut(runs, m.N, m.row_bytes / 2, BO, wide ? 1 : 0);
    }
    // the first 64 groups' runs, added up: where a tile is without a scan of its own
    int runs0 = 0, upto = 0, covered = 0;
    if (m.counts) {
        runs0 = runs_of(rows0, small_to, 0);
        upto = wave_inclusive_scan(runs0);
        covered = __builtin_amdgcn_readlane(upto, 63);
    }
    few_tiles<GROUP, GATED>(a, lds, cut.total, [&](int t) {
        int lw = cut.lw, n0 = 0;
        if (t >= cut.whole) {
            const int split = cut.lw - cut.last, u = t - cut.whole;
            lw = cut.last;
            n0 = (u & ((1 << split) - 1)) * (BO << lw);
            t = cut.whole + (u >> split);
        }
        Place at;
        if (!m.counts) {
            at = Place{0, m.rows, t};
        } else if (t < covered * cut.nt) {
            const int l = __builtin_ctzll(__ballot(upto * cut.nt > t));
            const int mine = __builtin_amdgcn_readlane(runs0, l);
            at.g = l;
            at.rows = __builtin_amdgcn_readlane(rows0, l);
            at.l = t - (__builtin_amdgcn_readlane(upto, l) - mine) * cut.nt;
        } else {
            at = find_tile(m, rows0, small_to, 0, cut.nt, t);
        }
        const int mt = (at.rows + kSmall - 1) / kSmall;
        const int col = mt == 1 ? at.l : at.l / mt;
        return few_setup<GROUP, GATED>(a, at.g, (at.l - col * mt) * kSmall, at.rows,
                                       col * (BO << cut.lw) + n0, lw);
    });
}

// ---------------------------------------------------------------------
// Big tiles: BM (160 to 256) rows of x by 256 rows of w. Eight waves in two rows of
// four, each with BM / 2 x 64 of the sums in registers.
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
constexpr int kStagesW = BM == 224 ? 3 : 4;

__device__ __forceinline__ int place_x(int r) {
    const int j = (r >> 2) & 3;                  // 0, 1, 2, 3 -> 0, 2, 3, 1
    return (r >> 1 & 1) | (j >> 1) << 1 | ((j >> 1) ^ (j & 1)) << 2;
}

template <int GROUP, bool GATED, int BM>
__device__ __forceinline__ void w4_tile(const W4Args& a, int g, int m0, int rows, int n0,
                                        uint8_t* lds) {
    constexpr int WN = 4;
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
    const int lane = tile_lane();
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

    // Products go half a slab at a time (8 of a lane's 16 columns), and under each
    // half's products the next half's fragments of x are read and its weights
    // widened. The wait in the middle of slab s is for slab s + 1.
    u32x4 fx[2][JF], fw[2][FRAGS];
    u32x2 c[FRAGS];                              // of the slab whose half 1 is to come
    float f[FRAGS];
    auto read_codes = [&](int s, int stage) {
        const uint8_t* pw = lds + rdw + stage * kPairCodes + ((((s & 1) * 2 + (q >> 1)) ^ swap) * 16);
        const uint8_t* ps = lds + rds + ((s >> 1) / SP) % kScaleSets * kScaleSet +
                            (s >> 1) % SP * (16 / SP) + (s & 1) * (8 / SP);
        const bool in = s * 64 + q * 16 < H;     // what follows the last scale may be anything
#pragma unroll
        for (int i = 0; i < FRAGS; ++i) {
            c[i] = *reinterpret_cast<const u32x2*>(pw + i * 16 * 64);
            const uint32_t code = ps[i * 16 * 16];
            f[i] = in ? scale_of<GROUP>(code) : 0.f;
        }
    };
    // Part n of 2 FRAGS of a half's widening.
    auto widen_part = [&](auto half, int n) {
        constexpr int h = decltype(half)::value;
        const int i = n >> 1;
        const u32x2 v = n & 1 ? widen_half<GROUP, 1>(c[i][h], f[i]) : widen_half<GROUP, 0>(c[i][h], f[i]);
        fw[h][i][(n & 1) * 2] = v[0];
        fw[h][i][(n & 1) * 2 + 1] = v[1];
    };
    // Multiplies half `now` while reading and widening the other one (of x at px).
    auto multiply = [&](auto now, const uint8_t* px) {
        constexpr int h = decltype(now)::value, o = 1 - h;
#pragma unroll
        for (int j = 0; j < JF; ++j) {
#pragma unroll
            for (int i = 0; i < FRAGS; ++i) acc[i][j] = mma_bf16(fw[h][i], fx[h][j], acc[i][j]);
            fx[o][j] = *reinterpret_cast<const u32x4*>(px + (rdx ^ (o * 16)) + j * 16 * kSlab);
#pragma unroll
            for (int n = j * 2 * FRAGS / JF; n < (j + 1) * 2 * FRAGS / JF; ++n)
                widen_part(std::integral_constant<int, o>{}, n);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (is_x) {
#pragma unroll
        for (int v = 0; v < XS; ++v) fetch_x(v, v);
        wait_and_barrier<(XS - 1) * FX>();
    } else {
#pragma unroll
        for (int p = 0; p < WS; ++p) fetch_w(p, p);
        wait_and_barrier<(WS - 1) * 4>();
    }
    read_codes(0, 0);
#pragma unroll
    for (int j = 0; j < JF; ++j)
        fx[0][j] = *reinterpret_cast<const u32x4*>(lds + rdx + j * 16 * kSlab);
#pragma unroll
    for (int n = 0; n < 2 * FRAGS; ++n) widen_part(std::integral_constant<int, 0>{}, n);
    int ix = 0, iw = 0;                           // stages of slab s and of its pair
    for (int s = 0; s < nslab; ++s) {
        multiply(std::integral_constant<int, 0>{}, lds + ix * SLAB_X);
        // Slab s is read; slab s + 1 (and its pair, with the scales asked for
        // before it) has arrived. Behind them are the loads of XS - 2 slabs, of
        // WS - 2 pairs and now and then of scales.
        if (is_x) wait_and_barrier<(XS - 2) * FX>();
        else wait_and_barrier<(WS - 2) * 4>();
        const int nix = ix + 1 < XS ? ix + 1 : 0, niw = iw + 1 < WS ? iw + 1 : 0;
        read_codes(s + 1, s & 1 ? niw : iw);
        if (is_x) fetch_x(s + XS, ix);
        else if (s & 1) fetch_w((s >> 1) + WS, iw);
        multiply(std::integral_constant<int, 1>{}, lds + nix * SLAB_X);
        ix = nix;
        if (s & 1) iw = niw;
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

// ---------------------------------------------------------------------
// Middle tiles: BM = 32, 64 or 128 rows of x by 256 of w, where a slab's products
// are over before LDS has answered. They go by pairs of slabs, one barrier each:
// a lane has 32 consecutive columns of a pair, 16 bytes of codes and four chunks
// of x, in two units of 16 columns (one E4M3 scale); under a unit's products the
// next unit's x is on its way into registers, and behind the barrier the next
// pair's codes. Bound by the weights' bytes as much as by widening them, so codes
// come by quads of slabs, 128 bytes of a row at a time (with 64 the loads alone
// of 8 experts of 115 rows, 7168 -> 2 x 2048, took 59 us, so 52).
//
// LDS: a 256-byte row of x holds chunk c at c ^ place_few(r), a 128-byte row of
// codes at c ^ (r / 2 & 7); the sets of 16 lanes of a 16-byte read (see the big
// tiles) meet on no bank.
// ---------------------------------------------------------------------
constexpr int kQuad = kCols * 128;               // codes of a quad
template <int BM>
constexpr int kMidX = BM == 128 ? 2 : 3;         // pairs of x in LDS
template <int BM>
constexpr int kMidW = BM == 128 ? 2 : 3;         // and quads of codes

template <int GROUP, bool GATED, int BM, int WN>
__device__ __forceinline__ void w4_mid_tile(const W4Args& a, int g, int m0, int rows, int n0,
                                            uint8_t* lds) {
    constexpr int JF = BM * WN / 128;             // fragments of x of a wave
    constexpr int FRAGS = 16 / WN;                // and of w
    constexpr int XS = kMidX<BM>, WS = kMidW<BM>;
    constexpr int PAIR_X = BM * 256;
    constexpr int FX = BM / 16;                   // loads of a wave per pair of x
    constexpr int FW = 9;                         // and per quad of codes and scales
    constexpr int AT_W = XS * PAIR_X, AT_S = AT_W + WS * kQuad;
    static_assert(AT_S + WS * kScaleSet <= kLds, "");
    const MatmulArgs& m = a.m;
    const int lane = tile_lane();
    const int wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const bool is_x = wave < 4;
    const int H = m.row_bytes / 2;
    const int npair = (H + 127) / 128;
    const int left = rows - m0 < BM ? rows - m0 : BM;
    const int nw = GATED ? 2 * m.N : m.N;
    const uint32_t lds0 = uniform((int)(uint32_t)(uintptr_t)(lds_byte*)lds);
    const i32x4 rx = row_rsrc4(m.x + g * m.x_stride + (int64_t)m0 * m.x_row,
                               (int64_t)(left - 1) * m.x_row + m.row_bytes);
    const i32x4 rw = row_rsrc4(m.w + g * m.w_stride, (int64_t)(nw - 1) * m.w_row + H / 2);
    const i32x4 rs = row_rsrc4(a.s + g * a.s_stride,
                               (int64_t)(nw - 1) * a.s_row + (H / GROUP + 15) / 16 * 16);

    // Load i of x fills rows (i * 4 + wave) * 4 .. + 3, of codes rows
    // (i * 4 + wave - 4) * 8 .. + 7 of the tile.
    const int row = is_x ? wave * 4 + (lane >> 4) : (wave - 4) * 8 + (lane >> 3);
    uint32_t at, at_s = kOutside;
    int n = 0, chunk;
    if (is_x) {
        chunk = ((lane & 15) ^ place_few(row)) * 16;
        at = (uint32_t)row * (uint32_t)m.x_row + chunk;
    } else {
        const int srow = wrow<GATED, FRAGS>((wave - 4) * 64 + lane, n0, m.N, n);
        if (n < m.N) at_s = (uint32_t)srow * (uint32_t)a.s_row;
        chunk = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
        at = (uint32_t)wrow<GATED, FRAGS>(row, n0, m.N, n) * (uint32_t)m.w_row + chunk;
    }
    // output columns between the first row of w and the row 32 i further
    auto apart = [](int i) {
        return (FRAGS == 2 ? i * 32 : (i & 1) * 8 + (i >> 1) * 64) / (GATED ? 2 : 1);
    };
    auto fetch_x = [&](int p, int stage) {
        const bool in = p * 256 + chunk < m.row_bytes;
        const uint32_t k = 2 * p * kSlab < m.row_bytes ? p * 256 : 0;
#pragma unroll
        for (int i = 0; i < FX; ++i)
            load_to_lds(rx, lds0 + stage * PAIR_X + (i * 4 + wave) * 1024,
                        in && row + i * 16 < left ? at + i * 16u * (uint32_t)m.x_row : kOutside,
                        k);
    };
    // Half h of quad p: the scales first, then half of the rows' codes (those
    // behind a row's end meet a scale of zero).
    auto fetch_w = [&](int p, int h, int stage) {
        const bool any = 2 * p < npair;
        if (h == 0)
            load_to_lds(rs, lds0 + AT_S + stage * kScaleSet + (wave - 4) * 1024,
                        any ? at_s : kOutside, any ? (GROUP == 16 ? p : p >> 1) * 16 : 0);
        const uint32_t k = any ? p * 128 : 0;
#pragma unroll
        for (int i = 4 * h; i < 4 * h + 4; ++i)
            load_to_lds(rw, lds0 + AT_W + stage * kQuad + (i * 4 + wave - 4) * 1024,
                        any && n + apart(i) < m.N ? at + apart(i) * (uint32_t)m.w_row : kOutside,
                        k);
    };

    const int r = lane & 15, q = lane >> 4;
    const int rdx = (wm * (JF * 16) + r) * 256 + ((4 * q) ^ place_few(r)) * 16;
    const int rdw = AT_W + (wn * (FRAGS * 16) + r) * 128 + (q ^ (r >> 1)) * 16;
    const int rds = AT_S + (wn * (FRAGS * 16) + r) * 16 + q * (32 / GROUP);
    f32x4 acc[FRAGS][JF];
#pragma unroll
    for (int i = 0; i < FRAGS; ++i)
#pragma unroll
        for (int j = 0; j < JF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 fx[2][2][JF];                           // of a unit's two chunks
    u32x4 c[2][FRAGS];                            // codes of this pair and of the next
    uint32_t sc[2][FRAGS];
    auto read_x = [&](auto unit, const uint8_t* px) {
        constexpr int u = decltype(unit)::value;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < JF; ++j)
                fx[u][h][j] = *reinterpret_cast<const u32x4*>(px + (rdx ^ ((2 * u + h) * 16)) +
                                                              j * 16 * 256);
    };
    auto read_codes = [&](int to, int p, int stage) {
        const uint8_t* pw = lds + stage * kQuad;
        const uint8_t* ps =
            lds + rds + stage * kScaleSet + (GROUP == 16 ? (p & 1) * 8 : (p & 3) * 4);
#pragma unroll
        for (int i = 0; i < FRAGS; ++i) {
            c[to][i] = *reinterpret_cast<const u32x4*>(pw + (rdw ^ ((p & 1) * 64)) + i * 16 * 128);
            sc[to][i] = GROUP == 16 ? *reinterpret_cast<const uint16_t*>(ps + i * 16 * 16)
                                    : ps[i * 16 * 16];
        }
    };
    auto multiply = [&](auto unit, int of) {
        constexpr int u = decltype(unit)::value;
#pragma unroll
        for (int i = 0; i < FRAGS; ++i) {
            const float f = GROUP == 16 ? __builtin_amdgcn_cvt_f32_fp8((int)sc[of][i], u)
                                        : __uint_as_float(sc[of][i] << 23);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 w = widen4<GROUP>(c[of][i][2 * u + h], f);
#pragma unroll
                for (int j = 0; j < JF; ++j) acc[i][j] = mma_bf16(w, fx[u][h][j], acc[i][j]);
            }
        }
    };
    const std::integral_constant<int, 0> first;
    const std::integral_constant<int, 1> second;

    if (is_x) {
#pragma unroll
        for (int v = 0; v < XS; ++v) fetch_x(v, v);
        wait_and_barrier<(XS - 1) * FX>();
    } else {
#pragma unroll
        for (int v = 0; v < WS; ++v) {
            fetch_w(v, 0, v);
            fetch_w(v, 1, v);
        }
        wait_and_barrier<(WS - 1) * FW>();
    }
    read_codes(0, 0, 0);
    read_x(first, lds);
    int ix = 0, iw = 0;                           // stages of pair p and of its quad
    auto one = [&](int p, auto of) {
        constexpr int now = decltype(of)::value;
        // what follows the last scale may be anything
        if (p * 128 + q * 32 >= H)
#pragma unroll
            for (int i = 0; i < FRAGS; ++i) sc[now][i] = 0;
        read_x(second, lds + ix * PAIR_X);
        __builtin_amdgcn_sched_barrier(0);
        multiply(first, now);
        // Pair p is read; pair p + 1 (and its quad) has arrived. Behind it are the
        // loads of XS - 2 pairs of x, of WS - 2 quads of codes.
        if (is_x) wait_and_barrier<(XS - 2) * FX>();
        else if (now == 1) wait_and_barrier<(WS - 2) * FW>();
        else asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const int nix = ix + 1 < XS ? ix + 1 : 0;
        const int niw = now == 0 ? iw : iw + 1 < WS ? iw + 1 : 0;
        read_codes(1 - now, p + 1, niw);
        read_x(first, lds + nix * PAIR_X);
        // a quad's codes are all read before its second pair's barrier: from
        // there on its place is filled again, half of it at a time
        if (is_x) fetch_x(p + XS, ix);
        else if (now == 1) fetch_w((p >> 1) + WS, 0, iw);
        else if (p > 0) fetch_w((p >> 1) + WS - 1, 1, iw == 0 ? WS - 1 : iw - 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(second, now);
        ix = nix;
        iw = niw;
    };
    for (int p = 0; p < npair; p += 2) {
        one(p, first);
        if (p + 1 < npair) one(p + 1, second);
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

// Tiles of each kind (n; of a few rows the runs) and of all but those, and up to how
// many rows a group takes few-row tiles: kSmall, or all groups do, or none.
template <int GROUP, bool GATED>
__device__ __forceinline__ int plan_tiles(const MatmulArgs& m, int rows0, int (&n)[kKinds],
                                          int& total) {
    constexpr int BB = GATED ? kCols / 2 : kCols;
    const int ntb = (m.N + BB - 1) / BB;
    int small_to = m.counts ? kSmall : 0;
    for (;;) {
        count_runs(m, rows0, small_to, n);
        total = 0;
#pragma unroll
        for (int k = 1; k < kKinds; ++k) {
            n[k] *= ntb;
            total += n[k];
        }
        if (!small_to || small_to == INT32_MAX || total == 0) break;
        if (total > kGrid) {
            // a few rows beside so much else: in part-filled tiles
            small_to = 0;
            continue;
        }
        // one round of big tiles, in parts of these rows, or few-row tiles for all
        int most = 0, runs = 0;
#pragma unroll
        for (int k = 1; k < kKinds; ++k)
            if (n[k]) most = k;
        for (int g0 = 0; g0 < m.groups; g0 += 64)
            runs += __builtin_amdgcn_readlane(
                wave_inclusive_scan(runs_of(g0 ? lane_rows(m, g0) : rows0, INT32_MAX, 0)), 63);
        if (!few_instead(total, most, runs, n[0], m.N, m.row_bytes / 2, GATED ? kSmall / 2 : kSmall,
                         GROUP))
            break;
        small_to = INT32_MAX;
    }
    return small_to;
}

// A block's share of all tiles; TALL: of all heights, else of 32 rows.
template <int GROUP, bool GATED, bool TALL>
__device__ __forceinline__ void all_tiles(const W4Args& a, uint8_t* lds, int rows0) {
    const MatmulArgs& m = a.m;
    constexpr int BB = GATED ? kCols / 2 : kCols;
    // 64 rows: each wave all of them, so that a weight is widened once, or with
    // powers of two, which take little of that, half of them and less of LDS
    constexpr int MID64 = GROUP == 16 ? 8 : 4;
    const int ntb = (m.N + BB - 1) / BB;
    int n[kKinds], total;
    // (in scalar registers, which is where the tiles' loads take what follows from
    // them: behind branches on fp32 numbers the compiler may hold them in vector ones)
    const int small_to = uniform(plan_tiles<GROUP, GATED>(m, rows0, n, total));
    total = uniform(total);
#pragma unroll
    for (int k = 0; k < kKinds; ++k) n[k] = uniform(n[k]);
    const int parts = last_parts(total);
    for (int t0 = 0; t0 < total; t0 += kGrid) {
        const Turn turn = turn_of(blockIdx.x, t0, total, parts);
        if (turn.t < 0) break;
        int t = turn.t;
        int kind = TALL ? kKinds - 1 : 1;
#pragma unroll
        for (int k = kKinds - 1; k > 1; --k)
            if (kind == k && t >= n[k]) {
                t -= n[k];
                --kind;
            }
        const Place at = find_tile(m, rows0, small_to, kind, ntb, t);
        const int runs = cut_rows(at.rows, small_to).runs;
        const Piece p = piece_of(at.l, at.rows, runs, kind, ntb, turn.sub, turn.cut);
        if (p.m0 >= p.end) continue;
        const int n0 = p.col * BB;
        auto run = [&](auto bm) {
            w4_tile<GROUP, GATED, decltype(bm)::value>(a, at.g, p.m0, p.end, n0, lds);
        };
        const int f = TALL ? p.fragments : 1;
        if (f == 8) run(std::integral_constant<int, 256>{});
        else if (f == 7) run(std::integral_constant<int, 224>{});
        else if (f == 6) run(std::integral_constant<int, 192>{});
        else if (f == 5) run(std::integral_constant<int, 160>{});
        else if (f > 2) w4_mid_tile<GROUP, GATED, 128, 4>(a, at.g, p.m0, p.end, n0, lds);
        else if (f == 2) w4_mid_tile<GROUP, GATED, 64, MID64>(a, at.g, p.m0, p.end, n0, lds);
        else w4_mid_tile<GROUP, GATED, 32, 8>(a, at.g, p.m0, p.end, n0, lds);
    }
    if (n[0] > 0) few_rows<GROUP, GATED>(a, lds, rows0, small_to, n[0]);
}

// Few-row tiles for all groups.
template <int GROUP, bool GATED>
__device__ __forceinline__ void only_few_rows(const W4Args& a, uint8_t* lds, int rows0) {
    int runs = 0;
    for (int g0 = 0; g0 < a.m.groups; g0 += 64)
        runs += __builtin_amdgcn_readlane(
            wave_inclusive_scan(runs_of(g0 ? lane_rows(a.m, g0) : rows0, INT32_MAX, 0)), 63);
    if (runs > 0) few_rows<GROUP, GATED>(a, lds, rows0, INT32_MAX, runs);
}

// Three kernels, since beside more code few rows take longer (by expert, 32 of one
// or two rows or none, 2048 -> 7168, powers of two: 43, 43 and 50 us): with few-row
// tiles only; with tiles of 32 rows too, for groups of up to 32 rows (32 experts of
// 32 rows, 7168 -> 2 x 2048, E4M3: 281 us without, 129 with); and with all.
template <int GROUP, bool GATED>
__global__ __launch_bounds__(kThreads, 2) void w4_few_kernel(const W4Args a) {
    __shared__ __align__(1024) uint8_t lds[kFewLds];
    if (!a.m.counts) return few_rows<GROUP, GATED>(a, lds, 0, INT32_MAX, 0);
    only_few_rows<GROUP, GATED>(a, lds, lane_rows(a.m, 0));
}

template <int GROUP, bool GATED>
__global__ __launch_bounds__(kThreads, 2) void w4_low_kernel(const W4Args a) {
    __shared__ __align__(1024) uint8_t lds[kLds];
    const int rows0 = lane_rows(a.m, 0);
    bool more = false;
    for (int g0 = 0; g0 < a.m.groups; g0 += 64)
        more |= __ballot((g0 ? lane_rows(a.m, g0) : rows0) > kSmall) != 0;
    if (!more) return only_few_rows<GROUP, GATED>(a, lds, rows0);
    all_tiles<GROUP, GATED, false>(a, lds, rows0);
}

template <int GROUP, bool GATED>
__global__ __launch_bounds__(kThreads, 2) void w4_big_kernel(const W4Args a) {
    __shared__ __align__(1024) uint8_t lds[kLds];
    all_tiles<GROUP, GATED, true>(a, lds, lane_rows(a.m, 0));
}

template <int GROUP, bool GATED>
hipError_t launch(const W4Args& a, hipStream_t st) {
    const MatmulArgs& m = a.m;
    constexpr int BO = GATED ? kSmall / 2 : kSmall, BB = GATED ? kCols / 2 : kCols;
    const int H = m.row_bytes / 2;
    bool few;
    W4Args b = a;
    if (m.counts) {
        few = m.rows <= 2 * kSmall && few_if_full(m.groups, m.rows, m.N, H, BO, BB, GROUP);
    } else {
        b.cut = few_cut((m.rows + kSmall - 1) / kSmall, m.N, H, BO, m.rows > 8 ? 1 : 0);
        few = few_over_all(b.cut, m.rows, m.N, H, BB, GROUP);
    }
    if (few) w4_few_kernel<GROUP, GATED><<<kGrid, kThreads, 0, st>>>(b);
    else if (m.counts && m.rows <= 2 * kSmall)
        w4_low_kernel<GROUP, GATED><<<kGrid, kThreads, 0, st>>>(b);
    else w4_big_kernel<GROUP, GATED><<<kGrid, kThreads, 0, st>>>(b);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul_w4(const W4Args& a, hipStream_t st) {
    const bool gated = a.m.act == MOE_EP_ACT_SILU_GATED;
    if (a.group == 16) return gated ? launch<16, true>(a, st) : launch<16, false>(a, st);
    return gated ? launch<32, true>(a, st) : launch<32, false>(a, st);
}

}  // namespace moe_ep
