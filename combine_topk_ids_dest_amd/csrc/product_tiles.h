// What the tiles of the products share: fragments and the matrix instruction,
// loads into LDS, the epilogue, and the list of tiles that a grid works through.
// Included by the files of kernels, which each get a copy of their own.
#pragma once

#include <type_traits>

#include "experts.h"
#include "tiles.h"

namespace moe_ep {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_byte;

constexpr int kThreads = 512;                    // of a block of big tiles
constexpr int kWaves = kThreads / 64;
constexpr int kSlab = 128;                       // bytes of k per step
constexpr uint32_t kOutside = 0x80000000u;       // past every buffer's range

// A value that every lane of the wave has, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// 32 bytes of k of one row: a lane's share of a fragment.
struct Frag {
    u32x4 v[2];
};

__device__ __forceinline__ f32x4 mma_bf16(const u32x4& w, const u32x4& x, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                   __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
}

// v * sigmoid(v). The hardware's reciprocal is within an ulp; a division would
// be most of an epilogue's instructions.
__device__ __forceinline__ float silu(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + expf(-v));
}

__device__ __forceinline__ float gelu(float v) {
    return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
}

__device__ __forceinline__ float apply_act(float v, int act) {
    if (act == MOE_EP_ACT_SILU) return silu(v);
    if (act == MOE_EP_ACT_GELU) return gelu(v);
    return v;
}

__device__ __forceinline__ float silu_gated(float gate, float up) {
    return silu(gate) * up;
}

// Rounded to bf16 to nearest even (the hardware's conversion: two values an
// instruction, against five for one in integers).
__device__ __forceinline__ u32x2 pack_bf16(f32x4 v) {
    return __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
}

// max(m, |x|) where a NaN x leaves m as it is
__device__ __forceinline__ float abs_max(float m, float x) {
    const float a = fabsf(x);
    return a > m ? a : m;
}

// amax / 448, or 1 without an amax. Among fp32's smallest numbers that rounds
// to 0, or so far down that amax / s is past what rounds to the largest code
// (464 to 448), and the codes would be NaN: there the scale is the number above.
// (A row of bf16, as the pack quantises it, has no amax so small.)
__device__ __forceinline__ float group_scale(float amax) {
    const float s = amax / 448.0f;
    if (s * 460.0f < amax) return __uint_as_float(__float_as_uint(s) + 1);
    return amax > 0.f ? s : 1.0f;
}

// Four e4m3 codes of v / s; each carries the sign of its input.
__device__ __forceinline__ uint32_t codes4(f32x4 v, float s) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = v[i] / s;
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    const uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    uint32_t sign = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sign |= (__float_as_uint(v[i]) >> 31) << (8 * i + 7);
    return (c & 0x7F7F7F7Fu) | sign;
}

__device__ __forceinline__ int group_rows(const MatmulArgs& a, int g) {
    if (!a.counts) return a.rows;
    const int c = a.counts[g];
    return c < 0 ? 0 : c > a.rows ? a.rows : c;
}

// The buffer resource of row_rsrc as four scalar registers.
__device__ __forceinline__ i32x4 row_rsrc4(const uint8_t* p, int64_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    i32x4 r;
    r[0] = uniform((int)(uint32_t)at);
    r[1] = uniform((int)(uint32_t)(at >> 32) & 0xFFFF);
    r[2] = uniform((int)(bytes < INT32_MAX ? bytes : INT32_MAX));
    r[3] = 0x00020000;
    return r;
}

// A resource that went through a branch, in scalar registers again: the loads
// below take nothing else, and at -O1 the compiler may hold it in vector ones.
__device__ __forceinline__ i32x4 uniform(i32x4 r) {
    return i32x4{uniform(r[0]), uniform(r[1]), uniform(r[2]), uniform(r[3])};
}

// 16 (or 4) bytes per lane from memory into LDS, lane l's at dst + 16 l (4 l);
// dst is uniform, in M0. Written out so that the compiler does not count it
// among the loads that an LDS read has to wait for: with its own form of this
// instruction it waits for every load in flight before the next LDS read,
// whatever that reads. The instruction has no output register; what it
// writes is ordered by the waits and barriers below.
//
// A memory instruction may read a scalar register five wait states after a
// vector instruction wrote it at the soonest (a readfirstlane, or the readlane
// that brings a spilled one back), and the compiler, which sees to that
// elsewhere, does not look in here: s_mov and s_nop 3 are the five, whatever
// comes before. (M0 itself needs one.)
__device__ __forceinline__ void load_to_lds(i32x4 r, uint32_t dst, uint32_t off, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(dst), "v"(off), "s"(r), "s"(soff)
                 : "m0");
}
__device__ __forceinline__ void load4_to_lds(i32x4 r, uint32_t dst, uint32_t off, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(dst), "v"(off), "s"(r), "s"(soff)
                 : "m0");
}

// Row of w behind row r of a tile whose first output column is n0, and its
// output column n (columns n >= N do not exist). A wave has FRAGS fragments of
// 16 rows. A fragment's row 4 q + t becomes the sums t of the lanes 16 q ..;
// with four, fragment i of a wave holds the columns 16 q + 4 i + t, gated
// fragments 2 p + h the gate (h = 0) and up rows of the columns 8 q + 4 p + t.
template <bool GATED, int FRAGS>
__device__ __forceinline__ int wrow(int r, int n0, int N, int& n) {
    const int i = (r >> 4) & (FRAGS - 1), q = (r >> 2) & 3, t = r & 3;
    const int wave = r / (FRAGS * 16);
    if (!GATED) {
        n = n0 + wave * FRAGS * 16 + q * FRAGS * 4 + i * 4 + t;
        return n;
    }
    n = n0 + wave * FRAGS * 8 + q * FRAGS * 2 + (i >> 1) * 4 + t;
    return (i & 1) ? N + n : n;
}

// Waits until at most LEFT of this wave's loads are in flight and for its LDS
// reads, then for the block.
template <int LEFT>
__device__ __forceinline__ void wait_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ f32x4 load_f32x4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(f32x4, ld_row_buf<false>(r, off));
}

// The epilogue of a tile: bias, activation, residual and rounding, or the
// quantising of rows.
template <int EB, bool GATED, int FRAGS, int JF, int WN>
__device__ __forceinline__ void finish_tile(const MatmulArgs& a, int g, int m0, int left, int n0,
                                            f32x4 (&acc)[FRAGS][JF], uint8_t* lds) {
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int nw = GATED ? 2 * a.N : a.N;
    // A lane has QN quads of consecutive columns from n on, of rows
    // 16 (wm JF + j) + lane % 16. Rows and columns that do not exist are
    // outside the buffers' ranges: their loads give 0, their stores nothing.
    constexpr int QN = GATED ? FRAGS / 2 : FRAGS;
    const int n = n0 + wn * QN * 16 + (lane >> 4) * QN * 4;
    if (a.bias) {
        const auto rb = row_rsrc(reinterpret_cast<const uint8_t*>(a.bias + g * a.bias_stride),
                                 (int64_t)nw * 4);
#pragma unroll
        for (int q = 0; q < QN; ++q) {
            const uint32_t at = n + q * 4 < a.N ? (uint32_t)(n + q * 4) * 4 : kOutside;
            const f32x4 b = load_f32x4(rb, at);
            const f32x4 bu = GATED ? load_f32x4(rb, at + (uint32_t)a.N * 4) : b;
#pragma unroll
            for (int j = 0; j < JF; ++j) {
                acc[GATED ? 2 * q : q][j] += b;
                if (GATED) acc[2 * q + 1][j] += bu;
            }
        }
    }
    uint8_t* const out = a.out + g * a.out_stride + (int64_t)m0 * a.out_row;
    const int mrow = wm * (JF * 16) + (lane & 15);

    // The rest once for each activation: one branch, not one for each value.
    auto rest = [&](auto activation) {
        auto value = [&](int q, int j) {
            f32x4 v = acc[GATED ? 2 * q : q][j];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = GATED ? silu_gated(v[e], acc[GATED ? 2 * q + 1 : q][j][e]) : activation(v[e]);
            return v;
        };

        if constexpr (EB == 1) {
            if (a.out_dtype == MOE_EP_E4M3) {
                // a row's 128 columns lie in 4 (gated) or 2 waves, 4 lanes each
                constexpr int WG = GATED ? 4 : 2;
                float* part = reinterpret_cast<float*>(lds);            // [BM][4]
                f32x4 y[QN][JF];
#pragma unroll
                for (int j = 0; j < JF; ++j) {
                    float mx = 0.f;
#pragma unroll
                    for (int q = 0; q < QN; ++q) {
                        y[q][j] = value(q, j);
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx = abs_max(mx, y[q][j][e]);
                    }
                    mx = abs_max(mx, __shfl_xor(mx, 16, 64));
                    mx = abs_max(mx, __shfl_xor(mx, 32, 64));
                    if (lane < 16) part[(mrow + j * 16) * 4 + wn] = mx;
                }
                __syncthreads();
                const int groups = a.N / kScaleBlock;
#pragma unroll
                for (int j = 0; j < JF; ++j) {
                    const int m = mrow + j * 16;
                    float mx = 0.f;
#pragma unroll
                    for (int w = 0; w < WG; ++w) mx = abs_max(mx, part[m * 4 + (GATED ? 0 : wn & 2) + w]);
                    const float s = group_scale(mx);
                    if (m < left && n < a.N) {
                        uint32_t* o = reinterpret_cast<uint32_t*>(out + (int64_t)m * a.out_row + n);
#pragma unroll
                        for (int q = 0; q < QN; ++q) o[q] = codes4(y[q][j], s);
                        float* os = a.os + g * a.os_stride + (int64_t)(m0 + m) * a.os_pitch;
                        if (lane < 16 && wn % WG == 0) {
                            os[n / kScaleBlock] = s;
                            // the last group's wave also writes the padding
                            if (n / kScaleBlock == groups - 1)
                                for (int p = groups; p < (int)a.os_pitch; ++p) os[p] = 0.f;
                        }
                    }
                }
                __syncthreads();   // the next tile writes lds again
                return;
            }
        }

        const bool f32 = a.out_dtype == MOE_EP_F32;
        const int eb = f32 ? 4 : 2;
        const auto ro = row_rsrc(out, (int64_t)(left - 1) * a.out_row + (int64_t)a.N * eb);
        const auto rr = row_rsrc(a.res ? a.res + (int64_t)m0 * a.res_row : out,
                                 a.res ? (int64_t)(left - 1) * a.res_row + (int64_t)a.N * eb : 0);
        auto at = [&](int j, int q, int64_t row) {
            const int m = mrow + j * 16, c = n + q * 4;
            return m < left && c < a.N ? (uint32_t)m * (uint32_t)row + (uint32_t)(c * eb) : kOutside;
        };
        if (f32) {
#pragma unroll
            for (int j = 0; j < JF; ++j) {
                f32x4 r[QN];
                if (a.res) {
#pragma unroll
                    for (int q = 0; q < QN; ++q) r[q] = load_f32x4(rr, at(j, q, a.res_row));
                }
#pragma unroll
                for (int q = 0; q < QN; ++q) {
                    f32x4 y = value(q, j);
                    if (a.res) y += r[q];
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), ro,
                                                           at(j, q, a.out_row), 0, 0);
                }
            }
            return;
        }
        if constexpr (QN == 1) {
#pragma unroll
            for (int j = 0; j < JF; ++j) {
                f32x4 y = value(0, j);
                if (a.res) {
                    const u32x2 v = __builtin_bit_cast(
                        u32x2, __builtin_amdgcn_raw_buffer_load_b64(rr, at(j, 0, a.res_row), 0, 0));
                    y += f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
                }
                __builtin_amdgcn_raw_buffer_store_b64(pack_bf16(y), ro, at(j, 0, a.out_row), 0, 0);
            }
            return;
        }
        // bf16: N is a multiple of 8, so eight columns exist together; the
        // residuals of four rows are on their way at once
        constexpr int JB = JF < 4 ? JF : 4;
#pragma unroll
        for (int j0 = 0; j0 < JF; j0 += JB) {
            u32x4 r[JB][QN < 2 ? 1 : QN / 2];
            if (a.res) {
#pragma unroll
                for (int j = 0; j < JB && j0 + j < JF; ++j)
#pragma unroll
                    for (int q = 0; q < QN / 2; ++q)
                        r[j][q] = ld_row_buf<false>(rr, at(j0 + j, 2 * q, a.res_row));
            }
#pragma unroll
            for (int j = 0; j < JB && j0 + j < JF; ++j)
#pragma unroll
                for (int q = 0; q < QN / 2; ++q) {
                    f32x4 lo = value(2 * q, j0 + j), hi = value(2 * q + 1, j0 + j);
                    if (a.res) {
                        const u32x4 v = r[j][q];
                        lo += f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
                        hi += f32x4{bf16_lo(v[2]), bf16_hi(v[2]), bf16_lo(v[3]), bf16_hi(v[3])};
                    }
                    const u32x2 l = pack_bf16(lo), h = pack_bf16(hi);
                    __builtin_amdgcn_raw_buffer_store_b128(u32x4{l[0], l[1], h[0], h[1]}, ro,
                                                           at(j0 + j, 2 * q, a.out_row), 0, 0);
                }
        }
    };
    if constexpr (GATED) {
        rest([](float v) { return v; });
    } else {
        if (a.act == MOE_EP_ACT_SILU) rest([](float v) { return silu(v); });
        else if (a.act == MOE_EP_ACT_GELU) rest([](float v) { return gelu(v); });
        else rest([](float v) { return v; });
    }
}

// ---------------------------------------------------------------------
// The work list. A group's rows are cut into equal runs of at most 256 rows (a
// multiple of 32), so that a group's weights are read by all of its runs at the
// same time, side by side on one XCD, and from HBM once. (Whole runs of 256 and
// a remainder read them twice: 1.7 times the bytes at 32 experts of 240 to 1280
// rows, 1066 against 835 us for products of 7168 columns with 2 x 2048 rows.)
// Groups of up to small_to rows get small tiles.
//
// Tiles are dealt out longest runs first, one to a block and round, one block
// per CU. Every block computes its share from the counts for itself: there is
// no queue, so nothing to clear and no order left to chance.
// ---------------------------------------------------------------------
constexpr int kRuns64 = kKinds;                  // every group in runs of 64 rows,
constexpr int kRuns128 = kKinds + 1;             // or of 128 (but for small ones)

// A group's runs of a kind.
__device__ __forceinline__ int runs_of(int rows, int small_to, int kind) {
    const Cut c = cut_rows(rows, small_to);
    if (kind >= kRuns64) {
        const int run = kind == kRuns64 ? 64 : 128;
        return c.kind ? (rows + run - 1) / run : 0;
    }
    return c.kind == kind ? c.runs : 0;
}

// The rows of the groups g0 + lane (0 past the last).
__device__ __forceinline__ int lane_rows(const MatmulArgs& a, int g0) {
    const int g = g0 + (int)(threadIdx.x & 63);
    return g < a.groups ? group_rows(a, g) : 0;
}

// Everything here is done by each wave for itself, with no LDS (the tiles take
// all of it): a group to a lane, 64 groups at a time. rows0: lane_rows(a, 0).

// Runs of each kind, of all groups.
__device__ __forceinline__ void count_runs(const MatmulArgs& a, int rows0, int small_to,
                                           int (&total)[kKinds]) {
#pragma unroll
    for (int k = 0; k < kKinds; ++k) total[k] = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
        const Cut c = cut_rows(g0 ? lane_rows(a, g0) : rows0, small_to);
        const int32_t inc = wave_inclusive_scan(c.runs);
#pragma unroll
        for (int k = 0; k < kKinds; ++k) {
            uint64_t mine = __ballot(c.kind == k && c.runs > 0);
            while (mine) {                       // few lanes, or all of one kind
                const int l = __builtin_ctzll(mine);
                // a stretch of lanes of this kind at once
                const uint64_t rest = ~(mine >> l);
                const int n = rest ? __builtin_ctzll(rest) : 64 - l;
                total[k] += __builtin_amdgcn_readlane(inc, l + n - 1) -
                            (l ? __builtin_amdgcn_readlane(inc, l - 1) : 0);
                mine = l + n < 64 ? mine >> (l + n) << (l + n) : 0;
            }
        }
    }
}

// The group of tile t of a kind (nt tiles to a run), its rows and the tile's
// number in it.
struct Place {
    int g, rows, l;
};

__device__ __forceinline__ Place find_tile(const MatmulArgs& a, int rows0, int small_to, int kind,
                                           int nt, int t) {
    for (int g0 = 0;; g0 += 64) {
        const int rows = g0 ? lane_rows(a, g0) : rows0;
        const int n = nt * runs_of(rows, small_to, kind);
        const int32_t inc = wave_inclusive_scan(n);
        const uint64_t behind = __ballot(inc > t);
        if (behind || g0 + 64 >= a.groups) {     // t is below the total: a lane is found
            const int lane = behind ? __builtin_ctzll(behind) : 0;
            Place p;
            p.g = uniform(g0 + lane);
            p.rows = __builtin_amdgcn_readlane(rows, lane);
            p.l = t - (__builtin_amdgcn_readlane(inc, lane) - __builtin_amdgcn_readlane(n, lane));
            return p;
        }
        t -= __builtin_amdgcn_readlane(inc, 63);
    }
}

}  // namespace
}  // namespace moe_ep
