// Products of rows with weight matrices, grouped by expert with ragged row
// counts or over all tokens of a rank:
//   out[g][r][n] = act(sum_k x[g][r][k] * w[g][n][k] + bias[g][n]) + residual.
// Sums are fp32 in the matrix cores. x and w are both stored with k innermost,
// so both operands of an MFMA load the same way: a lane of a 16-row fragment
// takes 32 consecutive bytes of row lane % 16 from every 128-byte slab of k
// (any assignment of k to lanes gives the same sum as long as both operands
// share it). w is the A operand: a lane's four accumulators are four
// consecutive output columns of one row, so the epilogue works on vectors.
//
// silu_gated: w holds N gate rows, then N up rows. Fragments alternate between
// the two, so gate and up of an output meet in one tile (wrow()).
//
// fp8: a slab of 128 codes is one scale block: acc += (sx * sw) * slab sum.
#include "experts.h"

namespace moe_ep {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kSlab = 128;                       // bytes of k per step
constexpr uint32_t kOutside = 0x80000000u;       // past every buffer's range

// 32 bytes of k of one row: a lane's share of a fragment.
struct Frag {
    u32x4 v[2];
};

// A value that every lane of the wave has, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int EB>
__device__ __forceinline__ f32x4 mma(const Frag& w, const Frag& x, f32x4 acc) {
    if constexpr (EB == 2) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.v[0]),
                                                      __builtin_bit_cast(bf16x8, x.v[0]), acc,
                                                      0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.v[1]),
                                                       __builtin_bit_cast(bf16x8, x.v[1]), acc,
                                                       0, 0, 0);
    } else {
        // e4m3 x e4m3 with the blocks' exponents at 1.0 (127)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            __builtin_bit_cast(i32x8, w), __builtin_bit_cast(i32x8, x), acc, 0, 0, 0,
            0x7F7F7F7F, 0, 0x7F7F7F7F);
    }
}

// Row of w behind row r of a tile whose first output column is n0; its
// output column in n (columns n >= N do not exist).
template <bool GATED>
__device__ __forceinline__ int wrow(int r, int n0, int N, int& n) {
    if (!GATED) {
        n = n0 + r;
        return n;
    }
    n = n0 + (r >> 5) * 16 + (r & 15);
    return (r & 16) ? N + n : n;
}

__device__ __forceinline__ float apply_act(float v, int act) {
    if (act == MOE_EP_ACT_SILU) return v / (1.0f + expf(-v));
    if (act == MOE_EP_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    return v;
}

__device__ __forceinline__ float silu_gated(float gate, float up) {
    return gate / (1.0f + expf(-gate)) * up;
}

// Four output columns n..n+3 of row m, from their sums.
template <bool GATED>
__device__ __forceinline__ f32x4 finish(const MatmulArgs& a, int g, int n, f32x4 v, f32x4 up) {
    if (a.bias) {
        const float* b = a.bias + (int64_t)g * a.bias_stride + n;
        v += *reinterpret_cast<const f32x4*>(b);
        if (GATED) up += *reinterpret_cast<const f32x4*>(b + a.N);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = GATED ? silu_gated(v[i], up[i]) : apply_act(v[i], a.act);
    return v;
}

__device__ __forceinline__ u32x2 pack_bf16(f32x4 v) {
    u32x2 o;
    o[0] = to_bf16_rne(v[0]) | (to_bf16_rne(v[1]) << 16);
    o[1] = to_bf16_rne(v[2]) | (to_bf16_rne(v[3]) << 16);
    return o;
}

__device__ __forceinline__ void store_out(const MatmulArgs& a, int g, int64_t m, int n, f32x4 v) {
    const int64_t col = (int64_t)n * (a.out_dtype == MOE_EP_F32 ? 4 : 2);
    uint8_t* o = a.out + g * a.out_stride + m * a.out_row + col;
    if (a.out_dtype == MOE_EP_F32) {
        if (a.res) v += *reinterpret_cast<const f32x4*>(a.res + m * a.res_row + col);
        *reinterpret_cast<f32x4*>(o) = v;
    } else {
        if (a.res) {
            const u32x2 r = *reinterpret_cast<const u32x2*>(a.res + m * a.res_row + col);
            v[0] += bf16_lo(r[0]);
            v[1] += bf16_hi(r[0]);
            v[2] += bf16_lo(r[1]);
            v[3] += bf16_hi(r[1]);
        }
        *reinterpret_cast<u32x2*>(o) = pack_bf16(v);
    }
}

// max(m, |x|) where a NaN x leaves m as it is
__device__ __forceinline__ float abs_max(float m, float x) {
    const float a = fabsf(x);
    return a > m ? a : m;
}

// Four e4m3 codes of v / s; each carries the sign of its input.
__device__ __forceinline__ uint32_t codes4(f32x4 v, float s) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = v[i] / s;
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
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

// ---------------------------------------------------------------------
// Small tiles: BM rows of x by BN rows of w, the slabs of k dealt to the
// block's waves in turn (so that a tile alone already keeps eight waves'
// loads in flight and the block reads 1 KB runs of each row), fragments
// loaded straight into registers, the waves' sums added in wave order.
// ---------------------------------------------------------------------
template <int EB, bool GATED, int BM, int BN, int DEPTH>
__device__ __forceinline__ void small_tile(const MatmulArgs& a, int g, int m0, int rows,
                                           int n0, float* lds) {
    constexpr int FM = BM / 16, FN = BN / 16;
    constexpr int PITCH = BN + 4;
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int kb = a.row_bytes;
    const int nslab = (kb + kSlab - 1) / kSlab;
    const int left = rows - m0;

    const int nw = GATED ? 2 * a.N : a.N;
    const uint8_t* xb = a.x + g * a.x_stride + (int64_t)m0 * a.x_row;
    const uint8_t* wb = a.w + g * a.w_stride;
    const auto rx = row_rsrc(xb, (int64_t)(left - 1) * a.x_row + kb);
    const auto rw = row_rsrc(wb, (int64_t)(nw - 1) * a.w_row + kb);
    const uint32_t kin = (uint32_t)(lane >> 4) * 32u;
    uint32_t vx[FM], vw[FN];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        const int m = f * 16 + (lane & 15);
        vx[f] = m < left ? (uint32_t)m * (uint32_t)a.x_row : kOutside;
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        int n;
        const int r = wrow<GATED>(f * 16 + (lane & 15), n0, a.N, n);
        vw[f] = n < a.N ? (uint32_t)r * (uint32_t)a.w_row : kOutside;
    }

    const float* xs[FM];
    const float* ws[FN];
    if constexpr (EB == 1) {
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            int m = f * 16 + (lane & 15);
            m = m < left ? m : left - 1;
            xs[f] = a.xs + g * a.xs_stride + (int64_t)(m0 + m) * a.xs_pitch;
        }
        const int per = (a.N + kScaleBlock - 1) / kScaleBlock;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            int n = GATED ? n0 + (f >> 1) * 16 : n0 + f * 16;
            n = n < a.N ? n : a.N - 1;
            const int blk = n / kScaleBlock + (GATED && (f & 1) ? per : 0);
            ws[f] = a.ws + g * a.ws_stride + (int64_t)blk * nslab;
        }
    }

    f32x4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    Frag fx[DEPTH][FM], fw[DEPTH][FN];
    float sx[DEPTH][FM], sw[DEPTH][FN];
    // A slab past the last loads nothing but zeros (the buffers' range check).
    auto load = [&](int d, int s) {
        const uint32_t k0 = (uint32_t)s * kSlab + kin;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t k = k0 + 16 * h;
            const uint32_t add = k < (uint32_t)kb ? k : kOutside;
#pragma unroll
            for (int f = 0; f < FN; ++f)
                fw[d][f].v[h] = ld_row_buf<false>(rw, (vw[f] | (add & kOutside)) + (add & ~kOutside));
#pragma unroll
            for (int f = 0; f < FM; ++f)
                fx[d][f].v[h] = ld_row_buf<false>(rx, (vx[f] | (add & kOutside)) + (add & ~kOutside));
        }
        if constexpr (EB == 1) {
            const int sc = s < nslab ? s : nslab - 1;
#pragma unroll
            for (int f = 0; f < FM; ++f) sx[d][f] = xs[f][sc];
#pragma unroll
            for (int f = 0; f < FN; ++f) sw[d][f] = ws[f][sc];
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(d, wave + d * kWaves);
    for (int s = wave; s < nslab; s += kWaves * DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) {
                    if constexpr (EB == 2) {
                        acc[i][j] = mma<EB>(fw[d][i], fx[d][j], acc[i][j]);
                    } else {
                        const f32x4 t = mma<EB>(fw[d][i], fx[d][j], f32x4{0.f, 0.f, 0.f, 0.f});
                        const float sc = sw[d][i] * sx[d][j];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[i][j][q] = __builtin_fmaf(t[q], sc, acc[i][j][q]);
                    }
                }
            load(d, s + (d + DEPTH) * kWaves);
        }
    }

#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
            *reinterpret_cast<f32x4*>(lds + ((wave * BM + j * 16 + (lane & 15)) * PITCH + i * 16 +
                                             (lane >> 4) * 4)) = acc[i][j];
    __syncthreads();
    auto sum = [&](int m, int r) {
        f32x4 v = *reinterpret_cast<const f32x4*>(lds + (m * PITCH + r));
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            v += *reinterpret_cast<const f32x4*>(lds + ((w * BM + m) * PITCH + r));
        return v;
    };
    constexpr int BO = GATED ? BN / 2 : BN;       // output columns
    constexpr int QUADS = BO / 4;
    const bool quant = EB == 1 && a.out_dtype == MOE_EP_E4M3;
    for (int q = threadIdx.x; q < BM * QUADS; q += kThreads) {
        const int m = q / QUADS;
        const int o = q % QUADS * 4;
        const int r = GATED ? (o >> 4) * 32 + (o & 15) : o;
        const f32x4 v = sum(m, r);
        const f32x4 up = GATED ? sum(m, r + 16) : v;
        const int n = n0 + o;
        const bool in = m < left && n < a.N;
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
        if (in) y = finish<GATED>(a, g, n, v, up);
        if constexpr (BO == kScaleBlock) {
            if (quant) {
                // 32 consecutive lanes hold the 128 columns of a row's group
                float mx = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) mx = abs_max(mx, y[i]);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) mx = abs_max(mx, __shfl_xor(mx, off, 32));
                const float s = mx > 0.f ? mx / 448.0f : 1.0f;
                if (in) {
                    *reinterpret_cast<uint32_t*>(a.out + g * a.out_stride +
                                                 (int64_t)(m0 + m) * a.out_row + n) = codes4(y, s);
                    if (o == 0)
                        a.os[g * a.os_stride + (int64_t)(m0 + m) * a.os_pitch + n / kScaleBlock] = s;
                }
                continue;
            }
        }
        if (in && !quant) store_out(a, g, m0 + m, n, y);
    }
    // the scale row's padding, by the blocks of its last group
    if (quant && BO == kScaleBlock && n0 + BO >= a.N) {
        const int groups = a.N / kScaleBlock;
        const int pad = (int)a.os_pitch - groups;
        for (int q = threadIdx.x; q < BM * pad; q += kThreads)
            if (q / pad < left)
                a.os[g * a.os_stride + (int64_t)(m0 + q / pad) * a.os_pitch + groups + q % pad] = 0.f;
    }
    __syncthreads();   // the next tile writes lds again
}

// ---------------------------------------------------------------------
// Big tiles: 256 rows of x by 256 rows of w. Eight waves in two rows of four,
// each with 128 x 64 of the sums in registers. Slabs of 128 bytes of k go
// from memory straight into LDS (no register is spent on a load in flight),
// one slab ahead of the one being multiplied; fragments are read from LDS
// half a slab ahead, so that the reads of one half run under the products
// of the other.
//
// LDS: row r of a slab holds its eight 16-byte chunks with chunk c at place
// c ^ ((r >> 1) & 7), so the 16 rows of a fragment's read fall on different
// banks. The load that fills LDS writes a wave's 64 x 16 bytes in lane order,
// so the permutation is applied to the addresses that the lanes read.
// ---------------------------------------------------------------------
constexpr int kBig = 256;
constexpr int kBigSlab = kBig * kSlab;           // bytes of one operand's slab
constexpr int kBigLds = 4 * kBigSlab;            // two slabs of both operands

typedef __attribute__((address_space(3))) uint8_t lds_byte;
typedef int i32x4 __attribute__((ext_vector_type(4)));

// The buffer resource of row_rsrc as four scalar registers.
__device__ __forceinline__ i32x4 row_rsrc4(const uint8_t* p, int64_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)at);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32) & 0xFFFF);
    r[2] = __builtin_amdgcn_readfirstlane((int)(bytes < INT32_MAX ? bytes : INT32_MAX));
    r[3] = 0x00020000;
    return r;
}

// 16 bytes per lane from memory into LDS, lane l's at dst + 16 l (dst is
// uniform, in M0). Written out so that the compiler does not count it among
// the loads that an LDS read has to wait for: with its own form of this
// instruction it waits for every load in flight before the next LDS read,
// whatever that reads. The instruction has no output register; what it
// writes is ordered by the waits and barriers below.
__device__ __forceinline__ void load_to_lds(i32x4 r, uint32_t dst, uint32_t off, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(dst), "v"(off), "s"(r), "s"(soff)
                 : "m0");
}

// Waits for this wave's loads into LDS and its LDS reads, then for the block.
__device__ __forceinline__ void wait_all_and_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <bool GATED>
__device__ __forceinline__ void big_tile(const MatmulArgs& a, int g, int m0, int rows, int n0,
                                         uint8_t* lds) {
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int wm = wave >> 2, wn = wave & 3;
    const int kb = a.row_bytes;
    const int nslab = (kb + kSlab - 1) / kSlab;
    const int left = rows - m0;
    const int nw = GATED ? 2 * a.N : a.N;
    const i32x4 rx = row_rsrc4(a.x + g * a.x_stride + (int64_t)m0 * a.x_row,
                               (int64_t)(left - 1) * a.x_row + kb);
    const i32x4 rw = row_rsrc4(a.w + g * a.w_stride, (int64_t)(nw - 1) * a.w_row + kb);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(
        (int)(uint32_t)(uintptr_t)(lds_byte*)lds + wave * 1024);

    // a wave's instruction i fills rows (i * 8 + wave) * 8 .. + 7
    const int sub = lane >> 3;
    const int chunk = (lane & 7) ^ ((((wave & 1) << 3 | sub) >> 1) & 7);
    uint32_t vx[4], vw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (i * 8 + wave) * 8 + sub;
        vx[i] = r < left ? (uint32_t)r * (uint32_t)a.x_row + chunk * 16 : kOutside;
        int n;
        const int q = wrow<GATED>(r, n0, a.N, n);
        vw[i] = n < a.N ? (uint32_t)q * (uint32_t)a.w_row + chunk * 16 : kOutside;
    }
    // the last slab may be short: its chunks past the end of k load zeros
    const int last = (kb - chunk * 16 + kSlab - 1) / kSlab;
    auto fetch = [&](int s) {
        const uint32_t none = s < last ? 0u : kOutside;
        const uint32_t d = lds0 + (s & 1) * 2 * kBigSlab;
#pragma unroll
        for (int i = 0; i < 4; ++i) load_to_lds(rx, d + i * 8192, vx[i] | none, s * kSlab);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load_to_lds(rw, d + kBigSlab + i * 8192, vw[i] | none, s * kSlab);
    };

    const int rd = (lane & 15) * kSlab + ((((lane >> 4) * 2) ^ ((lane >> 1) & 7)) * 16);
    const uint8_t* rdx = lds + wm * 128 * kSlab;
    const uint8_t* rdw = lds + kBigSlab + wn * 64 * kSlab;
    u32x4 fx[2][8], fw[2][4];
    auto read = [&](int s, int h, u32x4 (&x)[8], u32x4 (&w)[4]) {
        const int o = (s & 1) * 2 * kBigSlab + (rd ^ (h * 16));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const u32x4*>(rdw + o + i * 16 * kSlab);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = *reinterpret_cast<const u32x4*>(rdx + o + j * 16 * kSlab);
    };
    f32x4 acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const u32x4 (&x)[8], const u32x4 (&w)[4]) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, w[i]), __builtin_bit_cast(bf16x8, x[j]), acc[i][j],
                    0, 0, 0);
    };

    fetch(0);
    fetch(1);       // a slab past the last loads zeros
    asm volatile("s_waitcnt vmcnt(8)\n\ts_barrier" ::: "memory");
    read(0, 0, fx[0], fw[0]);
    // the reads of the half after, one to every two or three products
    auto spread = [&]() {
#pragma unroll
        for (int i = 0; i < 12; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);   // MFMA
        }
        __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
    };
    for (int s = 0; s < nslab; ++s) {
        read(s, 1, fx[1], fw[1]);
        multiply(fx[0], fw[0]);
        spread();
        // slab s is read; slab s + 1 has arrived
        wait_all_and_barrier();
        fetch(s + 2);
        read(s + 1, 0, fx[0], fw[0]);
        multiply(fx[1], fw[1]);
        spread();
        __builtin_amdgcn_sched_barrier(0);
    }
    wait_all_and_barrier();   // LDS is free for the next tile

#pragma unroll
    for (int i = 0; i < 4; i += GATED ? 2 : 1) {
        const int r = wn * 64 + i * 16 + (lane >> 4) * 4;
        int n;
        wrow<GATED>(r, n0, a.N, n);
        if (n >= a.N) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int m = wm * 128 + j * 16 + (lane & 15);
            if (m >= left) continue;
            const f32x4 y = finish<GATED>(a, g, n, acc[i][j], acc[GATED ? i + 1 : i][j]);
            store_out(a, g, m0 + m, n, y);
        }
    }
}

// The work list: big tiles of every group, then small ones. A group's rows
// are cut into runs of 256; what is left is a big tile too where it has more
// than `big_from` rows, else small tiles.
struct Plan {
    int32_t big[MOE_EP_MAX_LOCAL_EXPERTS + 1];      // tiles in front of a group
    int32_t small[MOE_EP_MAX_LOCAL_EXPERTS + 1];
};

__device__ __forceinline__ int big_runs(int rows, int big_from) {
    return rows / kBig + (rows % kBig > big_from ? 1 : 0);
}

template <int BM>
__device__ __forceinline__ void make_plan(const MatmulArgs& a, int big_from, int nt_big,
                                          int nt_small, Plan* p) {
    if (threadIdx.x < 64) {
        int32_t run_b = 0, run_s = 0;
        for (int g0 = 0; g0 < a.groups; g0 += 64) {
            const int g = g0 + (int)threadIdx.x;
            const int rows = g < a.groups ? group_rows(a, g) : 0;
            const int b = big_from < kBig ? big_runs(rows, big_from) : 0;
            const int rest = rows - b * kBig;
            const int32_t tb = b * nt_big;
            const int32_t ts = rest > 0 ? (rest + BM - 1) / BM * nt_small : 0;
            const int32_t ib = wave_inclusive_scan(tb), is = wave_inclusive_scan(ts);
            if (g < a.groups) {
                p->big[g] = run_b + ib - tb;
                p->small[g] = run_s + is - ts;
            }
            run_b += __shfl(ib, 63, 64);
            run_s += __shfl(is, 63, 64);
        }
        if (threadIdx.x == 0) {
            p->big[a.groups] = run_b;
            p->small[a.groups] = run_s;
        }
    }
    __syncthreads();
}

// Tile of block b in a round of `left` tiles over the grid, -1 for none.
// Blocks go to the eight XCDs in turn, so each XCD (with an L2 of its own)
// gets a run of neighbouring tiles, which share rows of x and w.
__device__ __forceinline__ int tile_of(int b, int grid, int left) {
    const int r = left < grid ? left : grid;
    const int per = (r + 7) / 8;
    const int slot = b >> 3;
    const int t = (b & 7) * per + slot;
    return slot < per && t < r ? t : -1;
}

template <int EB, bool GATED, int BM, int BN, int DEPTH, bool BIG>
__global__ __launch_bounds__(kThreads, 2) void matmul_kernel(const MatmulArgs a, int big_from) {
    constexpr int kSmallLds = kWaves * BM * (BN + 4) * 4;
    __shared__ __align__(1024) uint8_t lds[BIG && kBigLds > kSmallLds ? kBigLds : kSmallLds];
    __shared__ Plan p;
    constexpr int BO = GATED ? BN / 2 : BN;
    constexpr int BB = GATED ? kBig / 2 : kBig;
    const int nt = (a.N + BO - 1) / BO, ntb = (a.N + BB - 1) / BB;
    make_plan<BM>(a, BIG ? big_from : kBig, ntb, nt, &p);
    const int nbig = BIG ? uniform(p.big[a.groups]) : 0;
    const int total = nbig + uniform(p.small[a.groups]);
    for (int t0 = 0; t0 < total; t0 += gridDim.x) {
        const int at = tile_of(blockIdx.x, gridDim.x, total - t0);
        if (at < 0) break;      // a last, partial round
        const int t = t0 + at;
        if constexpr (BIG) {
            if (t < nbig) {
                const int g = uniform(find_source(p.big, a.groups, t));
                const int rows = uniform(group_rows(a, g));
                const int mt = big_runs(rows, big_from);
                // eight runs of rows at a time, over all columns
                const int l = t - uniform(p.big[g]);
                const int m8 = l / (8 * ntb) * 8;
                const int wide = mt - m8 < 8 ? mt - m8 : 8;
                const int in = l - m8 * ntb;
                big_tile<GATED>(a, g, (m8 + in % wide) * kBig, rows, in / wide * BB, lds);
                continue;
            }
        }
        const int l0 = t - nbig;
        const int g = uniform(find_source(p.small, a.groups, l0));
        const int rows = uniform(group_rows(a, g));
        const int from = BIG ? big_runs(rows, big_from) * kBig : 0;
        const int mt = (rows - from + BM - 1) / BM;
        const int l = l0 - uniform(p.small[g]);
        small_tile<EB, GATED, BM, BN, DEPTH>(a, g, from + l % mt * BM, rows, l / mt * BO,
                                             reinterpret_cast<float*>(lds));
    }
}

template <int EB, bool GATED, int BM, int BN, int DEPTH, bool BIG = false>
hipError_t launch(const MatmulArgs& a, hipStream_t st) {
    constexpr int BO = GATED ? BN / 2 : BN;
    const int64_t most = (int64_t)a.groups * ((a.rows + BM - 1) / BM) * ((a.N + BO - 1) / BO);
    const int64_t grid = most < 256 ? (most + 7) / 8 * 8 : 256;
    matmul_kernel<EB, GATED, BM, BN, DEPTH, BIG>
        <<<(unsigned)grid, kThreads, 0, st>>>(a, BIG ? 128 : kBig);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul(const MatmulArgs& a, hipStream_t st) {
    const bool gated = a.act == MOE_EP_ACT_SILU_GATED;
    if (a.fp8) {
        if (a.out_dtype == MOE_EP_E4M3)
            return gated ? launch<1, true, 16, 256, 1>(a, st) : launch<1, false, 16, 128, 2>(a, st);
        return gated ? launch<1, true, 64, 64, 1>(a, st) : launch<1, false, 64, 64, 1>(a, st);
    }
    if (a.rows > 128)
        return gated ? launch<2, true, 64, 64, 1, true>(a, st)
                     : launch<2, false, 64, 64, 1, true>(a, st);
    return gated ? launch<2, true, 64, 64, 1>(a, st) : launch<2, false, 64, 64, 1>(a, st);
}

}  // namespace moe_ep
