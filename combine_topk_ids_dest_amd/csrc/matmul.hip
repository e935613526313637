// Products of rows with weight matrices, grouped by expert with ragged row
// counts or over all tokens of a rank:
//   out[g][r][n] = act(sum_k x[g][r][k] * w[g][n][k] + bias[g][n]) + residual.
// Sums are fp32 in the matrix cores. x and w are both stored with k innermost,
// so both operands of an MFMA load the same way: a lane of a 16-row fragment
// takes two 16-byte chunks of row lane % 16 from every 128-byte slab of k (any
// assignment of k to lanes gives the same sum as long as both operands share
// it). w is the A operand: a lane's accumulators are consecutive output
// columns of one row of x, so the epilogue works on vectors.
//
// silu_gated: w holds N gate rows, then N up rows; a tile takes both rows of
// each of its output columns.
//
// fp8: a slab of 128 codes is one scale block: acc += (sx * sw) * slab sum. The
// codes are widened to bf16 (exactly) and multiplied there. The fp8 matrix
// instructions, of 32 and of 128 columns alike, drop product bits below 2^-13
// of the largest product they add: 448 * 448 - 448 * 448 and 126 ones come out
// as 120 (errors up to 9e-5 of the products' absolute sum were measured, in
// bf16 3e-7), and sums are held in 32 bits here whatever the result's type. In
// turn on one card, with the fp8 instruction and widened, bf16 results: 32
// experts of 15575 rows, 2048 -> 7168, 337 and 503 us; 8 experts of 917 rows, 30
// and 43; 8 experts of 480 rows, 7168 -> 2 x 2048, 50 and 82.
#include "product_tiles.h"

namespace moe_ep {
namespace {

// 32 e4m3 codes as bf16, in code order.
struct Wide {
    u32x4 v[4];
};

__device__ __forceinline__ Wide widen(const Frag& f) {
    Wide r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t c = f.v[i >> 2][i & 3];
        r.v[i >> 1][(i & 1) * 2] = __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
        r.v[i >> 1][(i & 1) * 2 + 1] = __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
    }
    return r;
}

__device__ __forceinline__ f32x4 mma_wide(const Wide& w, const Wide& x, f32x4 acc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = mma_bf16(w.v[i], x.v[i], acc);
    return acc;
}

// ---------------------------------------------------------------------
// Small tiles, for a few rows: 16 rows of x by 16 rows of w (gated: 8 gate
// rows and their 8 up rows). Bound by the weights' bytes, so what counts is
// loads in flight. A block's eight waves share out the slabs of k in runs of
// four (512 bytes of a row); each wave has its own four slabs of both operands
// in LDS, always on their way, with no barrier between them: behind the last
// slab of a tile it asks for the first of the block's next tile. The waves'
// sums are added in wave order through LDS.
//
// The way through LDS is for the loads' sake: an MFMA wants neighbouring lanes
// in different rows, and a load straight into that order takes 64 cycles for
// its 1 KB (one 16-byte piece at a time), which held a CU to 36 GB/s; eight
// neighbouring lanes to a row's 128 bytes take a quarter of that.
// ---------------------------------------------------------------------
constexpr int kSmallPitch = kSmall + 4;
constexpr int kRun = 4;                          // slabs of a wave in LDS
constexpr int kRing = kRun * 2 * kSmall * kSlab; // bytes of them
constexpr int kPartAt = kWaves * kRing;          // the waves' sums, twice
constexpr int kPart = kWaves * kSmall * kSmallPitch * 4;
constexpr int kSmallScaleAt = kPartAt + 2 * kPart;        // fp8: scales of two runs
constexpr int kSmallLds = kSmallScaleAt + kWaves * 2 * 512;

// What a wave needs to load a small tile.
struct SmallTile {
    i32x4 rx, rw, rxs, rws;
    uint32_t vx[2], vw[2], vxs, vws;
    int g, m0, rows, n0;
};

template <int EB, bool GATED>
__device__ __forceinline__ SmallTile small_setup(const MatmulArgs& a, int g, int m0, int rows,
                                                 int n0) {
    SmallTile t;
    const int lane = threadIdx.x & 63;
    const int kb = a.row_bytes;
    const int nslab = (kb + kSlab - 1) / kSlab;
    const int left = rows - m0;
    const int nw = GATED ? 2 * a.N : a.N;
    t.g = g;
    t.m0 = m0;
    t.rows = rows;
    t.n0 = n0;
    t.rx = row_rsrc4(a.x + g * a.x_stride + (int64_t)m0 * a.x_row,
                     (int64_t)(left - 1) * a.x_row + kb);
    t.rw = row_rsrc4(a.w + g * a.w_stride, (int64_t)(nw - 1) * a.w_row + kb);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = h * 8 + (lane >> 3);
        const uint32_t chunk = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
        t.vx[h] = r < left ? (uint32_t)r * (uint32_t)a.x_row + chunk : kOutside;
        const int n = GATED ? n0 + (r & 7) : n0 + r;
        t.vw[h] = n < a.N ? (uint32_t)(GATED && r >= 8 ? a.N + n : n) * (uint32_t)a.w_row + chunk
                          : kOutside;
    }
    t.rxs = t.rx;
    t.rws = t.rw;
    t.vxs = t.vws = kOutside;
    if constexpr (EB == 1) {
        // lane r: four scales of row r; lanes 4 b + i: block b's of slab i
        if (lane < 16 && lane < left) t.vxs = (uint32_t)lane * (uint32_t)a.xs_pitch * 4;
        t.rxs = row_rsrc4(
            reinterpret_cast<const uint8_t*>(a.xs + g * a.xs_stride + (int64_t)m0 * a.xs_pitch),
            (int64_t)left * a.xs_pitch * 4);
        const int per = (a.N + kScaleBlock - 1) / kScaleBlock;
        const int b = lane >> 2;
        if (b < (GATED ? 2 : 1))
            t.vws = ((uint32_t)(n0 / kScaleBlock + b * per) * (uint32_t)nslab + (lane & 3)) * 4;
        t.rws = row_rsrc4(reinterpret_cast<const uint8_t*>(a.ws + g * a.ws_stride),
                          (int64_t)(GATED ? 2 : 1) * per * nslab * 4);
    }
    return t;
}

// Slab s of a tile into place j of the wave's ring (a slab past the last: zeros).
__device__ __forceinline__ void small_fetch(const MatmulArgs& a, const SmallTile& t, int s, int j,
                                            uint32_t ring) {
    const int lane = threadIdx.x & 63;
    const int kb = a.row_bytes;
    const uint32_t k = s * kSlab < kb ? s * kSlab : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int chunk = ((lane & 7) ^ ((h * 4 + (lane >> 4)) & 7)) * 16;
        const uint32_t none = s * kSlab + chunk < kb ? 0u : kOutside;
        const uint32_t at = ring + j * 2 * kSmall * kSlab + h * 1024;
        load_to_lds(uniform(t.rw), at, t.vw[h] | none, k);
        // the last eight rows of x only where there are any (what LDS holds
        // there else belongs to sums that are not stored)
        if (h == 0 || t.rows - t.m0 > 8)
            load_to_lds(uniform(t.rx), at + kSmall * kSlab, t.vx[h] | none, k);
    }
}

// The scales of the four slabs from s on (a multiple of 4).
__device__ __forceinline__ void small_fetch_scales(const MatmulArgs& a, const SmallTile& t, int s,
                                                   uint32_t at) {
    const int nslab = (a.row_bytes + kSlab - 1) / kSlab;
    const uint32_t k = s < nslab ? s * 4 : 0;
    const uint32_t none = s < nslab ? 0u : kOutside;
    if ((threadIdx.x & 63) < 16) load_to_lds(uniform(t.rxs), at, t.vxs | none, k);
    if ((threadIdx.x & 63) < 16)
        load4_to_lds(uniform(t.rws), at + 256, s + (int)(threadIdx.x & 3) < nslab ? t.vws : kOutside, k);
}

// Works through the block's tiles, number t of `total` at place(t) = {g, m0,
// rows, n0}.
template <int EB, bool GATED, class Next>
__device__ __forceinline__ void small_tiles(const MatmulArgs& a, uint8_t* lds, int total,
                                            const Next& place) {
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int kb = a.row_bytes;
    const int nslab = (kb + kSlab - 1) / kSlab;
    const int runs = (nslab + kWaves * kRun - 1) / (kWaves * kRun);   // of each wave
    const uint32_t lds0 = uniform((int)(uint32_t)(uintptr_t)(lds_byte*)lds);
    const uint32_t ring = lds0 + wave * kRing;
    const uint32_t scales = lds0 + kSmallScaleAt + wave * 1024;
    const uint8_t* mine = lds + wave * kRing;
    const int r = lane & 15;
    const int rd = r * kSlab + (((lane >> 4) ^ ((r >> 1) & 7)) * 16);

    auto tile_at = [&](int t0) {
        const int t = t0 < total ? tile_of(blockIdx.x, gridDim.x, total - t0) : -1;
        return t < 0 ? -1 : t + t0;
    };
    int t0 = 0, at = tile_at(0);
    if (at < 0) return;
    SmallTile cur = place(at);
    if constexpr (EB == 1) small_fetch_scales(a, cur, wave * kRun, scales);
#pragma unroll
    for (int j = 0; j < kRun; ++j) small_fetch(a, cur, wave * kRun + j, j, ring);
    int odd = 0, run = 0;                        // parity of the tile and of the run
    for (;;) {
        t0 += gridDim.x;
        at = tile_at(t0);
        SmallTile nxt = cur;
        if (at >= 0) nxt = place(at);
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < runs; ++i) {
            const bool ahead = i + 1 < runs;     // the next run is this tile's
            const int s1 = at >= 0 || ahead ? ((ahead ? i + 1 : 0) * kWaves + wave) * kRun
                                            : nslab;
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                // the oldest slab has arrived (and, before it, its run's scales):
                // behind it are three slabs of three or four loads
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kRun - 1) * 3) : "memory");
                const uint8_t* p = mine + j * 2 * kSmall * kSlab;
                Frag w, x;
                w.v[0] = *reinterpret_cast<const u32x4*>(p + rd);
                w.v[1] = *reinterpret_cast<const u32x4*>(p + (rd ^ 64));
                x.v[0] = *reinterpret_cast<const u32x4*>(p + kSmall * kSlab + rd);
                x.v[1] = *reinterpret_cast<const u32x4*>(p + kSmall * kSlab + (rd ^ 64));
                float sc = 0.f;
                if constexpr (EB == 1) {
                    const float* q = reinterpret_cast<const float*>(lds + kSmallScaleAt + wave * 1024 +
                                                                    run * 512);
                    sc = q[r * 4 + j] * q[64 + (GATED && lane >= 32 ? 4 : 0) + j];
                    // a scale row's padding may hold anything
                    if ((i * kWaves + wave) * kRun + j >= nslab) sc = 0.f;
                }
                // read, so its place can be filled again
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if constexpr (EB == 1) {
                    if (j == 0) small_fetch_scales(a, ahead ? cur : nxt, s1, scales + (run ^ 1) * 512);
                }
                if (ahead) small_fetch(a, cur, s1 + j, j, ring);
                else small_fetch(a, nxt, s1 + j, j, ring);
                if constexpr (EB == 2) {
                    acc = mma_bf16(w.v[0], x.v[0], acc);
                    acc = mma_bf16(w.v[1], x.v[1], acc);
                } else {
                    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                    const f32x4 t = mma_wide(widen(w), widen(x), zero);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[q] = __builtin_fmaf(t[q], sc, acc[q]);
                }
            }
            run ^= 1;
        }

        float* part = reinterpret_cast<float*>(lds + kPartAt + odd * kPart);
        *reinterpret_cast<f32x4*>(part + ((wave * kSmall + r) * kSmallPitch + (lane >> 4) * 4)) = acc;
        // the waves' sums are written; loads stay in flight
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        constexpr int BO = GATED ? kSmall / 2 : kSmall;
        const int o = threadIdx.x % BO, m = threadIdx.x / BO;
        const int n = cur.n0 + o;
        if (m < kSmall && cur.m0 + m < cur.rows && n < a.N) {
            float v = 0.f, up = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                v += part[(w * kSmall + m) * kSmallPitch + o];
                if (GATED) up += part[(w * kSmall + m) * kSmallPitch + o + 8];
            }
            if (a.bias) {
                const float* b = a.bias + cur.g * a.bias_stride + n;
                v += b[0];
                if (GATED) up += b[a.N];
            }
            v = GATED ? silu_gated(v, up) : apply_act(v, a.act);
            const bool f32 = a.out_dtype == MOE_EP_F32;
            const int64_t row = cur.m0 + m;
            if (a.res) {
                const uint8_t* q = a.res + row * a.res_row;
                v += f32 ? reinterpret_cast<const float*>(q)[n]
                         : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(q)[n] << 16);
            }
            uint8_t* p = a.out + cur.g * a.out_stride + row * a.out_row;
            if (f32) reinterpret_cast<float*>(p)[n] = v;
            else reinterpret_cast<uint16_t*>(p)[n] = (uint16_t)to_bf16_rne(v);
        }
        if (at < 0) break;
        cur = nxt;
        odd ^= 1;
    }
    // nothing of this block's is on its way into LDS when the block ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ---------------------------------------------------------------------
// Big tiles: BM (128 to 256) rows of x by 256 rows of w. Eight waves in
// two rows of four, each with BM / 2 x 64 of the sums in registers. Slabs of
// 128 bytes of k go from memory straight into LDS (no register is spent on a
// load in flight), one to three slabs ahead of the one being multiplied.
//
// LDS: row r of a slab holds its eight 16-byte chunks with chunk c at place
// c ^ ((r >> 1) & 7), and lane l of a fragment takes the chunks l / 16 and
// l / 16 + 4 of row l % 16. A 16-byte read is served 16 lanes at a time,
// lanes 0-3, 12-15, 20-27 first and 4-11, 16-19, 28-31 next (then the same of
// the upper half): both sets fall on all 64 banks. (With chunks 2 (l / 16) and
// the one after, every read met a conflict: 8 cycles instead of 4.) The load
// that fills LDS writes a wave's 64 x 16 bytes in lane order, so the
// permutation is applied to the addresses that the lanes read.
//
// The 64 rows of w of a wave are permuted so that a lane's sums are 16
// consecutive output columns (gated: 8): see wrow().
// ---------------------------------------------------------------------
constexpr int kBig = 256;                        // rows of w
constexpr int kBigSlab = kBig * kSlab;
constexpr int kLds = 160 << 10;                  // all of a CU's
constexpr int kScaleLds = 2 * (kBig * 16 + 256); // fp8: two sets of scales of four slabs
constexpr int kScaleAt = kLds - kScaleLds;

// Slabs of x and of w in LDS: as many as fit. Weights of experts come from
// HBM, x more often from L2, so where one of the two can be deeper it is w.
// (256 rows: with two slabs of each, a slab's time is below HBM's loaded
// latency of about 2 us, and the products wait for the weights.)
template <int EB, int BM>
constexpr int kStagesX = BM > 128 ? 2 : 3;
template <int EB, int BM>
constexpr int kStagesW = EB == 2 ? 3 : BM > 128 ? 2 : 3;

// fp8: a tile's scales in LDS, of four slabs at a time: 16 bytes per row of x,
// and 4 bytes per slab and block of w (two: runs of 128 columns, or gate and
// up). Slab s's set is s / 4 & 1.
template <int EB, bool GATED>
struct TileScales {
    static constexpr int kSet = kBig * 16 + 256;
    i32x4 rx, rw;
    uint32_t lds0;
    int nslab, wave, left, pitch, per, n0, N;

    __device__ __forceinline__ TileScales(const MatmulArgs& a, int g, int m0, int left_, int n0_,
                                          uint32_t lds) {
        if constexpr (EB == 1) {
            wave = uniform(threadIdx.x >> 6);
            lds0 = lds + kScaleAt;
            nslab = a.row_bytes / kSlab;
            left = left_;
            pitch = (int)a.xs_pitch * 4;
            n0 = n0_;
            N = a.N;
            per = (N + kScaleBlock - 1) / kScaleBlock;
            rx = row_rsrc4(reinterpret_cast<const uint8_t*>(a.xs + g * a.xs_stride +
                                                            (int64_t)m0 * a.xs_pitch),
                           (int64_t)left * pitch);
            rw = row_rsrc4(reinterpret_cast<const uint8_t*>(a.ws + g * a.ws_stride),
                           (int64_t)(GATED ? 2 : 1) * per * nslab * 4);
        }
    }

    // The four slabs from s on (a multiple of 4). The lanes' addresses are made
    // here: one register held over the loop too many is one spilled, and to
    // load it back waits for every load in flight.
    __device__ __forceinline__ void fetch(int s) const {
        const int lane = threadIdx.x & 63;
        const uint32_t d = lds0 + ((s >> 2) & 1) * kSet;
        const uint32_t k = s < nslab ? s * 4 : 0;
        if (wave < kBig / 64) {
            const int row = wave * 64 + lane;
            load_to_lds(rx, d + wave * 1024,
                        s < nslab && row < left ? (uint32_t)row * (uint32_t)pitch : kOutside, k);
        }
        if (wave == kWaves - 1) {
            const int b = lane >> 2;
            const int n = n0 + (GATED ? 0 : b * kScaleBlock);
            const uint32_t at =
                ((uint32_t)(n / kScaleBlock + (GATED ? b * per : 0)) * (uint32_t)nslab + (lane & 3)) *
                4;
            load4_to_lds(rw, d + kBig * 16,
                         b < 2 && n < N && s + (lane & 3) < nslab ? at : kOutside, k);
        }
    }

    // slab s's: row r's of x at [4 r + s % 4], block b's at [4 kBig + 4 b + s % 4]
    __device__ __forceinline__ const float* at(const uint8_t* lds, int s) const {
        return reinterpret_cast<const float*>(lds + kScaleAt + ((s >> 2) & 1) * kSet);
    }
};

template <int EB, bool GATED, int BM>
__device__ __forceinline__ void big_tile(const MatmulArgs& a, int g, int m0, int rows, int n0,
                                         uint8_t* lds) {
    constexpr int JF = BM / 32;                   // fragments of x of a wave
    constexpr int XS = kStagesX<EB, BM>, WS = kStagesW<EB, BM>;
    constexpr int FX = (BM + 63) / 64;            // loads of x of a wave and slab
    constexpr int SLAB_X = FX * 64 * kSlab;
    constexpr int AT_W = XS * SLAB_X;             // slabs of w behind those of x
    constexpr int FETCH = FX + 4;
    static_assert(XS <= WS && AT_W + WS * kBigSlab <= (EB == 1 ? kScaleAt : kLds), "");
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int kb = a.row_bytes;
    const int nslab = (kb + kSlab - 1) / kSlab;
    const int left = rows - m0 < BM ? rows - m0 : BM;
    const int nw = GATED ? 2 * a.N : a.N;
    const i32x4 rx = row_rsrc4(a.x + g * a.x_stride + (int64_t)m0 * a.x_row,
                               (int64_t)(left - 1) * a.x_row + kb);
    const i32x4 rw = row_rsrc4(a.w + g * a.w_stride, (int64_t)(nw - 1) * a.w_row + kb);
    const uint32_t lds0 = uniform((int)(uint32_t)(uintptr_t)(lds_byte*)lds);

    // a wave's load i fills rows (i * 8 + wave) * 8 .. + 7
    const int sub = lane >> 3;
    const int chunk = (lane & 7) ^ ((((wave & 1) << 3 | sub) >> 1) & 7);
    // Rows 64 apart: one offset for x and one for w, and how many of the loads
    // have a row (in one register, with four bits each). Offsets for every load
    // are five registers more, and the loop has none to spare: what it spills
    // it waits for, behind all loads in flight.
    const int row = wave * 8 + sub;
    int n;
    const int wr = wrow<GATED, 4>(row, n0, a.N, n);
    const uint32_t vx = (uint32_t)row * (uint32_t)a.x_row + chunk * 16;
    const uint32_t vw = (uint32_t)wr * (uint32_t)a.w_row + chunk * 16;
    constexpr int STEP_N = GATED ? 32 : 64;       // output columns of 64 rows of w
    const int have_x = left > row ? (left - row + 63) / 64 : 0;
    const int have_w = a.N > n ? (a.N - n + STEP_N - 1) / STEP_N : 0;
    const int have = (have_x < 8 ? have_x : 8) | (have_w < 8 ? have_w : 8) << 4;
    const uint32_t step_x = 64u * (uint32_t)a.x_row, step_w = (uint32_t)STEP_N * (uint32_t)a.w_row;
    // the last slab may be short: its chunks past the end of k load zeros, and
    // so do slabs past the last
    const int last = (kb - chunk * 16 + kSlab - 1) / kSlab;
    auto fetch_x = [&](int i, int s, int stage) {
        load_to_lds(rx, lds0 + stage * SLAB_X + wave * 1024 + i * 8192,
                    s < last && i < (have & 15) ? vx + i * step_x : kOutside,
                    s < nslab ? s * kSlab : 0);
    };
    auto fetch_w = [&](int i, int s, int stage) {
        load_to_lds(rw, lds0 + AT_W + stage * kBigSlab + wave * 1024 + i * 8192,
                    s < last && i < have >> 4 ? vw + i * step_w : kOutside,
                    s < nslab ? s * kSlab : 0);
    };

    const TileScales<EB, GATED> scales(a, g, m0, left, n0, lds0);

    const int rd = (lane & 15) * kSlab + (((lane >> 4) ^ ((lane >> 1) & 7)) * 16);
    const uint8_t* rdx = lds + wm * (JF * 16) * kSlab;
    const uint8_t* rdw = lds + AT_W + wn * 64 * kSlab;
    f32x4 acc[4][JF];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < JF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // The order of the loads is that of a loop started WS slabs early: step v
    // loads slab v + XS of x, then slab v + WS of w.
    if constexpr (EB == 1) scales.fetch(0);
#pragma unroll
    for (int v = -WS; v < (EB == 2 ? 0 : -1); ++v) {
#pragma unroll
        for (int i = 0; i < FX; ++i)
            if (v + XS >= 0) fetch_x(i, v + XS, v + XS);
#pragma unroll
        for (int i = 0; i < 4; ++i) fetch_w(i, v + WS, v + WS);
    }
    // Loads behind those of slab s + 1 when step s waits for it.
    constexpr int LEFT = (XS - 2) * FETCH + (WS > XS ? 4 : 0);

    if constexpr (EB == 2) {
        // Fragments are read half a slab ahead, so that the reads of one half
        // run under the products of the other.
        u32x4 fx[2][JF], fw[2][4];
        // Multiplies one half while reading half h of the slab at stages ix
        // and iw, and with FETCHES does step f's loads, in small steps: a wave
        // issues in order.
        auto step = [&](const u32x4 (&x)[JF], const u32x4 (&w)[4], int ix, int iw, int h,
                        u32x4 (&nx)[JF], u32x4 (&nwf)[4], auto fetches, int f, int tx, int tw) {
            const int o = rd ^ (h * 64);
#pragma unroll
            for (int j = 0; j < JF; ++j) {
                if constexpr (decltype(fetches)::value) {
#pragma unroll
                    for (int i = j * FETCH / JF; i < (j + 1) * FETCH / JF; ++i) {
                        if (i < FX) fetch_x(i, f + XS, tx);
                        else fetch_w(i - FX, f + WS, tw);
                    }
                }
#pragma unroll
                for (int i = j * 4 / JF; i < (j + 1) * 4 / JF; ++i)
                    nwf[i] = *reinterpret_cast<const u32x4*>(rdw + iw * kBigSlab + o + i * 16 * kSlab);
                nx[j] = *reinterpret_cast<const u32x4*>(rdx + ix * SLAB_X + o + j * 16 * kSlab);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = mma_bf16(w[i], x[j], acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        wait_and_barrier<LEFT + FETCH>();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            fw[0][i] = *reinterpret_cast<const u32x4*>(rdw + rd + i * 16 * kSlab);
#pragma unroll
        for (int j = 0; j < JF; ++j)
            fx[0][j] = *reinterpret_cast<const u32x4*>(rdx + rd + j * 16 * kSlab);
        int ix = 0, iw = 0;                       // stages of slab s
        for (int s = 0; s < nslab; ++s) {
            step(fx[0], fw[0], ix, iw, 1, fx[1], fw[1], std::false_type{}, 0, 0, 0);
            // slab s is read; slab s + 1 has arrived
            wait_and_barrier<LEFT>();
            const int nix = ix + 1 < XS ? ix + 1 : 0, niw = iw + 1 < WS ? iw + 1 : 0;
            step(fx[1], fw[1], nix, niw, 0, fx[0], fw[0], std::true_type{}, s, ix, iw);
            ix = nix;
            iw = niw;
        }
    } else {
        // Slab by slab: the sums of a slab are complete before they are
        // scaled, so the halves cannot be taken apart.
        const int bw = GATED ? 0 : wn >> 1;       // the wave's block (gated: both)
        static_assert(XS == WS, "");
        // A register loaded in front of the loop (a spilled one) is waited for
        // at its first use in the loop, in every round, and with it all loads
        // into LDS: wait for it here, in a form that the compiler sees (vmcnt 0).
        __builtin_amdgcn_s_waitcnt(0x0F70);
        int now = 0;
        for (int s = 0; s < nslab; ++s) {
            // slab s and its scales (older than the loads that may still be
            // in flight) have arrived; slab s - 1 is read
            wait_and_barrier<LEFT>();
            const int to = now == 0 ? XS - 1 : now - 1;
#pragma unroll
            for (int i = 0; i < FX; ++i) fetch_x(i, s + XS - 1, to);
#pragma unroll
            for (int i = 0; i < 4; ++i) fetch_w(i, s + WS - 1, to);
            if ((s & 3) == 2) scales.fetch((s & ~3) + 4);
            const float* sc = scales.at(lds, s);
            const float sg = sc[kBig * 4 + bw * 4 + (s & 3)];
            const float su = GATED ? sc[kBig * 4 + 4 + (s & 3)] : sg;
            auto frag = [&](const uint8_t* p) {
                Frag f;
                f.v[0] = *reinterpret_cast<const u32x4*>(p + rd);
                f.v[1] = *reinterpret_cast<const u32x4*>(p + (rd ^ 64));
                return f;
            };
            const uint8_t* px = rdx + now * SLAB_X;
            const uint8_t* pw = rdw + now * kBigSlab;
            auto scale = [&](int i, int j, f32x4 t, float sx) {
                const float f = sx * (GATED && (i & 1) ? su : sg);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(t[q], f, acc[i][j][q]);
            };
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            Wide w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = widen(frag(pw + i * 16 * kSlab));
#pragma unroll
            for (int j = 0; j < JF; ++j) {
                const Wide x = widen(frag(px + j * 16 * kSlab));
                const float sx = sc[(wm * (JF * 16) + j * 16 + (lane & 15)) * 4 + (s & 3)];
                // two chains of products at a time: each waits for its own sum
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    f32x4 t0 = zero, t1 = zero;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        t0 = mma_bf16(w[i].v[q], x.v[q], t0);
                        t1 = mma_bf16(w[i + 1].v[q], x.v[q], t1);
                    }
                    scale(i, j, t0, sx);
                    scale(i + 1, j, t1, sx);
                }
            }
            now = now + 1 < XS ? now + 1 : 0;
        }
    }
    wait_and_barrier<0>();   // LDS is free for what follows
    finish_tile<EB, GATED, 4, JF, 4>(a, g, m0, left, n0, acc, lds);
}

// ---------------------------------------------------------------------
// Narrow tiles: up to 64 rows of x by 256 rows of w, bound by the weights'
// bytes. HBM gives runs of 128 bytes of many rows at 4 to 5 TB/s and runs of
// 256 bytes at 6 (measured with plain loads of 470 MB), so here k goes by
// pairs of slabs, and to fit that into LDS with loads in flight the rows of w
// go by halves: unit u is half u % 2 (fragments 2 h and 2 h + 1 of each wave)
// of pair u / 2, 128 rows of 256 bytes. Two or three units are on their way
// while one is multiplied; the fragments of x stay in registers for both
// halves of a pair.
//
// LDS: chunk c of a 256-byte row r is at place c ^ (r & 15): the sets of 16
// lanes named above meet on no bank.
// ---------------------------------------------------------------------
constexpr int kNarrow = 64;
constexpr int kPair = 2 * kSlab;
constexpr int kPairX = kNarrow * kPair;
constexpr int kUnit = 128 * kPair;

template <int EB, bool GATED>
__device__ __forceinline__ void narrow_tile(const MatmulArgs& a, int g, int m0, int rows, int n0,
                                            uint8_t* lds) {
    constexpr int JF = 2;
    constexpr int WU = EB == 2 ? 4 : 3;           // units of w in LDS
    constexpr int AT_W = 2 * kPairX;              // behind two pairs of x
    static_assert(AT_W + WU * kUnit <= (EB == 1 ? kScaleAt : kLds), "");
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int kb = a.row_bytes;
    const int nslab = (kb + kSlab - 1) / kSlab;
    const int npair = (nslab + 1) / 2;
    const int left = rows - m0 < kNarrow ? rows - m0 : kNarrow;
    const int nw = GATED ? 2 * a.N : a.N;
    const i32x4 rx = row_rsrc4(a.x + g * a.x_stride + (int64_t)m0 * a.x_row,
                               (int64_t)(left - 1) * a.x_row + kb);
    const i32x4 rw = row_rsrc4(a.w + g * a.w_stride, (int64_t)(nw - 1) * a.w_row + kb);
    const uint32_t lds0 = uniform((int)(uint32_t)(uintptr_t)(lds_byte*)lds);

    // a wave's load i fills rows (i * 8 + wave) * 4 .. + 3
    const int sub = lane >> 4;
    const uint32_t chunk = ((lane & 15) ^ ((wave & 3) * 4 + sub)) * 16;
    uint32_t vx[2], vw[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (i * 8 + wave) * 4 + sub;
        if (i < 2) vx[i] = r < left ? (uint32_t)r * (uint32_t)a.x_row + chunk : kOutside;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int n;
            const int q = wrow<GATED, 4>((r >> 5) * 64 + h * 32 + (r & 31), n0, a.N, n);
            vw[h][i] = n < a.N ? (uint32_t)q * (uint32_t)a.w_row + chunk : kOutside;
        }
    }
    auto fetch_x = [&](int p) {
        const uint32_t none = p * kPair + (int)chunk < kb ? 0u : kOutside;
        const uint32_t k = p * kPair < kb ? p * kPair : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            load_to_lds(rx, lds0 + (p & 1) * kPairX + (i * 8 + wave) * 1024, vx[i] | none, k);
    };
    auto fetch_w = [&](int p, int h, int slot) {
        const uint32_t none = p * kPair + (int)chunk < kb ? 0u : kOutside;
        const uint32_t k = p * kPair < kb ? p * kPair : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load_to_lds(rw, lds0 + AT_W + slot * kUnit + (i * 8 + wave) * 1024, vw[h][i] | none, k);
    };
    const TileScales<EB, GATED> scales(a, g, m0, left, n0, lds0);

    const int r = lane & 15;
    const int rd = r * kPair + (((lane >> 4) ^ r) * 16);
    const uint8_t* rdx = lds + wm * 32 * kPair;
    const uint8_t* rdw = lds + AT_W + wn * 32 * kPair;
    f32x4 acc[4][JF];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < JF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // The order of the loads is that of a loop started three units early: odd
    // units load x of the pair after the next, then every unit w of the unit
    // WU - 1 ahead.
    if constexpr (EB == 1) scales.fetch(0);
    fetch_x(0);
    fetch_w(0, 0, 0);
    if (WU == 4) fetch_w(0, 1, 1);
    fetch_x(1);
    if (WU == 4) fetch_w(1, 0, 2);
    else fetch_w(0, 1, 1);
    int slot = 0;                                 // of unit u
    u32x4 x[JF][4];
    for (int p = 0; p < npair; ++p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // unit u (and x of its pair, older) has arrived: behind it are the
            // units after it and the x asked for between them
            if (h == 0) wait_and_barrier<WU == 4 ? 10 : 6>();
            else wait_and_barrier<WU == 4 ? 10 : 4>();
            const int to = slot == 0 ? WU - 1 : slot - 1;
            if (EB == 1 && h == 0 && (p & 1)) scales.fetch(2 * (p + 1));
            if (h == 1) fetch_x(p + 2);
            if (WU == 4) fetch_w(h == 0 ? p + 1 : p + 2, 1 - h, to);
            else fetch_w(p + 1, h, to);
            if (h == 0) {
#pragma unroll
                for (int j = 0; j < JF; ++j)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        x[j][t] = *reinterpret_cast<const u32x4*>(
                            rdx + (p & 1) * kPairX + j * 16 * kPair + (rd ^ (t * 64)));
            }
            u32x4 w[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    w[i][t] = *reinterpret_cast<const u32x4*>(rdw + slot * kUnit + i * 16 * kPair +
                                                              (rd ^ (t * 64)));
            if constexpr (EB == 2) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < JF; ++j)
                            acc[2 * h + i][j] = mma_bf16(w[i][t], x[j][t], acc[2 * h + i][j]);
            } else {
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const int sl = 2 * p + d;
                    const float* sc = scales.at(lds, sl);
                    const bool in = sl < nslab;   // a scale row's padding may hold anything
                    Frag f[2], fx[JF];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        f[i].v[0] = w[i][2 * d];
                        f[i].v[1] = w[i][2 * d + 1];
                    }
#pragma unroll
                    for (int j = 0; j < JF; ++j) {
                        fx[j].v[0] = x[j][2 * d];
                        fx[j].v[1] = x[j][2 * d + 1];
                        const float sx = sc[(wm * 32 + j * 16 + r) * 4 + (sl & 3)];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                            const f32x4 t = mma_wide(widen(f[i]), widen(fx[j]), zero);
                            const float b = sc[kBig * 4 + (GATED ? i : wn >> 1) * 4 + (sl & 3)];
                            const float v = in ? sx * b : 0.f;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                acc[2 * h + i][j][q] =
                                    __builtin_fmaf(t[q], v, acc[2 * h + i][j][q]);
                        }
                    }
                }
            }
            slot = slot + 1 < WU ? slot + 1 : 0;
        }
    }
    wait_and_barrier<0>();   // LDS is free for what follows
    finish_tile<EB, GATED, 4, JF, 4>(a, g, m0, left, n0, acc, lds);
}

// ---------------------------------------------------------------------
// Middle tiles, for products whose 256-column tiles would leave most CUs idle
// (the router's logits, some rows of a few experts): 64 rows of x by 64 of w
// or 128 by 128, rings of pairs of slabs. What they reach goes by the bytes of
// weights on their way (HBM's latency under load is about 3 us): four pairs of
// 16 KB of a CU give 5.5 TB/s, three 3.7. Half of the waves load x, half w: a
// wave's loads complete in order, so a wave that loaded both would wait for the
// weights of pairs to come before the rows of the pair at hand, which come from
// nearer.
// ---------------------------------------------------------------------
template <bool GATED, int BM>
__device__ __forceinline__ void mid_tile(const MatmulArgs& a, int g, int m0, int rows, int n0,
                                         uint8_t* lds) {
    constexpr int WN = BM == 64 ? 2 : 4;          // waves over the rows of w
    constexpr int JF = BM * WN / 128;             // fragments of x of a wave
    constexpr int XR = BM == 64 ? 5 : 2, WR = BM == 64 ? 5 : 3;     // pairs in LDS
    constexpr int NX = BM / 16;                   // loads of a wave per pair, of x or w
    constexpr int PAIR = BM * kPair;
    constexpr int AT_W = XR * PAIR;
    static_assert(AT_W + WR * PAIR <= kLds, "");
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const bool is_x = wave < 4;
    const int kb = a.row_bytes;
    const int npair = (kb + kPair - 1) / kPair;
    const int left = rows - m0 < BM ? rows - m0 : BM;
    const int nw = GATED ? 2 * a.N : a.N;
    const i32x4 rx = row_rsrc4(a.x + g * a.x_stride + (int64_t)m0 * a.x_row,
                               (int64_t)(left - 1) * a.x_row + kb);
    const i32x4 rw = row_rsrc4(a.w + g * a.w_stride, (int64_t)(nw - 1) * a.w_row + kb);
    const i32x4 rs = is_x ? rx : rw;
    const uint32_t lds0 = uniform((int)(uint32_t)(uintptr_t)(lds_byte*)lds);

    // a wave's load i fills rows (i * 4 + wave % 4) * 4 .. + 3
    const int sub = lane >> 4;
    const uint32_t chunk = ((lane & 15) ^ ((wave & 3) * 4 + sub)) * 16;
    uint32_t v[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int r = (i * 4 + (wave & 3)) * 4 + sub;
        if (is_x) {
            v[i] = r < left ? (uint32_t)r * (uint32_t)a.x_row + chunk : kOutside;
        } else {
            int n;
            const int q = wrow<GATED, 2>(r, n0, a.N, n);
            v[i] = n < a.N ? (uint32_t)q * (uint32_t)a.w_row + chunk : kOutside;
        }
    }
    const int ahead = (is_x ? XR : WR) - 1;
    const uint32_t ring = lds0 + (is_x ? 0 : AT_W) + (wave & 3) * 1024;
    auto fetch = [&](int p, int slot) {
        const uint32_t none = p * kPair + (int)chunk < kb ? 0u : kOutside;
        const uint32_t k = p * kPair < kb ? p * kPair : 0;
#pragma unroll
        for (int i = 0; i < NX; ++i)
            load_to_lds(rs, ring + slot * PAIR + i * 4096, v[i] | none, k);
    };
    const int r = lane & 15;
    const int rd = r * kPair + (((lane >> 4) ^ r) * 16);
    const uint8_t* rdx = lds + wm * JF * 16 * kPair;
    const uint8_t* rdw = lds + AT_W + wn * 32 * kPair;
    f32x4 acc[2][JF];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < JF; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < ahead; ++p) fetch(p, p);
    int ix = 0, iw = 0;                           // slots of pair p
    for (int p = 0; p < npair; ++p) {
        // pair p has arrived; p - 1 is read
        if (is_x) wait_and_barrier<(XR - 2) * NX>();
        else wait_and_barrier<(WR - 2) * NX>();
        fetch(p + ahead, is_x ? (ix == 0 ? XR - 1 : ix - 1) : (iw == 0 ? WR - 1 : iw - 1));
        u32x4 x[JF][4], w[2][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int j = 0; j < JF; ++j)
                x[j][t] = *reinterpret_cast<const u32x4*>(rdx + ix * PAIR + j * 16 * kPair +
                                                          (rd ^ (t * 64)));
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i][t] = *reinterpret_cast<const u32x4*>(rdw + iw * PAIR + i * 16 * kPair +
                                                          (rd ^ (t * 64)));
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < JF; ++j) acc[i][j] = mma_bf16(w[i][t], x[j][t], acc[i][j]);
        ix = ix + 1 < XR ? ix + 1 : 0;
        iw = iw + 1 < WR ? iw + 1 : 0;
    }
    wait_and_barrier<0>();   // LDS is free for the next tile
    finish_tile<2, GATED, 2, JF, WN>(a, g, m0, left, n0, acc, lds);
}

template <bool GATED, int BM>
__global__ __launch_bounds__(kThreads, 2) void mid_kernel(const MatmulArgs a) {
    __shared__ __align__(1024) uint8_t lds[kLds];
    constexpr int BO = GATED ? BM / 2 : BM;
    const int mt = (a.rows + BM - 1) / BM;
    const int total = mt * ((a.N + BO - 1) / BO);
    for (int t0 = 0; t0 < total; t0 += gridDim.x) {
        const int t = tile_of(blockIdx.x, gridDim.x, total - t0);
        if (t < 0) break;        // a last, partial round
        mid_tile<GATED, BM>(a, 0, (t0 + t) % mt * BM, a.rows, (t0 + t) / mt * BO, lds);
    }
}

template <int EB, bool GATED>
__global__ __launch_bounds__(kThreads, 2) void matmul_kernel(const MatmulArgs a, int small_to) {
    __shared__ __align__(1024) uint8_t lds[kLds];
    constexpr int BO = GATED ? kSmall / 2 : kSmall;
    constexpr int BB = GATED ? kBig / 2 : kBig;
    const int nt = (a.N + BO - 1) / BO, ntb = (a.N + BB - 1) / BB;
    const int rows0 = lane_rows(a, 0);
    int n[kKinds], total = 0;
    for (;;) {
        count_runs(a, rows0, small_to, n);
        total = 0;
#pragma unroll
        for (int k = 1; k < kKinds; ++k) {
            n[k] *= ntb;
            total += n[k];
        }
        // small tiles beside so much else cost more than part-filled ones
        if (!small_to || total <= kGrid) break;
        small_to = 0;
    }
    const int nsmall = n[0] * nt;
    if constexpr (EB == 2) {
        // Few enough of them that even cut in parts they would leave CUs idle
        // or share their weights' bytes among them: middle tiles, where one
        // round does (8 experts of 115 rows, 7168 -> 2 x 2048: 101 us with them,
        // 113 without; one of 200: 31 and 73).
        constexpr int G = GATED ? 2 : 1;
        const int nt64 = (a.N * G + 63) / 64, nt128 = (a.N * G + 127) / 128;
        if (total > 0 && total <= kGrid / 2) {
            int runs64 = 0, runs128 = 0;
            for (int g0 = 0; g0 < a.groups; g0 += 64) {
                const int rows = g0 ? lane_rows(a, g0) : rows0;
                runs64 += __builtin_amdgcn_readlane(
                    wave_inclusive_scan(runs_of(rows, small_to, kRuns64)), 63);
                runs128 += __builtin_amdgcn_readlane(
                    wave_inclusive_scan(runs_of(rows, small_to, kRuns128)), 63);
            }
            const int kind = runs64 * nt64 <= kGrid    ? kRuns64
                             : runs128 * nt128 <= kGrid ? kRuns128
                                                        : 0;
            if (kind) {
                const bool wide = kind == kRuns128;
                const int tiles = wide ? runs128 * nt128 : runs64 * nt64;
                const int t = tile_of(blockIdx.x, kGrid, tiles);
                if (t >= 0) {
                    const Place at = find_tile(a, rows0, small_to, kind, wide ? nt128 : nt64, t);
                    const int mt = runs_of(at.rows, small_to, kind);
                    const int m = at.l % mt, c = at.l / mt;
                    if (wide) mid_tile<GATED, 128>(a, at.g, m * 128, at.rows, c * (128 / G), lds);
                    else mid_tile<GATED, 64>(a, at.g, m * 64, at.rows, c * (64 / G), lds);
                }
                total = 0;
            }
        }
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
        const Place at = find_tile(a, rows0, small_to, kind, ntb, t);
        const int runs = cut_rows(at.rows, small_to).runs;
        const Piece p = piece_of(at.l, at.rows, runs, kind, ntb, turn.sub, turn.cut);
        if (p.m0 >= p.end) continue;
        const int n0 = p.col * BB;
        // (a tile of a run-time number of fragments was 18 % slower: its loop
        // is full of branches)
        auto run = [&](auto bm) {
            big_tile<EB, GATED, decltype(bm)::value>(a, at.g, p.m0, p.end, n0, lds);
        };
        const int bm = tile_rows(p.fragments);
        if (bm == 256) run(std::integral_constant<int, 256>{});
        else if (bm == 224) run(std::integral_constant<int, 224>{});
        else if (bm == 192) run(std::integral_constant<int, 192>{});
        else if (bm == 160) run(std::integral_constant<int, 160>{});
        else if (bm == 128) run(std::integral_constant<int, 128>{});
        else narrow_tile<EB, GATED>(a, at.g, p.m0, p.end, n0, lds);
    }
    if (nsmall > 0)
        small_tiles<EB, GATED>(a, lds, nsmall, [&](int t) {
            const Place at = find_tile(a, rows0, small_to, 0, nt, t);
            const int mt = cut_rows(at.rows, small_to).runs;
            return small_setup<EB, GATED>(a, at.g, at.l % mt * kSmall, at.rows, at.l / mt * BO);
        });
}

// Small tiles alone, where the host knows that there are few rows.
template <int EB, bool GATED>
__global__ __launch_bounds__(kThreads, 2) void small_kernel(const MatmulArgs a) {
    __shared__ __align__(1024) uint8_t lds[kSmallLds];
    constexpr int BO = GATED ? kSmall / 2 : kSmall;
    const int nt = (a.N + BO - 1) / BO;
    const int rows0 = lane_rows(a, 0);
    int n[kKinds];
    count_runs(a, rows0, INT32_MAX, n);
    small_tiles<EB, GATED>(a, lds, n[0] * nt, [&](int t) {
        const Place at = find_tile(a, rows0, INT32_MAX, 0, nt, t);
        const int mt = cut_rows(at.rows, INT32_MAX).runs;
        return small_setup<EB, GATED>(a, at.g, at.l % mt * kSmall, at.rows, at.l / mt * BO);
    });
}

// What a product over all tokens takes with each kind of tile, in us, from the
// tiles' measured times: rounds of the grid times a tile's start and its pairs
// of slabs. Both sides measured where the choice turns, in us: 4096 x 7168 by
// 256 rows of w: 64 x 64 tiles 37, big 39, 16 x 16 138; 128 rows of that: 16 x 16
// 8, 64 x 64 26; 2048 x 7168 by 4096 rows: big 99, 128 x 128 127; 576 x 2048 by
// 7168 rows: big 29 to 31 (parts of 96 rows, priced so, in 128-row tiles), 128 x
// 128 37 to 39.
struct Estimate {
    double small, mid64, mid128, big;
};

Estimate estimate(int64_t rows, int64_t nw, int64_t row_bytes) {
    const double pairs = (double)((row_bytes + 2 * kSlab - 1) / (2 * kSlab));
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    Estimate e;
    e.small = (double)up(up(rows, kSmall) * up(nw, kSmall), kGrid) * (2.0 + 0.125 * pairs);
    e.mid64 = (double)up(up(rows, 64) * up(nw, 64), kGrid) * (2.5 + 0.45 * pairs);
    e.mid128 = (double)up(up(rows, 128) * up(nw, 128), kGrid) * (2.5 + 1.0 * pairs);
    // a tile of 32 j rows takes 0.75 + 0.27 j us a pair
    const int64_t runs = up(rows, 256), tiles = runs * up(nw, kBig), rest = tiles % kGrid;
    const int64_t j = up(up(rows, runs), 32);
    const int64_t last = rest * 4 <= kGrid ? up(j, 4) : rest * 2 <= kGrid ? up(j, 2) : j;
    e.big = 3.0 + (double)(tiles / kGrid) * (5.0 + (0.75 + 0.27 * (double)j) * pairs) +
            (rest ? 5.0 + (0.75 + 0.27 * (double)last) * pairs : 0.0);
    return e;
}

template <int EB, bool GATED>
hipError_t launch(const MatmulArgs& a, hipStream_t st) {
    constexpr int BO = GATED ? kSmall / 2 : kSmall;
    const bool e4m3 = a.out_dtype == MOE_EP_E4M3;
    const int64_t small =
        (int64_t)a.groups * ((a.rows + kSmall - 1) / kSmall) * ((a.N + BO - 1) / BO);
    bool few = !e4m3 && a.counts && a.rows <= 2 * kSmall;
    if constexpr (EB == 2) {
        if (!a.counts) {
            const Estimate e = estimate(a.rows, GATED ? 2 * (int64_t)a.N : a.N, a.row_bytes);
            const double mid = e.mid64 < e.mid128 ? e.mid64 : e.mid128;
            few = e.small <= mid && e.small <= e.big;
            if (!few && mid <= e.big) {
                if (e.mid64 <= e.mid128)
                    mid_kernel<GATED, 64><<<kGrid, kThreads, 0, st>>>(a);
                else
                    mid_kernel<GATED, 128><<<kGrid, kThreads, 0, st>>>(a);
                return hipGetLastError();
            }
        }
    }
    if (few) {
        const int64_t grid = small < kGrid ? (small + 7) / 8 * 8 : kGrid;
        small_kernel<EB, GATED><<<(unsigned)grid, kThreads, 0, st>>>(a);
    } else {
        matmul_kernel<EB, GATED>
            <<<kGrid, kThreads, 0, st>>>(a, e4m3 || !a.counts ? 0 : kSmall);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul(const MatmulArgs& a, hipStream_t st) {
    const bool gated = a.act == MOE_EP_ACT_SILU_GATED;
    if (!a.fp8) return gated ? launch<2, true>(a, st) : launch<2, false>(a, st);
    return gated ? launch<1, true>(a, st) : launch<1, false>(a, st);
}

}  // namespace moe_ep
