// A router's training terms: per-expert counts, mean scores and the balance
// loss of sequences of tokens, and the gradient of the logits.
//
//   q[t,e]  softmax(x)[e], or sigmoid(x[e]) / sum_j sigmoid(x[j])
//   c[e]    picks of e, n tokens that have a pick; P[e] = sum_t q[t,e] / n
//   loss    E * sum_e (c[e] / sum c) P[e]; c is a constant to its gradient:
//   dx[t,e] = q[t,e] (a[e] - sum_j q[t,j] a[j]), a[e] = g E c[e] / (sum c * n),
//             for sigmoid scores times 1 - sigmoid(x[e])
//
// Lane l of a wave has a token's experts l, l + 64, ..., of one to four tokens at a
// time. Exponentials and sums over a token's experts are fp32 (a result is used
// once, in fp32: no choice hangs on its last bit); sums over tokens are fp32 within
// a block's tokens, at most 256 to a wave, and fp64 over blocks, always in the same
// order. Counts are integers. Where terms of the gradient cancel they are fp64.
//
// Bound by the logits' bytes only at many tokens (65536 x 256, fp32: the sums 18 us
// at 3.7 TB/s and their join 7, the gradient 38, of 270 vector instructions a token);
// below by chains of loads and of sums over lanes, so a wave has several tokens at
// once (8192 tokens: 15 us the loss, 12 the gradient; 128: 13 and 5.6).
#include <type_traits>

#include "experts.h"

namespace moe_ep {
namespace {

constexpr int kTokenWaves = 16;                  // of a block of the sums
constexpr int kTokenThreads = kTokenWaves * 64;
constexpr int kGradWaves = 4;
constexpr float kLargest = 3.402823466e38f;
const float kNothing = -__builtin_huge_valf();

// Tokens that a wave has at once, so that their loads and their sums over lanes
// (chains of dependent steps) run side by side.
template <int V>
constexpr int kAtOnce = V >= 16 ? 2 : 4;

// Tokens of a wave of the gradient, whose picks lie in KP lanes each.
template <int V, int KP>
constexpr int kGradAtOnce = 64 / KP < kAtOnce<V> ? 64 / KP : kAtOnce<V>;

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

// The sum of fp64 values by lane moves and not through LDS, for each token. (The
// one above, made once a sequence, holds fewer registers: 123, not 129, of the
// gradient of 256 sigmoid scores, where 128 leave room for one wave more.)
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF,
                                                              false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL,
                                                              ROWS, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32);
}

__device__ __forceinline__ double token_sum(double v) {
    v += moved<0x111, 0xF>(v);
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);
    v += moved<0x143, 0xC>(v);
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(
        double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63) |
                    (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63) << 32);
}

__device__ __forceinline__ float token_sum(float v) { return wave_sum(v); }

// A logit as the scores take it: -inf for one that belongs to no expert (-inf
// or NaN), the largest fp32 for +inf.
__device__ __forceinline__ float clean(float x) {
    return x > kNothing ? fminf(x, kLargest) : kNothing;
}

__device__ __forceinline__ float load_logit(const uint8_t* row, bool bf16, int e) {
    return clean(bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << 16)
                      : reinterpret_cast<const float*>(row)[e]);
}

// The logits of B tokens, number b at row(b): one branch for the type, so that
// all loads are on their way together.
template <int B, int V, class Row>
__device__ __forceinline__ void load_tokens(const Row& row, bool bf16, int E, int lane,
                                            float (&x)[B][V]) {
    auto each = [&](auto value) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const uint8_t* p = row(b);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 64 * i;
                x[b][i] = value(p, e < E ? e : 0);
            }
        }
    };
    if (bf16)
        each([](const uint8_t* p, int e) {
            return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << 16);
        });
    else
        each([](const uint8_t* p, int e) { return reinterpret_cast<const float*>(p)[e]; });
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < V; ++i) x[b][i] = lane + 64 * i < E ? clean(x[b][i]) : kNothing;
}

// The hardware's 2^x, within a place. v's rounding times log2 e, half a place
// of a product, is that of the difference in front of it once more.
__device__ __forceinline__ float exp_fast(float v) {
    return __builtin_amdgcn_exp2f(v * 1.44269504f);
}

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

// A token's scores before their sum divides them, and 1 / sum (0 without a
// score). For sigmoid scores also rest = 1 - sigmoid(x), and they are taken
// times e^-m, m = min(0, the largest logit), so that a token of far negative
// logits has scores too. top: the largest logit. all: the sum, and with WIDE one
// of fp64, where the few large scores may be replaced and the others are left.
template <int V, bool SIGMOID, bool WIDE = false>
__device__ __forceinline__ float scores(const float (&x)[V], float (&q)[V], float (&rest)[V],
                                        float& top, double& all) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
    m = fmaxf(wave_max(m), -kLargest);
    top = m;
    if (SIGMOID) m = fminf(m, 0.f);
    const float em = SIGMOID ? exp_fast(m) : 0.f;
    std::conditional_t<WIDE, double, float> sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (SIGMOID) {
            const bool up = x[i] > 0.f;
            const float z = exp_fast(up ? -x[i] : x[i] - m);
            const float d = __builtin_amdgcn_rcpf(1.f + (up ? z : z * em));
            q[i] = (up ? 1.f : z) * d;
            rest[i] = (up ? z : 1.f) * d;
        } else {
            q[i] = exp_fast(x[i] - m);
        }
        sum += q[i];
    }
    sum = token_sum(sum);
    all = sum;
    return sum > 0 ? __builtin_amdgcn_rcpf((float)sum) : 0.f;
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
    if (TILES && blockIdx.x == 0)
        for (int s = threadIdx.x; s < a.S; s += kTokenThreads) a.ticket[s] = 0;
    const int64_t t0 = TILES ? (int64_t)blockIdx.x * a.tile : 0;
    const int64_t t1 = TILES ? (t0 + a.tile < a.T ? t0 + a.tile : a.T) : a.T;
    for (int s = TILES ? first_behind(a.start, a.S, a.T, t0) : (int)blockIdx.x; s < a.S;
         s += TILES ? 1 : (int)gridDim.x) {
        const Span span = span_of(a.start, a.T, s);
        if (TILES && span.lo >= t1) break;
        const int64_t lo = span.lo > t0 ? span.lo : t0, hi = span.hi < t1 ? span.hi : t1;
        if (TILES && hi <= lo) continue;
        for (int e = threadIdx.x; e < a.E; e += kTokenThreads) hist[e] = 0;
        __syncthreads();
        float acc[V] = {};
        int32_t tokens = 0;
        constexpr int B = kAtOnce<V> / 2;
        for (int64_t t = lo + wave; t < hi; t += kTokenWaves * B) {
            float x[B][V];
            int32_t id[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {        // behind the last token: that one again
                const int64_t u = t + b * kTokenWaves < hi ? t + b * kTokenWaves : hi - 1;
                id[b] = a.ids[u * a.K + (lane < a.K ? lane : 0)];
                if (lane >= a.K) id[b] = -1;
            }
            load_tokens<B, V>(
                [&](int b) {
                    const int64_t u = t + b * kTokenWaves < hi ? t + b * kTokenWaves : hi - 1;
                    return a.logits + u * a.logits_stride;
                },
                a.bf16, a.E, lane, x);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const bool pick = id[b] >= 0 && id[b] < a.E && t + b * kTokenWaves < hi;
                const bool count = __ballot(pick) != 0;       // no padding token
                tokens += count;
                if (pick) atomicAdd(&hist[id[b]], 1);
                float q[V], rest[V], top;
                double sum;
                const float inv = scores<V, SIGMOID>(x[b], q, rest, top, sum);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += q[i] * (count ? inv : 0.f);
            }
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
            continue;                            // behind a barrier that all have passed
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

// The sums of a sequence's tiles, a block for 64 experts: its waves share out
// the tiles, each in their order, and are added in theirs. The block that comes
// last adds up the blocks' parts of the loss, in the experts' order. (One block
// for all experts took 40 us for 256 tiles of 256 experts: 512 KB through one
// CU.)
__global__ __launch_bounds__(kTokenThreads) void balance_join_kernel(const BalanceArgs a) {
    __shared__ double scores_of[kTokenWaves][64];
    __shared__ int32_t counts_of[kTokenWaves][64];
    constexpr int U = 16;                        // loads on their way
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int slices = (a.E + 63) / 64;
    for (int64_t u = blockIdx.x; u < (int64_t)a.S * slices; u += gridDim.x) {
        const int s = (int)(u / slices), slice = (int)(u % slices);
        const int e = slice * 64 + lane;
        const int col = e < a.E ? e : a.E - 1;
        const Span span = span_of(a.start, a.T, s);
        const bool any = span.hi > span.lo;
        const int64_t first = span.lo / a.tile + s;      // slots [first, end)
        const int64_t end = any ? (span.hi - 1) / a.tile + 1 + s : first;
        int32_t count = 0;
        double score = 0.0;
        for (int64_t b = first + wave; b < end; b += kTokenWaves * U) {
            int32_t c[U];
            float v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t slot = b + i * kTokenWaves < end ? b + i * kTokenWaves : end - 1;
                c[i] = a.slot_count[slot * a.E + col];
                v[i] = a.slot_score[slot * a.E + col];
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (b + i * kTokenWaves < end) {
                    count += c[i];
                    score += (double)v[i];
                }
        }
        __syncthreads();                         // the sums before are read
        scores_of[wave][lane] = score;
        counts_of[wave][lane] = count;
        __syncthreads();
        if (wave != 0) continue;
        double n = 0.0;
        for (int64_t b = first + lane; b < end; b += 64) n += (double)a.slot_tokens[b];
        n = wave_sum(n);
        for (int w = 1; w < kTokenWaves; ++w) {
            score += scores_of[w][lane];
            count += counts_of[w][lane];
        }
        const double mean = n > 0.0 ? score / n : 0.0;
        if (e < a.E) {
            a.counts[(int64_t)s * a.E + e] = count;
            a.mean[(int64_t)s * a.E + e] = (float)mean;
        }
        double picks = wave_sum(e < a.E ? (double)count : 0.0);
        double both = wave_sum(e < a.E ? (double)count * mean : 0.0);
        if (slices > 1) {
            double* const parts = a.part + (int64_t)s * slices * 2;
            int before = 0;
            if (lane == 0) {
                __hip_atomic_store(parts + 2 * slice, picks, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
                __hip_atomic_store(parts + 2 * slice + 1, both, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
                before = __hip_atomic_fetch_add(a.ticket + s, 1, __ATOMIC_ACQ_REL,
                                                __HIP_MEMORY_SCOPE_AGENT);
            }
            if (__builtin_amdgcn_readfirstlane(before) != slices - 1) continue;
            picks = both = 0.0;
            if (lane == 0)
                for (int i = 0; i < slices; ++i) {
                    picks += __hip_atomic_load(parts + 2 * i, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT);
                    both += __hip_atomic_load(parts + 2 * i + 1, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT);
                }
        }
        if (lane == 0) {
            a.tokens[s] = (int32_t)n;
            a.loss[s] = (float)(picks > 0.0 ? (double)a.E * both / picks : 0.0);
        }
    }
}

// v of the lane whose number differs in the bits of MASK: 1 to 3 within quads, 7
// (half rows mirrored) and 15 (rows mirrored).
template <int MASK>
__device__ __forceinline__ int other(int v) {
    constexpr int ctrl = MASK == 1   ? 0xB1
                         : MASK == 2 ? 0x4E
                         : MASK == 3 ? 0x1B
                         : MASK == 7 ? 0x141
                                     : 0x140;
    return __builtin_amdgcn_update_dpp(0, v, ctrl, 0xF, 0xF, true);
}

template <int MASK>
__device__ __forceinline__ double other(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)other<MASK>((int)(uint32_t)u) |
                                          (uint64_t)(uint32_t)other<MASK>((int)(u >> 32)) << 32);
}

// The sum over a token's picks in the first K of KP neighbouring lanes (the others
// have zeros), in those lanes.
template <int KP>
__device__ __forceinline__ double picks_sum(double v, int K) {
    if (K == 1) return v;
    if (K > 16) return token_sum(v);
    v += other<1>(v);
    v += other<2>(v);
    v += other<7>(v);                            // a quad's lanes have the same by now
    if (KP > 8 && K > 8) v += other<15>(v);
    return v;
}

// Whether one of the wave's tokens, whose picks are in groups of N neighbouring
// lanes, has an expert twice.
template <int N>
__device__ __forceinline__ bool repeats(int id, bool pick) {
    bool same = false;
    if constexpr (N == 64) {
        for (uint64_t m = __ballot(pick); m; m &= m - 1) {
            const int at = __builtin_amdgcn_readlane(id, __builtin_ctzll(m));
            const uint64_t equal = __ballot(pick && id == at);
            same |= (equal & (equal - 1)) != 0;
        }
        return same;
    }
    // each lane against those that differ in the bits of 1 to N - 1
    auto quads = [&](int v) {
        same |= other<1>(v) == id || other<2>(v) == id || other<3>(v) == id;
    };
    auto halves = [&](int v) {
        quads(v);
        const int m = other<7>(v);
        same |= m == id;
        quads(m);
    };
    halves(id);
    if constexpr (N == 16) {
        const int m = other<15>(id);
        same |= m == id;
        halves(m);
    }
    return __ballot(pick && same) != 0;
}

// The gradient of the logits. Through the picks' weights w = scale * p[pick]
// (renormalize: / the picks' sum) with g their gradient:
//   softmax, renormalised    dx[pick] += w (g - sum g w / scale)
//   softmax                  dx[e]    += scale p[e] (G[e] - sum over picks of p g),
//                            G[e] the sum of g over the picks of e
//   sigmoid                  the first form (plain: w g) times 1 - sigmoid(x[pick])
// The picks' part, one exponential a token, is fp64: g - sum g w and G - sum p g
// cancel where the picks have almost all of the scores (of one pick with p =
// 1 - 4e-8, fp32 left a gradient 18 % off). A plain softmax's sum is fp64 for that
// too, its picks' scores replaced by their fp64 ones, and picks get their
// experts' gradient whole instead of a correction to an fp32 one.
//
// A wave has B tokens at once, and 64 / B lanes have the picks of each (KP), so
// that the fp64 part is done for all of them in one go.
//
// PLAIN: a softmax's weights that are not renormalised have a gradient. (Up to 256
// experts at many tokens it is held to the registers of five waves a SIMD: 65536
// tokens 37.5 us, with five registers more and four waves 39.9.)
template <int V, bool SIGMOID, bool PLAIN, int KP>
__global__ __launch_bounds__(kGradWaves * 64, PLAIN && V == 4 && KP == 8 ? 5 : 1) void
route_backward_kernel(const RouteGradArgs a) {
    constexpr int B = kGradAtOnce<V, KP>;
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int of = lane / KP, pk = lane % KP;    // the lane's token and pick
    extern __shared__ __align__(16) float grad_lds[];    // PLAIN: [waves][B][E]
    float each[V] = {};                          // a[e] of the sequence at hand
    int s = -1, at_s = -1;
    Span span = {0, 0};                          // of sequence s
    const int64_t t0 = (int64_t)blockIdx.x * a.tile;
    const int64_t t1 = t0 + a.tile < a.T ? t0 + a.tile : a.T;
    for (int64_t t = t0 + wave * B; t < t1; t += kGradWaves * B) {
        // all loads first; behind the last token that one again
        const bool mine = of < B && pk < a.K && t + of < t1;
        const int64_t tp = mine ? t + of : t;
        const int32_t id = mine ? a.ids[tp * a.K + pk] : -1;
        const bool pick = id >= 0 && id < a.E;
        float g = 0.f;
        if (pick && a.grad_weights) g = a.grad_weights[tp * a.K + pk];
        float q[B][V], rest[B][SIGMOID ? V : 1], xs[B][V];
        load_tokens<B, V>(
            [&](int b) {
                return a.logits + (t + b < t1 ? t + b : t1 - 1) * a.logits_stride;
            },
            a.bf16, a.E, lane, xs);
        float xp = kNothing;
        if (pick) xp = load_logit(a.logits + tp * a.logits_stride, a.bf16, id);
        const uint64_t picks = __ballot(pick);
        uint64_t given = picks;                  // those that have their expert's gradient

        float my_top = 0.f;                      // of the lane's token
        double my_all = 0.0;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            float top, left[V];
            double all;
            const float inv = scores<V, SIGMOID, PLAIN>(xs[b], q[b], left, top, all);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                q[b][i] *= inv;
                if (SIGMOID) rest[b][i] = left[i];
            }
            if (of == b) {
                my_top = top;
                my_all = all;
            }
        }

        float back = 0.f, backs = 0.f;           // what reaches the logit of the lane's pick
        if (PLAIN || a.grad_weights) {
            bool live = pick && xp > kNothing;
            double gw = live ? (double)g : 0.0;
            if (PLAIN && a.K > 1 &&
                (a.K <= 8    ? repeats<8>(id, pick)
                 : a.K <= 16 ? repeats<16>(id, pick)
                             : repeats<64>(id, pick))) {
                // the first of an expert's picks has the gradients of all
                const double mine = gw;
                bool first = true;
                gw = 0.0;
                for (int j = 0; j < a.K; ++j) {
                    const int from = of * KP + j;
                    const bool same = __shfl(id, from, 64) == id;
                    const double v = __shfl(mine, from, 64);
                    if (same) gw += v;
                    if (same && j < pk) first = false;
                }
                live = live && first;
                given = __ballot(pick && first);
            }
            const double v = live ? (double)xp : 0.0;
            double w, left = 1.0;
            if (SIGMOID) {
                const double z = exp(-fabs(v));
                w = (v >= 0.0 ? 1.0 : z) / (1.0 + z);
                left = (v >= 0.0 ? z : 1.0) / (1.0 + z);
            } else {
                w = exp(v - (double)my_top);     // times 1 / sum, left out of a ratio
            }
            if (!live) w = 0.0;
            if (!PLAIN && a.renormalize) {
                const double all = picks_sum<KP>(w, a.K);
                w = all > 0.0 ? w / all : 0.0;
                gw -= picks_sum<KP>(gw * w, a.K);
            }
            if constexpr (PLAIN) {
                // the pick's score as the sum has it, from the same fp32 steps
                const double had = live ? (double)exp_fast(xp - my_top) : 0.0;
                const double all = my_all + picks_sum<KP>(w - had, a.K);
                w = live ? w / all : 0.0;
                const double through = picks_sum<KP>(gw * w, a.K);
                backs = (float)((double)a.scale * through);
                gw -= through;
            }
            back = live ? (float)((double)a.scale * w * gw * left) : 0.f;
        }

        // a plain softmax's part of all experts, the picks' put in their places,
        // in LDS of the wave's own (which serves a wave in order)
        float* const part = grad_lds + (PLAIN ? wave * B * a.E : 0);
        if constexpr (PLAIN) {
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const float all = lane_value(backs, b * KP & 63);
#pragma unroll
                for (int i = 0; i < V; ++i)      // (where q = 0, `all` may be no number)
                    if (lane + 64 * i < a.E)
                        part[b * a.E + lane + 64 * i] = q[b][i] == 0.f ? 0.f : -(q[b][i] * all);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (given >> lane & 1) part[of * a.E + id] = back;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }

#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (t + b >= t1) break;
            constexpr uint64_t kGroup = KP == 64 ? ~0ull : (1ull << (KP & 63)) - 1;
            uint64_t mask = picks >> (b * KP & 63) & kGroup;     // of a padding token 0
            bool aux = false;
            if (a.grad_loss && mask) {
                if (s < 0 || span.hi <= t + b) {
                    if (s < a.S) s = s < 0 ? first_behind(a.start, a.S, a.T, t + b) : s + 1;
                    for (; s < a.S && (span = span_of(a.start, a.T, s)).hi <= t + b; ++s) {}
                }
                aux = s < a.S && span.lo <= t + b;
            }
            if (aux && at_s != s) {
                const int32_t* c = a.counts + (int64_t)s * a.E;
                float n[V];
                double all = 0.0;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = lane + 64 * i;
                    const int32_t v = e < a.E ? c[e] : 0;
                    n[i] = (float)v;
                    all += (double)v;
                }
                all = wave_sum(all);
                const int32_t tokens = a.tokens[s];
                const float f = all > 0.0 && tokens > 0
                                    ? a.grad_loss[s] * (float)a.E / (float)all / (float)tokens
                                    : 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) each[i] = f * n[i];
                at_s = s;
            }
            float through = 0.f;                 // sum_j q[j] (what reaches q[j])
            if (aux) {
#pragma unroll
                for (int i = 0; i < V; ++i) through += q[b][i] * each[i];
                through = wave_sum(through);
            }
            float dx[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dx[i] = q[b][i] * ((aux ? each[i] : 0.f) - through);
                if (SIGMOID) dx[i] *= rest[b][i];
                if (q[b][i] == 0.f) dx[i] = 0.f; // also where `through` is no number
            }
            if constexpr (PLAIN) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (lane + 64 * i < a.E) dx[i] += part[b * a.E + lane + 64 * i];
            } else if (a.grad_weights) {
                for (; mask; mask &= mask - 1) {
                    const int from = b * KP + __builtin_ctzll(mask);
                    const int e = __builtin_amdgcn_readlane(id, from);
                    const float v = (e & 63) == lane ? lane_value(back, from) : 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (e >> 6 == i) dx[i] += v;
                }
            }
            uint8_t* out = a.grad + (t + b) * a.grad_stride;
            if (a.grad_bf16) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (lane + 64 * i < a.E)
                        reinterpret_cast<uint16_t*>(out)[lane + 64 * i] =
                            (uint16_t)to_bf16_rne(dx[i]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (lane + 64 * i < a.E)
                        reinterpret_cast<float*>(out)[lane + 64 * i] = dx[i];
            }
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
    // a grid has fewer than 2^32 threads: blocks stride over many sequences
    auto at_most = [](int64_t n) { return (unsigned)(n < 1 << 20 ? n : 1 << 20); };
    const unsigned grid = tiles ? (unsigned)((a.T + a.tile - 1) / a.tile) : at_most(a.S);
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
    balance_join_kernel<<<at_most((int64_t)a.S * ((a.E + 63) / 64)), kTokenThreads, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteGradArgs& a, hipStream_t st) {
    const unsigned grid = (unsigned)((a.T + a.tile - 1) / a.tile);
    return by_width(a.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        auto run = [&](auto sigmoid, auto plain, auto kp) {
            constexpr int KP = decltype(kp)::value;
            constexpr bool P = decltype(plain)::value;
            const size_t lds = P ? (size_t)kGradWaves * kGradAtOnce<V, KP> * a.E * 4 : 0;
            route_backward_kernel<V, decltype(sigmoid)::value, P, KP>
                <<<grid, kGradWaves * 64, lds, st>>>(a);
        };
        // One token a wave, over more of the CUs and with fewer registers, or (of up to
        // 16 picks) several, which share the fp64 part. Both in us, one and several:
        // 64 experts, 4096 tokens 6.1 and 6.5, 8192 8.9 and 7.6; 256, softmax, 16384
        // tokens 17.8 and 19.3, 32768 30 and 27; 512, 32768 tokens renormalised 41 and
        // 45, plain 37 and 34; 1024, 65536 tokens 126 and 132.
        auto by_picks = [&](auto sigmoid, auto plain) {
            if constexpr (V <= 4 || (V == 8 && decltype(plain)::value))
                if (a.T > (V <= 2 ? 8191 : 16384) && a.K <= 16) {
                    if (a.K <= 8) run(sigmoid, plain, std::integral_constant<int, 8>{});
                    else run(sigmoid, plain, std::integral_constant<int, 16>{});
                    return;
                }
            run(sigmoid, plain, std::integral_constant<int, 64>{});
        };
        if (a.score == MOE_EP_SIGMOID) by_picks(std::true_type{}, std::false_type{});
        else if (a.grad_weights && !a.renormalize) by_picks(std::false_type{}, std::true_type{});
        else by_picks(std::false_type{}, std::false_type{});
    });
}

}  // namespace moe_ep
