// Balance loss of the router and its gradient.  With c the routed slots of
// sequence s with expert e, L its tokens that are no padding, S' the sequences
// that have any, p the scores:
//     loss = coef/S' * sum_s sum_e  E c / (k L) * (1/L) sum_t p[t][e]
//     dloss/dp[t][e] = w[s][e] = coef E c / (S' k L^2)
//     softmax: dz[e] = p[e] (w[e] - sum_j p[j] w[j]);  sigmoid: the same times 1 - s(z[e])
//
// Forward: workgroups sum p and count slots over tiles of tokens, then the
// tiles are summed in their order.  Backward: one pass, the scores computed
// again from the logits (writing them in the forward pass would cost more than
// reading the logits twice).  No sum depends on the order of atomics: those
// count slots.  131072 rows of 256 bf16 logits: 17 us for the tiles (67 MB, 4.3
// TB/s), 9 us for their sums, 35 us backward (134 MB, 3.9 TB/s), each group of
// lanes working on one row at a time, with the dependent lane exchanges of
// its sums.  4096 rows of 256 fp32 logits: 4, 7 and 7 us, latency.
#include "experts_common.h"

namespace moedisp {
namespace {

constexpr int kBalThreads = 256;
constexpr int kSeqThreads = 1024;
constexpr int kSeqCols = 64;  // experts of a workgroup that sums tiles

template <int LPR>
__device__ inline int lanes_count(int v) {
    return __float_as_int(row_reduce<LPR>(__int_as_float(v), [](float x, float y) {
        return __int_as_float(__float_as_int(x) + __float_as_int(y));
    }));
}

// Whether any of the row's LPR lanes has it.
template <int LPR>
__device__ inline bool lanes_any(bool v) {
    const uint64_t b = __ballot(v);
    if (LPR == 64) return b != 0;
    const int at = (threadIdx.x & 63) / LPR * LPR;
    return ((b >> at) & ((1ull << (LPR & 63)) - 1ull)) != 0;
}

// The row's logits as they are stored: lane l of its LPR lanes holds experts
// (c * LPR + l) * 8 .. + 7 of chunk c; one or two 16-byte loads a chunk where
// rows are whole multiples of 8 experts (VEC).
template <int LPR, int CH, bool BF16, bool VEC>
struct Row {
    v4u raw[VEC ? CH * (BF16 ? 1 : 2) : 1];
    float one[VEC ? 1 : CH * 8];

    // -inf everywhere: lanes past the last expert keep it (VEC)
    __device__ inline void clear() {
        const uint32_t v = BF16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
        for (int i = 0; i < (VEC ? CH * (BF16 ? 1 : 2) : 1); ++i) raw[i] = v4u{v, v, v, v};
    }

    __device__ inline void load(const BalanceArgs& a, size_t row, int l) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int e0 = (c * LPR + l) * 8;
            if (VEC) {
                const size_t at = row * a.E + e0;
                if (e0 >= a.E) continue;
                if (BF16) {
                    raw[c] = *reinterpret_cast<const v4u*>(reinterpret_cast<const uint16_t*>(a.logits) + at);
                } else {
                    const v4u* p = reinterpret_cast<const v4u*>(reinterpret_cast<const float*>(a.logits) + at);
                    raw[2 * c] = p[0];
                    raw[2 * c + 1] = p[1];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const size_t at = row * a.E + (e0 + i < a.E ? e0 + i : 0);
                    one[c * 8 + i] =
                        BF16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(a.logits)[at] << 16)
                             : reinterpret_cast<const float*>(a.logits)[at];
                }
            }
        }
    }
    __device__ inline void values(const BalanceArgs& a, int l, float z[CH * 8]) const {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float& v = z[c * 8 + i];
                if (!VEC)
                    v = (c * LPR + l) * 8 + i < a.E ? one[c * 8 + i] : -INFINITY;
                else if (BF16)
                    v = (i & 1) ? bf16_high(raw[c][i >> 1]) : bf16_low(raw[c][i >> 1]);
                else
                    v = __uint_as_float(raw[2 * c + (i >> 2)][i & 3]);
            }
    }
};

__device__ inline float exp_of(float v) { return __builtin_amdgcn_exp2f(v * 0x1.715476p+0f); }

// Scores of one row times a common factor, and the factor's inverse: score v
// is p[v] * the result.  For the sigmoid also the slopes 1 - s(z) if wanted.
template <int LPR, int N, bool SLOPE>
__device__ inline float row_scores(bool sigmoid, const float z[N], float p[N], float slope[N]) {
    float sum = 0.0f;
    if (sigmoid) {
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const float x = exp_of(-z[v]);
            p[v] = __builtin_amdgcn_rcpf(1.0f + x);
            if (SLOPE) slope[v] = z[v] >= 0.0f ? x * p[v] : 1.0f - p[v];
            sum += p[v];
        }
        sum = lanes_sum<LPR>(sum);
        // Where every logit is so far below zero that the scores vanish
        // together, s(z) is exp(z): the factor exp(-m) keeps their ratios.
        if (__any(sum < 0x1p-100f)) {
            float m = -INFINITY, low = 0.0f;
#pragma unroll
            for (int v = 0; v < N; ++v) m = fmaxf(m, z[v]);
            m = lanes_max<LPR>(m);
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const float x = z[v] == -INFINITY ? 0.0f : exp_of(z[v] - m);
                if (sum < 0x1p-100f) p[v] = x;
                low += x;
            }
            low = lanes_sum<LPR>(low);
            if (sum < 0x1p-100f) sum = low;
        }
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int v = 0; v < N; ++v) m = fmaxf(m, z[v]);
        m = lanes_max<LPR>(m);
        m = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            p[v] = exp_of(z[v] - m);
            sum += p[v];
        }
        sum = lanes_sum<LPR>(sum);
    }
    return sum == 0.0f ? 0.0f : 1.0f / sum;  // no score at all: 0
}

// Slot l of the row (loaded with the row's logits, a row ahead), masked where
// there is none.
__device__ inline int first_slot(const BalanceArgs& a, size_t row, int l) {
    return l < a.k ? a.topk_idx[row * a.k + l] : -1;
}

// Whether the row has a routed slot, counted per expert if `count` is given.
// `id` is the lane's first_slot.
template <int LPR>
__device__ inline bool row_routed(const BalanceArgs& a, size_t row, int l, bool valid, int id, int* count, bool* bad) {
    bool routed = false;
    if (valid)
        for (int j = l; j < a.k; j += LPR) {
            if (j != l) id = a.topk_idx[row * a.k + j];
            if (id >= 0 && id < a.E) {
                if (count) atomicAdd(&count[id], 1);
                routed = true;
            } else if (id != -1) {
                *bad = true;
            }
        }
    return lanes_any<LPR>(routed);
}

// Forward, first launch: the score sums [E], slot counts [E] and token count
// of one tile.  A row's lanes keep the sums of their experts over the tile's
// rows; the next row is loaded before the present one is worked on.
template <int LPR, int CH, bool BF16, bool VEC>
__global__ __launch_bounds__(kBalThreads) void moedisp_balance_tile(BalanceArgs a) {
    constexpr int kRows = kBalThreads / LPR;  // rows at a time
    constexpr int N = CH * 8;
    extern __shared__ float s_p[];            // [kRows][E], then int [E], int
    int* s_c = reinterpret_cast<int*>(s_p + kRows * a.E);
    int* s_n = s_c + a.E;
    const int tid = threadIdx.x;
    const int seq = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int t0 = tile * a.tile_tokens, t1 = min(a.L, t0 + a.tile_tokens);
    const int l = tid % LPR, r = tid / LPR;
    const size_t row0 = (size_t)seq * a.L;
    Row<LPR, CH, BF16, VEC> cur;
    cur.clear();
    cur.load(a, row0 + min(t0 + r, t1 - 1), l);
    int id = first_slot(a, row0 + min(t0 + r, t1 - 1), l);
    for (int e = tid; e < a.E + 1; e += kBalThreads) s_c[e] = 0;
    __syncthreads();
    float acc[N];
#pragma unroll
    for (int v = 0; v < N; ++v) acc[v] = 0.0f;
    bool bad = false;
    int n = 0;
    for (int base = t0; base < t1; base += kRows) {
        const int t = base + r;
        const bool valid = t < t1;
        Row<LPR, CH, BF16, VEC> next = cur;
        if (CH == 1 && base + kRows < t1) next.load(a, row0 + min(t + kRows, t1 - 1), l);
        const int next_id = base + kRows < t1 ? first_slot(a, row0 + min(t + kRows, t1 - 1), l) : -1;
        const bool routed = row_routed<LPR>(a, row0 + t, l, valid, id, s_c, &bad);
        float z[N], p[N], slope[N];
        cur.values(a, l, z);
        const float inv = row_scores<LPR, N, false>(a.sigmoid, z, p, slope);
        if (routed) {
            ++n;
#pragma unroll
            for (int v = 0; v < N; ++v) acc[v] = __builtin_fmaf(p[v], inv, acc[v]);
        }
        id = next_id;
        if (CH == 1)
            cur = next;
        else if (base + kRows < t1)
            cur.load(a, row0 + min(t + kRows, t1 - 1), l);
    }
    if (l == 0 && n) atomicAdd(s_n, n);
#pragma unroll
    for (int v = 0; v < N; ++v) {
        const int e = ((v >> 3) * LPR + l) * 8 + (v & 7);
        if (e < a.E) s_p[r * a.E + e] = acc[v];
    }
    if (bad) atomicOr(&a.hdr->status, (uint32_t)MOEDISP_DEV_BAD_EXPERT_ID);
    __syncthreads();
    // the rows' sums: first every parts-th row (parts * E lanes, each into the
    // row that only it reads), then those
    const int parts = min(kRows, max(1, kBalThreads / a.E));
    if (parts > 1) {
        if (tid < parts * a.E) {
            float sum = 0.0f;
            for (int i = tid / a.E; i < kRows; i += parts) sum += s_p[i * a.E + tid % a.E];
            s_p[tid] = sum;
        }
        __syncthreads();
    }
    for (int e = tid; e < a.E; e += kBalThreads) {
        float sum = 0.0f;
        for (int i = 0; i < (parts > 1 ? parts : kRows); ++i) sum += s_p[i * a.E + e];
        a.psum[(size_t)blockIdx.x * a.E + e] = sum;
        a.count[(size_t)blockIdx.x * a.E + e] = s_c[e];
    }
    if (tid == 0) a.tokens[blockIdx.x] = *s_n;
}

// Sum over the workgroup in a fixed order, for every lane.
__device__ inline double block_sum(double v, double* s) {
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < (int)blockDim.x / 64; ++w) t += s[w];
    return t;
}

// Forward, second launch: a workgroup sums the tiles of 64 experts of one
// sequence (its 16 waves every 16th tile, joined in order) and their part of
// the loss; the last workgroup to finish adds the parts up in order.
__global__ __launch_bounds__(kSeqThreads) void moedisp_balance_seq(BalanceArgs a) {
    constexpr int kW = kSeqThreads / 64;
    __shared__ double s_sum[kW];
    __shared__ float s_p[kW][kSeqCols];
    __shared__ int s_c[kW][kSeqCols];
    __shared__ int s_n[kW];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cols = (a.E + kSeqCols - 1) / kSeqCols;
    if (a.S > 0) {
        const int seq = blockIdx.x / cols, e = blockIdx.x % cols * kSeqCols + lane;
        float p = 0.0f;
        int c = 0;
        if (e < a.E) {
            const size_t at = (size_t)seq * a.tiles * a.E + e;
#pragma unroll 4
            for (int t = wave; t < a.tiles; t += kW) {
                p += a.psum[at + (size_t)t * a.E];
                c += a.count[at + (size_t)t * a.E];
            }
        }
        s_p[wave][lane] = p;
        s_c[wave][lane] = c;
        int tok = 0;
        for (int t = tid; t < a.tiles; t += kSeqThreads) tok += a.tokens[(size_t)seq * a.tiles + t];
        tok = wave_sum_dpp(tok);
        if (lane == 0) s_n[wave] = tok;
        __syncthreads();
        double n = 0.0;
        for (int w = 0; w < kW; ++w) n += s_n[w];
        if (wave == 0) {
            double pt = 0.0;
            int ct = 0;
            for (int w = 0; w < kW; ++w) {
                pt += s_p[w][lane];
                ct += s_c[w][lane];
            }
            if (e < a.E) a.tokens_per_expert[(size_t)seq * a.E + e] = ct;
            double part = pt * ct;
            for (int m = 1; m < 64; m <<= 1) part += __shfl_xor(part, m);
            if (lane == 0) {
                if (blockIdx.x % cols == 0) a.tokens_per_seq[seq] = (int)n;
                part = n > 0.0 ? part * a.E / ((double)a.k * n * n) : 0.0;
                __hip_atomic_store(a.part + blockIdx.x, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                if (blockIdx.x % cols == 0)
                    __hip_atomic_store(a.some + seq, n > 0.0 ? 1 : 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
    }
    if (tid == 0) {
        // The parts above are stored past the caches of the XCD and read past
        // them below; they have arrived before the counter goes up.  (Release
        // and acquire order would write back and drop a whole L2: 4 us.)
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const uint32_t before =
            __hip_atomic_fetch_add(&a.hdr->finished, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = before == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    double sum = 0.0, some = 0.0;
    for (int i = tid; i < a.S * cols; i += kSeqThreads)
        sum += __hip_atomic_load(a.part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int i = tid; i < a.S; i += kSeqThreads)
        some += __hip_atomic_load(a.some + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum = block_sum(sum, s_sum);
    some = block_sum(some, s_sum);
    if (tid == 0) {
        if (a.S > 0) a.hdr->tables_lost = 1;  // the sums above lie where a split dispatch keeps its tables
        *a.loss = some > 0.0 ? (float)(a.coef * sum / some) : 0.0f;
        __hip_atomic_store(&a.hdr->finished, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
    }
}

// Backward: one pass over the rows as in the forward's first launch.  Every
// workgroup counts the sequences that have tokens: with one workgroup to a tile
// that would be S reads for each of at least S workgroups, so beyond 4096 tiles
// (more than 2048 sequences) 2048 workgroups take tile after tile (65536
// sequences of 16 tokens and 64 experts: 330 us against 1442).
template <int LPR, int CH, bool BF16, bool VEC>
__global__ __launch_bounds__(kBalThreads) void moedisp_balance_backward(BalanceArgs args) {
    BalanceArgs a = args;
    constexpr int kRows = kBalThreads / LPR;
    constexpr int N = CH * 8;
    const int tid = threadIdx.x;
    const int l = tid % LPR, r = tid / LPR;
    const int items = a.S * a.tiles;
    int seq, t0, t1, id;
    size_t row0;
    Row<LPR, CH, BF16, VEC> cur;
    auto begin = [&](int item) {
        seq = item / a.tiles;
        t0 = item % a.tiles * a.tile_tokens;
        t1 = min(a.L, t0 + a.tile_tokens);
        row0 = (size_t)seq * a.L;
        cur.clear();
        cur.load(a, row0 + min(t0 + r, t1 - 1), l);
        id = first_slot(a, row0 + min(t0 + r, t1 - 1), l);
    };
    int item = blockIdx.x;
    begin(item);
    int some = 0;
#pragma unroll 8
    for (int s = tid; s < a.S; s += kBalThreads) some += a.tokens_per_seq[s] > 0 ? 1 : 0;
    for (int m = 1; m < 64; m <<= 1) some += __shfl_xor(some, m);
    __shared__ int s_some[kBalThreads / 64];
    if ((tid & 63) == 0) s_some[tid >> 6] = some;
    __syncthreads();
    some = s_some[0] + s_some[1] + s_some[2] + s_some[3];
    // Beyond 1024 experts a lane's 64 conditions e < E, kept over the loops, would
    // drive others out of the registers (16 x 1024 rows of 1030 experts: forward and
    // backward 330 us in bf16 and 378 in fp32, against 280 and 303).
    auto make_anew = [&] {
        if constexpr (CH > 2) asm volatile("" : "+s"(a.E));
    };
    for (;;) {
        make_anew();
        const double n = a.tokens_per_seq[seq];
        const float scale = n > 0.0 ? (float)((double)a.coef * a.E * *a.d_loss / ((double)some * a.k * n * n)) : 0.0f;
        // As the scores of a row add up to 1, the same may be taken from all counts:
        // with their mean taken away what differs between them is not lost in
        // w - dot where they are nearly equal.  (Their own mean: masked slots are
        // not counted.)
        int c[N], slots = 0;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int e = ((v >> 3) * LPR + l) * 8 + (v & 7);
            c[v] = e < a.E ? a.tokens_per_expert[(size_t)seq * a.E + e] : 0;
            slots += c[v];
        }
        const int mean = lanes_count<LPR>(slots) / a.E;
        float w[N];
#pragma unroll
        for (int v = 0; v < N; ++v)
            w[v] = ((v >> 3) * LPR + l) * 8 + (v & 7) < a.E ? scale * (float)(c[v] - mean) : 0.0f;
        bool bad = false;
        for (int base = t0; base < t1; base += kRows) {
            make_anew();
            const int t = base + r;
            const bool valid = t < t1;
            Row<LPR, CH, BF16, VEC> next = cur;
            if (CH == 1 && base + kRows < t1) next.load(a, row0 + min(t + kRows, t1 - 1), l);
            const int next_id = base + kRows < t1 ? first_slot(a, row0 + min(t + kRows, t1 - 1), l) : -1;
            const bool routed = row_routed<LPR>(a, row0 + t, l, valid, id, nullptr, &bad);
            float z[N], p[N], slope[N];
            cur.values(a, l, z);
            const float inv = row_scores<LPR, N, true>(a.sigmoid, z, p, slope);
            float dot = 0.0f;
#pragma unroll
            for (int v = 0; v < N; ++v) {
                p[v] *= inv;
                dot = __builtin_fmaf(p[v], w[v], dot);
            }
            dot = lanes_sum<LPR>(dot);
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const float dz = p[v] * (w[v] - dot);
                z[v] = a.sigmoid ? dz * slope[v] : dz;
            }
            if (!routed) {
#pragma unroll
                for (int v = 0; v < N; ++v) z[v] = 0.0f;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e0 = (c * LPR + l) * 8;
                const size_t at = (row0 + t) * a.E + e0;
                const float* d = z + c * 8;
                if (VEC) {
                    if (valid && e0 < a.E) {
                        if (BF16) {
                            const v4u o = {pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]), pack_bf16x2(d[4], d[5]),
                                           pack_bf16x2(d[6], d[7])};
                            *reinterpret_cast<v4u*>(reinterpret_cast<uint16_t*>(a.d_logits) + at) = o;
                        } else {
                            v4f* o = reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.d_logits) + at);
                            o[0] = v4f{d[0], d[1], d[2], d[3]};
                            o[1] = v4f{d[4], d[5], d[6], d[7]};
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (valid && e0 + i < a.E) {
                            if (BF16)
                                reinterpret_cast<uint16_t*>(a.d_logits)[at + i] = (uint16_t)pack_bf16x2(d[i], 0.0f);
                            else
                                reinterpret_cast<float*>(a.d_logits)[at + i] = d[i];
                        }
                }
            }
            id = next_id;
            if (CH == 1)
                cur = next;
            else if (base + kRows < t1)
                cur.load(a, row0 + min(t + kRows, t1 - 1), l);
        }
        item += gridDim.x;
        if (item >= items) return;
        begin(item);
    }
}

template <int LPR, int CH, bool BF16, bool VEC>
hipError_t launch_pass(const BalanceArgs& a, bool backward, hipStream_t stream) {
    const long long blocks = (long long)a.S * a.tiles;
    if (!grid_fits(blocks, kBalThreads)) return hipErrorInvalidConfiguration;
    if (backward) {
        hipLaunchKernelGGL((moedisp_balance_backward<LPR, CH, BF16, VEC>),
                           dim3((unsigned)balance_backward_blocks(blocks)), dim3(kBalThreads), 0, stream, a);
    } else {
        const size_t lds = ((size_t)(kBalThreads / LPR) * a.E + a.E + 1) * 4;
        hipLaunchKernelGGL((moedisp_balance_tile<LPR, CH, BF16, VEC>), dim3((unsigned)blocks), dim3(kBalThreads), lds,
                           stream, a);
    }
    return hipGetLastError();
}

template <bool BF16, bool VEC>
hipError_t launch_rows(const BalanceArgs& a, bool backward, hipStream_t stream) {
    switch (balance_lanes(a.E)) {
        case 1: return launch_pass<1, 1, BF16, VEC>(a, backward, stream);
        case 2: return launch_pass<2, 1, BF16, VEC>(a, backward, stream);
        case 4: return launch_pass<4, 1, BF16, VEC>(a, backward, stream);
        case 8: return launch_pass<8, 1, BF16, VEC>(a, backward, stream);
        case 16: return launch_pass<16, 1, BF16, VEC>(a, backward, stream);
        case 32: return launch_pass<32, 1, BF16, VEC>(a, backward, stream);
        default: break;
    }
    if (a.E <= 512) return launch_pass<64, 1, BF16, VEC>(a, backward, stream);
    if (a.E <= 1024) return launch_pass<64, 2, BF16, VEC>(a, backward, stream);
    return launch_pass<64, 8, BF16, VEC>(a, backward, stream);
}

hipError_t launch_type(const BalanceArgs& a, bool bf16, bool backward, hipStream_t stream) {
    const bool vec = a.E % 8 == 0;
    if (bf16) return vec ? launch_rows<true, true>(a, backward, stream) : launch_rows<true, false>(a, backward, stream);
    return vec ? launch_rows<false, true>(a, backward, stream) : launch_rows<false, false>(a, backward, stream);
}

}  // namespace

hipError_t launch_balance(const BalanceArgs& a, bool bf16, hipStream_t stream) {
    const long long blocks = a.S > 0 ? (long long)a.S * ((a.E + kSeqCols - 1) / kSeqCols) : 1;
    if (!grid_fits(blocks, kSeqThreads)) return hipErrorInvalidConfiguration;  // before anything is enqueued
    if (a.S > 0 && a.tiles > 0) {
        const hipError_t e = launch_type(a, bf16, false, stream);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(moedisp_balance_seq, dim3((unsigned)blocks), dim3(kSeqThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, bool bf16, hipStream_t stream) {
    if (a.S == 0 || a.tiles == 0) return hipSuccess;
    return launch_type(a, bf16, true, stream);
}

}  // namespace moedisp
