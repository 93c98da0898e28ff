// Balance loss of the router and its gradient.  With c the routed slots of
// sequence s with expert e, L its tokens that are no padding, S' the sequences
// that have any, p the scores:
//     loss = coef/S' * sum_s sum_e  E c / (k L) * (1/L) sum_t p[t][e]
//     dloss/dp[t][e] = w[s][e] = coef E c / (S' k L^2)
//     softmax: dz[e] = p[e] (w[e] - sum_j p[j] w[j]);  sigmoid: the same times 1 - s(z[e])
//
// Forward: workgroups sum p and count slots over tiles of tokens, then the
// tiles are summed in their order.  Backward: one pass, the scores computed
// again from the logits.
#include "experts_common.h"

namespace moedisp {
namespace {

constexpr int kBalThreads = 256;

template <bool BF16>
__device__ inline float load_logit(const void* p, size_t i) {
    if (BF16) return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16);
    return reinterpret_cast<const float*>(p)[i];
}

// Sum (or largest) over a row's LPR lanes; every lane gets it.
template <int LPR>
__device__ inline float lanes_sum(float v) {
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) v += __shfl_xor(v, m);
    return v;
}
template <int LPR>
__device__ inline float lanes_max(float v) {
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

// Scores p and their slopes (1 for softmax, 1 - s(z) for sigmoid) of one row;
// lane l of the row's LPR lanes holds experts l, l + LPR, ...
template <int LPR, int VPL, bool BF16>
__device__ inline void row_scores(const BalanceArgs& a, size_t row, int l, float p[VPL], float slope[VPL]) {
    float z[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = v * LPR + l;
        z[v] = e < a.E ? load_logit<BF16>(a.logits, row * a.E + e) : -INFINITY;
    }
    float sum = 0.0f, m = -INFINITY;
#pragma unroll
    for (int v = 0; v < VPL; ++v) m = fmaxf(m, z[v]);
    m = lanes_max<LPR>(m);
    if (a.sigmoid) {
        // a common factor cancels: where every logit is negative the scores
        // are taken times exp(-m), so that they do not vanish together
        m = fminf(m, 0.0f);
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const float x = expf(-fabsf(z[v]));
            const float inv = 1.0f / (1.0f + x);
            slope[v] = z[v] >= 0.0f ? x * inv : inv;
            p[v] = z[v] >= 0.0f ? inv : z[v] == -INFINITY ? 0.0f : expf(z[v] - m) * inv;
            sum += p[v];
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            p[v] = z[v] == -INFINITY ? 0.0f : expf(z[v] - m);
            slope[v] = 1.0f;
            sum += p[v];
        }
    }
    sum = lanes_sum<LPR>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // no score at all: p = 0
#pragma unroll
    for (int v = 0; v < VPL; ++v) p[v] *= inv;
}

// Forward, first launch: the score sums [E], slot counts [E] and token count
// of one tile.
template <int LPR, int VPL, bool BF16>
__global__ __launch_bounds__(kBalThreads) void moedisp_balance_tile(BalanceArgs a) {
    constexpr int kRows = kBalThreads / LPR;  // rows at a time
    extern __shared__ float s_p[];            // [kRows][E], then int [E], int
    int* s_c = reinterpret_cast<int*>(s_p + kRows * a.E);
    int* s_n = s_c + a.E;
    const int tid = threadIdx.x;
    const int seq = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int t0 = tile * a.tile_tokens, t1 = min(a.L, t0 + a.tile_tokens);
    for (int e = tid; e < a.E + 1; e += kBalThreads) s_c[e] = 0;
    __syncthreads();
    const int l = tid % LPR, r = tid / LPR;
    float acc[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] = 0.0f;
    bool bad = false;
    for (int t = t0 + r; t < t1; t += kRows) {
        const size_t row = (size_t)seq * a.L + t;
        int routed = 0;
        for (int j = l; j < a.k; j += LPR) {
            const int id = a.topk_idx[row * a.k + j];
            if (id >= 0 && id < a.E) {
                atomicAdd(&s_c[id], 1);
                routed = 1;
            } else if (id != -1) {
                bad = true;
            }
        }
#pragma unroll
        for (int m = 1; m < LPR; m <<= 1) routed |= __shfl_xor(routed, m);
        if (!routed) continue;  // all of the row's lanes
        if (l == 0) atomicAdd(s_n, 1);
        float p[VPL], slope[VPL];
        row_scores<LPR, VPL, BF16>(a, row, l, p, slope);
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] += p[v];
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        if (v * LPR + l < a.E) s_p[r * a.E + v * LPR + l] = acc[v];
    if (bad) atomicOr(&a.hdr->status, (uint32_t)MOEDISP_DEV_BAD_EXPERT_ID);
    __syncthreads();
    for (int e = tid; e < a.E; e += kBalThreads) {
        float sum = 0.0f;
        for (int i = 0; i < kRows; ++i) sum += s_p[i * a.E + e];
        a.psum[(size_t)blockIdx.x * a.E + e] = sum;
        a.count[(size_t)blockIdx.x * a.E + e] = s_c[e];
    }
    if (tid == 0) a.tokens[blockIdx.x] = *s_n;
}

__device__ inline double block_sum(double v, double* s) {
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < (int)blockDim.x / 64; ++w) t += s[w];
    return t;
}

// Forward, second launch: one workgroup per sequence sums its tiles.
__global__ __launch_bounds__(1024) void moedisp_balance_seq(BalanceArgs a) {
    __shared__ double s_sum[16];
    const int seq = blockIdx.x, tid = threadIdx.x;
    long long n = 0;
    for (int t = 0; t < a.tiles; ++t) n += a.tokens[(size_t)seq * a.tiles + t];
    double part = 0.0;
    for (int e = tid; e < a.E; e += blockDim.x) {
        double p = 0.0;
        int c = 0;
        for (int t = 0; t < a.tiles; ++t) {
            const size_t at = ((size_t)seq * a.tiles + t) * a.E + e;
            p += a.psum[at];
            c += a.count[at];
        }
        a.tokens_per_expert[(size_t)seq * a.E + e] = c;
        part += p * c;
    }
    const double sum = block_sum(part, s_sum);
    if (tid == 0) {
        a.tokens_per_seq[seq] = (int)n;
        a.seq_loss[seq] = n > 0 ? (float)(sum * a.E / ((double)a.k * n * n)) : 0.0f;
    }
}

// Forward, third launch: the mean over the sequences.
__global__ __launch_bounds__(256) void moedisp_balance_loss(BalanceArgs a) {
    __shared__ double s_sum[4];
    double part = 0.0, some = 0.0;
    for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
        part += a.seq_loss[s];
        some += a.tokens_per_seq[s] > 0 ? 1.0 : 0.0;
    }
    const double sum = block_sum(part, s_sum);
    const double n = block_sum(some, s_sum);
    if (threadIdx.x == 0) *a.loss = n > 0.0 ? (float)(a.coef * sum / n) : 0.0f;
}

// Backward.
template <int LPR, int VPL, bool BF16>
__global__ __launch_bounds__(kBalThreads) void moedisp_balance_backward(BalanceArgs a) {
    constexpr int kRows = kBalThreads / LPR;
    __shared__ double s_sum[4];
    const int tid = threadIdx.x;
    const int seq = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int t0 = tile * a.tile_tokens, t1 = min(a.L, t0 + a.tile_tokens);
    double some = 0.0;
    for (int s = tid; s < a.S; s += kBalThreads) some += a.tokens_per_seq[s] > 0 ? 1.0 : 0.0;
    some = block_sum(some, s_sum);
    const double n = a.tokens_per_seq[seq];
    const float scale = n > 0.0 ? (float)((double)a.coef * a.E * *a.d_loss / (some * a.k * n * n)) : 0.0f;
    const int l = tid % LPR, r = tid / LPR;
    float w[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = v * LPR + l;
        w[v] = e < a.E ? scale * (float)a.tokens_per_expert[(size_t)seq * a.E + e] : 0.0f;
    }
    for (int t = t0 + r; t < t1; t += kRows) {
        const size_t row = (size_t)seq * a.L + t;
        int routed = 0;
        for (int j = l; j < a.k; j += LPR) {
            const int id = a.topk_idx[row * a.k + j];
            routed |= id >= 0 && id < a.E;
        }
#pragma unroll
        for (int m = 1; m < LPR; m <<= 1) routed |= __shfl_xor(routed, m);
        float p[VPL], slope[VPL];
        float dot = 0.0f;
        if (routed) {
            row_scores<LPR, VPL, BF16>(a, row, l, p, slope);
#pragma unroll
            for (int v = 0; v < VPL; ++v) dot += p[v] * w[v];
            dot = lanes_sum<LPR>(dot);
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = v * LPR + l;
            if (e >= a.E) continue;
            const float dz = routed ? p[v] * slope[v] * (w[v] - dot) : 0.0f;
            if (BF16)
                reinterpret_cast<uint16_t*>(a.d_logits)[row * a.E + e] = (uint16_t)pack_bf16x2(dz, 0.0f);
            else
                reinterpret_cast<float*>(a.d_logits)[row * a.E + e] = dz;
        }
    }
}

template <int LPR, int VPL, bool BF16>
hipError_t launch_pass(const BalanceArgs& a, bool backward, hipStream_t stream) {
    const long long blocks = (long long)a.S * a.tiles;
    if (!grid_fits(blocks, kBalThreads)) return hipErrorInvalidConfiguration;
    if (backward) {
        hipLaunchKernelGGL((moedisp_balance_backward<LPR, VPL, BF16>), dim3((unsigned)blocks), dim3(kBalThreads), 0,
                           stream, a);
    } else {
        const size_t lds = ((size_t)(kBalThreads / LPR) * a.E + a.E + 1) * 4;
        hipLaunchKernelGGL((moedisp_balance_tile<LPR, VPL, BF16>), dim3((unsigned)blocks), dim3(kBalThreads), lds,
                           stream, a);
    }
    return hipGetLastError();
}

// Lanes per row: at most 4 experts a lane up to 256 experts, a wave per row
// beyond.
template <bool BF16>
hipError_t launch_rows(const BalanceArgs& a, bool backward, hipStream_t stream) {
    if (a.E <= 8) return launch_pass<2, 4, BF16>(a, backward, stream);
    if (a.E <= 16) return launch_pass<4, 4, BF16>(a, backward, stream);
    if (a.E <= 32) return launch_pass<8, 4, BF16>(a, backward, stream);
    if (a.E <= 64) return launch_pass<16, 4, BF16>(a, backward, stream);
    if (a.E <= 128) return launch_pass<32, 4, BF16>(a, backward, stream);
    if (a.E <= 256) return launch_pass<64, 4, BF16>(a, backward, stream);
    if (a.E <= 512) return launch_pass<64, 8, BF16>(a, backward, stream);
    if (a.E <= 1024) return launch_pass<64, 16, BF16>(a, backward, stream);
    return launch_pass<64, 64, BF16>(a, backward, stream);
}

}  // namespace

hipError_t launch_balance(const BalanceArgs& a, bool bf16, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.S > 0 && a.tiles > 0) e = bf16 ? launch_rows<true>(a, false, stream) : launch_rows<false>(a, false, stream);
    if (e != hipSuccess) return e;
    if (a.S > 0) {
        hipLaunchKernelGGL(moedisp_balance_seq, dim3(a.S), dim3(1024), 0, stream, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(moedisp_balance_loss, dim3(1), dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, bool bf16, hipStream_t stream) {
    if (a.S == 0 || a.tiles == 0) return hipSuccess;
    return bf16 ? launch_rows<true>(a, true, stream) : launch_rows<false>(a, true, stream);
}

}  // namespace moedisp
