// Weight gradient of the experts' product:
//     dw[e][n][k] (+)= sum over e's rows r of dy[r][n] * sx[r][k/128] * x[r][k]
#include "experts_common.h"

namespace moedisp {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kT = 256;     // tile: 256 columns of dy by 256 channels of x
constexpr int kStep = 32;   // rows per step
constexpr int kWaves = 8;   // waves 0..3 stage dy, 4..7 stage x; each multiplies 64 columns by 128 channels

// Position of column (or channel) i of the tile among the 256 16-byte units
// of one group of 8 rows.  A lane that stages writes units 4l..4l+3 and the
// operand reads take 16 units whose low bits run over {0,1,2,3} or {0,1,3,4}:
// mixing bits 4 and 5 into the low ones puts 16 neighbouring lanes of either
// on 16 different units modulo 16, so that no two share LDS banks.
__device__ inline int unit_of(int i) { return i ^ ((i & 16) ? 5 : 0) ^ ((i & 32) ? 2 : 0); }

__device__ inline uint32_t perm_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ inline uint32_t perm_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

template <int FMT, bool F32, bool ADD>
__global__ __launch_bounds__(64 * kWaves) void moedisp_expert_wgrad(ExpertWgradArgs a) {
    __shared__ v4u lds[2][2][kStep / 8][kT];  // [buffer][dy, x][rows / 8][unit]
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    int incl, own;
    const int rows_total = expert_tiles<1>(a.r, &incl, &own);
    if (rows_total < 0) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(&a.hdr->status, (uint32_t)MOEDISP_DEV_BAD_LAYOUT);
        return;
    }
    const int per_expert = a.nt * a.kt;
    const int e = blockIdx.x / per_expert;
    const int rest = blockIdx.x - e * per_expert;
    const int n0 = (rest / a.kt) * kT, k0 = (rest % a.kt) * kT;
    int first, rows;
    expert_rows(a.r, e, a.r.bounds[e], a.r.bounds[a.r.stride > 0 ? e : e + 1], &first, &rows);
    first = __builtin_amdgcn_readfirstlane(first);
    rows = __builtin_amdgcn_readfirstlane(rows);

    // staging: a wave takes 8 rows; a lane 4 columns of dy or 4 channels of x
    const bool is_x = wave >= 4;
    const int g = wave & 3;
    const int c4 = 4 * lane;
    const int col = is_x ? min(k0 + c4, a.k - 4) : min(n0 + c4, a.n - 4);
    v2i d[8];
    float sc[8];
    auto load = [&](int step) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = step * kStep + g * 8 + i;
            const size_t row = (size_t)first + min(r, rows - 1);
            if (is_x) {
                d[i].x = *reinterpret_cast<const int*>(a.x + row * a.k + col);
                const size_t at = row * a.kb + col / kScaleBlock;
                sc[i] = FMT == MOEDISP_SCALE_FP32
                            ? reinterpret_cast<const float*>(a.x_scales)[at]
                            : ue8m0_value(reinterpret_cast<const uint8_t*>(a.x_scales)[at]);
            } else {
                d[i] = *reinterpret_cast<const v2i*>(a.dy + row * a.n + col);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (step * kStep + g * 8 + i >= rows) d[i] = v2i{0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (step * kStep + g * 8 + i >= rows) sc[i] = 0.0f;
    };
    auto stage = [&](int buf) {
        v4u u[4];
        if (is_x) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const v2f lo0 = __builtin_amdgcn_cvt_pk_f32_fp8(d[2 * p].x, false);
                const v2f hi0 = __builtin_amdgcn_cvt_pk_f32_fp8(d[2 * p].x, true);
                const v2f lo1 = __builtin_amdgcn_cvt_pk_f32_fp8(d[2 * p + 1].x, false);
                const v2f hi1 = __builtin_amdgcn_cvt_pk_f32_fp8(d[2 * p + 1].x, true);
                const float s0 = sc[2 * p], s1 = sc[2 * p + 1];
                u[0][p] = pack_bf16x2(lo0.x * s0, lo1.x * s1);
                u[1][p] = pack_bf16x2(lo0.y * s0, lo1.y * s1);
                u[2][p] = pack_bf16x2(hi0.x * s0, hi1.x * s1);
                u[3][p] = pack_bf16x2(hi0.y * s0, hi1.y * s1);
            }
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const v2i r0 = d[2 * p], r1 = d[2 * p + 1];
                u[0][p] = perm_lo(r0.x, r1.x);
                u[1][p] = perm_hi(r0.x, r1.x);
                u[2][p] = perm_lo(r0.y, r1.y);
                u[3][p] = perm_hi(r0.y, r1.y);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) lds[buf][is_x ? 1 : 0][g][unit_of(c4 + i)] = u[i];
    };

    constexpr int kKT = 8, kNT = 4;  // 16-wide tiles of a wave: channels, columns
    const int wk = (wave & 1) * 128, wn = (wave >> 1) * 64;
    v4f acc[kKT][kNT];
#pragma unroll
    for (int i = 0; i < kKT; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int q = lane >> 4, c = lane & 15;
    const int steps = (rows + kStep - 1) / kStep;
    if (steps > 0) {
        load(0);
        stage(0);
    }
    for (int s = 0; s < steps; ++s) {
        __syncthreads();
        if (s + 1 < steps) load(s + 1);
        v8bf b[kNT];
#pragma unroll
        for (int j = 0; j < kNT; ++j)
            b[j] = __builtin_bit_cast(v8bf, lds[s & 1][0][q][unit_of(wn + j * 16 + c)]);
#pragma unroll
        for (int i = 0; i < kKT; ++i) {
            const int ch = wk + (i >> 1) * 32 + (c >> 2) * 8 + (i & 1) * 4 + (c & 3);
            const v8bf av = __builtin_bit_cast(v8bf, lds[s & 1][1][q][unit_of(ch)]);
#pragma unroll
            for (int j = 0; j < kNT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, b[j], acc[i][j], 0, 0, 0);
        }
        if (s + 1 < steps) stage((s + 1) & 1);
    }

#pragma unroll
    for (int j = 0; j < kNT; ++j) {
        const int n = n0 + wn + j * 16 + c;
        if (n >= a.n) continue;
#pragma unroll
        for (int t = 0; t < kKT / 2; ++t) {
            const int k = k0 + wk + t * 32 + q * 8;
            if (k >= a.k) continue;
            const size_t at = ((size_t)e * a.n + n) * a.k + k;
            v4f lo = acc[2 * t][j], hi = acc[2 * t + 1][j];
            if (F32) {
                v4f* o = reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.dw) + at);
                if (ADD) {
                    lo += o[0];
                    hi += o[1];
                }
                o[0] = lo;
                o[1] = hi;
            } else {
                const v4u v = {pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]),
                               pack_bf16x2(hi[2], hi[3])};
                *reinterpret_cast<v4u*>(reinterpret_cast<uint16_t*>(a.dw) + at) = v;
            }
        }
    }
}

template <int FMT, bool F32, bool ADD>
hipError_t launch_one(ExpertWgradArgs a, hipStream_t stream) {
    a.nt = (a.n + kT - 1) / kT;
    a.kt = (a.k + kT - 1) / kT;
    const long long blocks = (long long)a.r.E * a.nt * a.kt;
    if (!grid_fits(blocks, 64 * kWaves)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((moedisp_expert_wgrad<FMT, F32, ADD>), dim3((unsigned)blocks), dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

template <int FMT>
hipError_t launch_fmt(const ExpertWgradArgs& a, bool f32_out, bool accumulate, hipStream_t stream) {
    if (!f32_out) return launch_one<FMT, false, false>(a, stream);
    return accumulate ? launch_one<FMT, true, true>(a, stream) : launch_one<FMT, true, false>(a, stream);
}

}  // namespace

hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, int scale_fmt, bool f32_out, bool accumulate,
                               hipStream_t stream) {
    return scale_fmt == MOEDISP_SCALE_UE8M0 ? launch_fmt<MOEDISP_SCALE_UE8M0>(a, f32_out, accumulate, stream)
                                            : launch_fmt<MOEDISP_SCALE_FP32>(a, f32_out, accumulate, stream);
}

}  // namespace moedisp
