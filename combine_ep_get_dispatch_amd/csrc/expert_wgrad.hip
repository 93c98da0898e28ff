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

// Scale number `at` where it is the same in all lanes: a scalar load (of the
// aligned word that holds it).
template <int FMT>
__device__ inline float uniform_scale(const void* p, size_t at) {
    typedef const __attribute__((address_space(4))) uint32_t* cptr;
    if (FMT == MOEDISP_SCALE_FP32) return __uint_as_float(((cptr)(uintptr_t)p)[at]);
    const uintptr_t b = (uintptr_t)p + at;
    return ue8m0_value((*(cptr)(b & ~(uintptr_t)3) >> ((b & 3) * 8)) & 255u);
}

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

    // Staging: a wave takes 8 rows of a step; a lane 4 columns of dy or 4
    // channels of x.  Rows past the expert's last lie past the end of the
    // step's buffer and read as zero; columns past a row's end hold what
    // follows in memory and go into results that are not stored.
    const bool is_x = wave >= 4;
    const int g = wave & 3;
    const int c4 = 4 * lane;
    const int rb = is_x ? a.k : a.n * 2;  // bytes of a row
    const int c0 = is_x ? k0 + c4 : (n0 + c4) * 2;
    v2i d[2][8];
    float sc[2][8][2];
    const int steps = (rows + kStep - 1) / kStep;
    auto load = [&](int step, int u) {
        if (step >= steps) return;
        const int r0 = step * kStep + g * 8;
        const int left = max(0, min(8, rows - r0));
        const size_t row = (size_t)first + min(r0, rows - 1);
        const char* base = (is_x ? (const char*)a.x : (const char*)a.dy) + row * rb;
        const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, left * rb, kRawBufferWord3);
        if (is_x) {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[u][i].x = (int)__builtin_amdgcn_raw_buffer_load_b32(rs, c0 + i * rb, 0, 0);
            // the two scales of each row that the tile spans, by scalar loads
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const size_t at = ((size_t)first + min(r0 + i, rows - 1)) * a.kb;
                const int b0 = k0 / kScaleBlock, b1 = min(b0 + 1, a.kb - 1);
                sc[u][i][0] = uniform_scale<FMT>(a.x_scales, at + b0);
                sc[u][i][1] = uniform_scale<FMT>(a.x_scales, at + b1);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[u][i] = __builtin_bit_cast(v2i, __builtin_amdgcn_raw_buffer_load_b64(rs, c0 + i * rb, 0, 0));
        }
    };
    auto stage = [&](int step, int u) {
        if (step >= steps) return;
        v4u o[4];
        if (is_x) {
            const bool second = lane >= 32;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const v2f lo0 = __builtin_amdgcn_cvt_pk_f32_fp8(d[u][2 * p].x, false);
                const v2f hi0 = __builtin_amdgcn_cvt_pk_f32_fp8(d[u][2 * p].x, true);
                const v2f lo1 = __builtin_amdgcn_cvt_pk_f32_fp8(d[u][2 * p + 1].x, false);
                const v2f hi1 = __builtin_amdgcn_cvt_pk_f32_fp8(d[u][2 * p + 1].x, true);
                const int r = step * kStep + g * 8 + 2 * p;
                const float s0 = r < rows ? (second ? sc[u][2 * p][1] : sc[u][2 * p][0]) : 0.0f;
                const float s1 = r + 1 < rows ? (second ? sc[u][2 * p + 1][1] : sc[u][2 * p + 1][0]) : 0.0f;
                o[0][p] = pack_bf16x2(lo0.x * s0, lo1.x * s1);
                o[1][p] = pack_bf16x2(lo0.y * s0, lo1.y * s1);
                o[2][p] = pack_bf16x2(hi0.x * s0, hi1.x * s1);
                o[3][p] = pack_bf16x2(hi0.y * s0, hi1.y * s1);
            }
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const v2i r0 = d[u][2 * p], r1 = d[u][2 * p + 1];
                o[0][p] = perm_lo(r0.x, r1.x);
                o[1][p] = perm_hi(r0.x, r1.x);
                o[2][p] = perm_lo(r0.y, r1.y);
                o[3][p] = perm_hi(r0.y, r1.y);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) lds[step & 1][is_x ? 1 : 0][g][unit_of(c4 + i)] = o[i];
    };

    constexpr int kKT = 8, kNT = 4;  // 16-wide tiles of a wave: channels, columns
    const int wk = (wave & 1) * 128, wn = (wave >> 1) * 64;
    v4f acc[kKT][kNT];
#pragma unroll
    for (int i = 0; i < kKT; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int q = lane >> 4, c = lane & 15;
    load(0, 0);
    load(1, 1);
    stage(0, 0);
    load(2, 0);
    for (int s0 = 0; s0 < steps; s0 += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int s = s0 + h;
            if (s >= steps) break;
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            // the waves of x have the conversions: they stage before their
            // products, those of dy behind them, so that one of the two waves
            // of a SIMD unit keeps the matrix unit busy
            if (is_x) {
                stage(s + 1, h ^ 1);
                load(s + 3, h ^ 1);
            }
            v8bf b[kNT];
#pragma unroll
            for (int j = 0; j < kNT; ++j) b[j] = __builtin_bit_cast(v8bf, lds[h][0][q][unit_of(wn + j * 16 + c)]);
#pragma unroll
            for (int i = 0; i < kKT; ++i) {
                const int ch = wk + (i >> 1) * 32 + (c >> 2) * 8 + (i & 1) * 4 + (c & 3);
                const v8bf av = __builtin_bit_cast(v8bf, lds[h][1][q][unit_of(ch)]);
#pragma unroll
                for (int j = 0; j < kNT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, b[j], acc[i][j], 0, 0, 0);
            }
            if (!is_x) {
                stage(s + 1, h ^ 1);
                load(s + 3, h ^ 1);
            }
        }
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
