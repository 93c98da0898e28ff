// Gated activation between an expert's two products, with quantisation or in
// bf16, and its gradient:
//     h = g * s * u,  s = 1 / (1 + exp(-g))
//     dg = dh * u * s * (1 + g * (1 - s)),  du = dh * g * s
// each binary32, and E4M3 codes with one scale per block of 128 channels.
//
// One pass over the rows.  A block of 128 channels belongs to 16 lanes (8
// channels, one 16-byte load of each input, per lane); its largest magnitude
// is four exchanges among them.  32768 rows of 2048: 338 MB in 71 us forward
// (4.7 TB/s; 68 us without the exponential), 769 MB in 154 us backward with
// both forms of the gradient (5.0 TB/s).  Workgroups stay resident and take
// row after row, so that the row bounds are checked once each; one workgroup
// a row took 98 us, two or four resident a unit 99 and 88.  bf16 results: 403 MB
// in 72 us (5.6 TB/s).
#include "experts_common.h"

namespace moedisp {
namespace {

constexpr int kSwigluThreads = 256;
constexpr int kUnits = kSwigluThreads / 16;  // blocks of 128 channels at a time

// Whether the row bounds keep the rules (all lanes of the workgroup get the
// answer); *rows is one past the last row of any expert.
__device__ inline bool check_bounds(const RowsArg& r, int* first, int* end) {
    bool bad = false;
    const int up = r.stride > 0 ? 0 : 1;
    for (int e = threadIdx.x; e < r.E; e += kSwigluThreads) {
        int f, c;
        bad |= !expert_rows(r, e, r.bounds[e], r.bounds[e + up], &f, &c);
    }
    const bool any = __syncthreads_or(bad);
    *first = r.stride > 0 ? 0 : r.bounds[0];
    *end = r.stride > 0 ? r.max_rows : r.bounds[r.E];
    return !any;
}

__device__ inline bool row_used(const RowsArg& r, int row) {
    if (r.stride == 0) return true;
    const int e = row / r.stride;
    const int i = row - e * r.stride - r.base;
    return i >= 0 && i < min(r.bounds[e], r.cap);
}

// s = 1 / (1 + exp(-v)), good to about one step.  exp(-v) = 2^h (1 + l ln 2)
// with h + l = -v / ln 2 to twice the bits of binary32; the quotient is
// v_rcp_f32 with one correction.  The rows' memory traffic leaves room for
// about 30 instructions per value: expf and a division are 27 of their own.
// Beyond +-87, where 2^h would leave the normal range, s is 0 or 1 (for NaN
// any: its factor v is NaN); bf16 results below take gated_below.
__device__ inline float sigmoid(float v) {
    const float x = __builtin_amdgcn_fmed3f(v, -87.0f, 87.0f);
    const float h = x * -0x1.715476p+0f;
    float l = __builtin_fmaf(x, -0x1.715476p+0f, -h);
    l = __builtin_fmaf(x, -0x1.4ae0c0p-26f, l);
    const float p = __builtin_amdgcn_exp2f(h);
    const float d = 1.0f + __builtin_fmaf(p, l * 0x1.62e430p-1f, p);
    const float r = __builtin_amdgcn_rcpf(d);
    const float s = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
    return v < -87.0f ? 0.0f : s;
}

// g * s * u for a finite g < -87, where s = exp(g) (but for a part of 2^-125) and
// may lie below binary32's normal range while the product does not: exp(g) =
// 2^n 2^f (1 + l ln 2), n + f + l = g / ln 2, and 2^n comes last.  2^-20 of u keeps
// the product before it in range; where that is inexact, the result is zero.
__device__ inline float gated_below(float g, float u) {
    const float x = fmaxf(g, -1000.0f);
    const float h = x * 0x1.715476p+0f;
    float l = __builtin_fmaf(x, 0x1.715476p+0f, -h);
    l = __builtin_fmaf(x, 0x1.4ae0c0p-26f, l);
    const float n = __builtin_rintf(h);
    const float p = __builtin_amdgcn_exp2f(h - n);
    const float e = __builtin_fmaf(p, l * 0x1.62e430p-1f, p);
    return __builtin_ldexpf(x * e * (u * 0x1p-20f), (int)n + 20);
}

__device__ inline void unpack8(v4u v, float f[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_low(v[i]);
        f[2 * i + 1] = bf16_high(v[i]);
    }
}

__device__ inline v4u pack8(const float f[8]) {
    return v4u{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// Codes and scale of a block from its 16 lanes' 8 values each.
template <int FMT>
__device__ inline void quantise(const float f[8], uint8_t* q, void* scales, size_t at, bool lead) {
    uint32_t top = 0;  // magnitudes compare as integers; NaN and infinity are the largest
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        top = max(max(__float_as_uint(f[i]) & 0x7FFFFFFFu, __float_as_uint(f[i + 1]) & 0x7FFFFFFFu), top);
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    const bool finite = top < 0x7F800000u;
    const float amax = finite ? __uint_as_float(top) : 0.0f;
    v2i out;
    float scale = 1.0f;
    int sx = 0;
    if (FMT == MOEDISP_SCALE_FP32) {
        scale = amax > 0.0f ? amax / 448.0f : 1.0f;
        // The quotient by the reciprocal: two roundings, which exceed 448 by
        // so little that E4M3 rounds it to 448.  A scale whose reciprocal
        // overflows (below 2^-127) takes the division.
        const float inv = 1.0f / scale;
        if (inv < INFINITY) {
            out.x = (int)pack4_e4m3(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
            out.y = (int)pack4_e4m3(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
        } else {
            out.x = (int)pack4_e4m3(clamp448(f[0] / scale), clamp448(f[1] / scale), clamp448(f[2] / scale),
                                    clamp448(f[3] / scale));
            out.y = (int)pack4_e4m3(clamp448(f[4] / scale), clamp448(f[5] / scale), clamp448(f[6] / scale),
                                    clamp448(f[7] / scale));
        }
    } else {
        sx = ue8m0_exponent(amax);
        out.x = (int)pack4_e4m3(clamp448(ldexpf(f[0], -sx)), clamp448(ldexpf(f[1], -sx)), clamp448(ldexpf(f[2], -sx)),
                                clamp448(ldexpf(f[3], -sx)));
        out.y = (int)pack4_e4m3(clamp448(ldexpf(f[4], -sx)), clamp448(ldexpf(f[5], -sx)), clamp448(ldexpf(f[6], -sx)),
                                clamp448(ldexpf(f[7], -sx)));
    }
    if (!finite) out = v2i{0x7F7F7F7F, 0x7F7F7F7F};
    *reinterpret_cast<v2i*>(q) = out;
    if (lead) {
        if (FMT == MOEDISP_SCALE_FP32)
            reinterpret_cast<float*>(scales)[at] = scale;
        else
            reinterpret_cast<uint8_t*>(scales)[at] = (uint8_t)(sx + 127);
    }
}

// FMT of the forward pass in bf16; rows that are read and written past the caches
constexpr int kBf16 = -1, kBf16Past = -2;

template <bool PAST>
__device__ inline v4u load16(const uint16_t* p) {
    const v4u* at = reinterpret_cast<const v4u*>(p);
    return PAST ? __builtin_nontemporal_load(at) : *at;
}

template <int FMT, bool BACKWARD>
__global__ __launch_bounds__(kSwigluThreads, BACKWARD ? 7 : 8) void moedisp_swiglu(SwigluArgs a) {
    int first, end;
    if (!check_bounds(a.r, &first, &end)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&a.hdr->status, (uint32_t)MOEDISP_DEV_BAD_LAYOUT);
        return;
    }
    const int unit = threadIdx.x >> 4;
    const int l = threadIdx.x & 15;
    // a workgroup takes a row, or several short ones, at a time
    const int rows_at_once = max(1, kUnits / a.blocks);
    const int sub = unit / a.blocks;
    if (rows_at_once > 1 && sub >= rows_at_once) return;
    const int b0 = rows_at_once > 1 ? unit - sub * a.blocks : unit;
    for (long long base = (long long)first + (long long)blockIdx.x * rows_at_once; base < end;
         base += (long long)gridDim.x * rows_at_once) {
        const int row = (int)base + (rows_at_once > 1 ? sub : 0);
        if (row >= end || !row_used(a.r, row)) continue;
        for (int b = b0; b < a.blocks; b += kUnits) {
            const int c = b * kScaleBlock + l * 8;
            float g[8], u[8], o[8];
            const v4u gv = load16<FMT == kBf16Past>(a.gu + (size_t)row * 2 * a.inner + c);
            const v4u uv = load16<FMT == kBf16Past>(a.gu + (size_t)row * 2 * a.inner + a.inner + c);
            v4u dv = {0u, 0u, 0u, 0u};
            if (BACKWARD) dv = *reinterpret_cast<const v4u*>(a.dh + (size_t)row * a.inner + c);
            __builtin_amdgcn_sched_barrier(0);  // all loads before the first use
            unpack8(gv, g);
            unpack8(uv, u);
            if (!BACKWARD) {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = g[i] * sigmoid(g[i]) * u[i];
                if constexpr (FMT < 0) {  // (codes are zero there)
                    float least = g[0];
#pragma unroll
                    for (int i = 1; i < 8; ++i) least = fminf(least, g[i]);
                    if (least < -87.0f) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (g[i] < -87.0f && g[i] > -INFINITY) o[i] = gated_below(g[i], u[i]);
                    }
                }
                v4u* const h = reinterpret_cast<v4u*>(a.h + (size_t)row * a.inner + c);
                if constexpr (FMT == kBf16)
                    *h = pack8(o);
                else if constexpr (FMT == kBf16Past)
                    __builtin_nontemporal_store(pack8(o), h);
                else
                    quantise<FMT>(o, a.q + (size_t)row * a.inner + c, a.q_scales, (size_t)row * a.blocks + b, l == 0);
            } else {
                float d[8], o2[8];
                unpack8(dv, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s = sigmoid(g[i]);
                    o[i] = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
                    o2[i] = d[i] * (g[i] * s);
                }
                if (a.dgu) {
                    *reinterpret_cast<v4u*>(a.dgu + (size_t)row * 2 * a.inner + c) = pack8(o);
                    *reinterpret_cast<v4u*>(a.dgu + (size_t)row * 2 * a.inner + a.inner + c) = pack8(o2);
                }
                if (a.q) {
                    quantise<FMT>(o, a.q + (size_t)row * 2 * a.inner + c, a.q_scales, (size_t)row * 2 * a.blocks + b,
                                  l == 0);
                    quantise<FMT>(o2, a.q + (size_t)row * 2 * a.inner + a.inner + c, a.q_scales,
                                  (size_t)row * 2 * a.blocks + a.blocks + b, l == 0);
                }
            }
        }
    }
}

template <bool BACKWARD>
hipError_t launch(const SwigluArgs& a, int scale_fmt, hipStream_t stream) {
    const long long blocks = swiglu_blocks(a.r.max_rows, a.blocks, BACKWARD);
    if (scale_fmt == MOEDISP_SCALE_UE8M0)
        hipLaunchKernelGGL((moedisp_swiglu<MOEDISP_SCALE_UE8M0, BACKWARD>), dim3((unsigned)blocks),
                           dim3(kSwigluThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((moedisp_swiglu<MOEDISP_SCALE_FP32, BACKWARD>), dim3((unsigned)blocks),
                           dim3(kSwigluThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

long long swiglu_rows_at_once(int blocks) { return blocks >= kUnits ? 1 : kUnits / blocks; }

long long swiglu_blocks(int max_rows, int blocks, bool backward) {
    const long long once = swiglu_rows_at_once(blocks);
    const long long all = ((long long)max_rows + once - 1) / once;
    const long long resident = (long long)kCus * (backward ? 7 : 8);
    return all < 1 ? 1 : all < resident ? all : resident;  // the bounds are checked even where no row can be
}

hipError_t launch_swiglu(const SwigluArgs& a, int scale_fmt, hipStream_t stream) {
    return launch<false>(a, scale_fmt, stream);
}
// Where rows and results are more than the memory-side cache holds, they go
// past the caches: 72 us instead of 80 (32768 rows of 2048, none of them cached;
// called again on the same rows 71 instead of 64 with results alone past them).
// Between an expert's two products it makes no difference: activation and second
// product of 32768 rows take 565 us either way (8 experts, 2048 -> 4096), 1687 and
// 1709 through the caches (256 experts, 2048 -> 7168); nor where few of a padded
// buffer's rows are used (32 experts, 32 of 1024 rows each: 112 and 113; 256 of
// 1024: 138 and 145), so that max_rows may decide.
hipError_t launch_swiglu_bf16(const SwigluArgs& a, hipStream_t stream) {
    const long long blocks = swiglu_blocks(a.r.max_rows, a.blocks, false);
    if ((long long)a.r.max_rows * a.inner * 6 > kCacheBytes)
        hipLaunchKernelGGL((moedisp_swiglu<kBf16Past, false>), dim3((unsigned)blocks), dim3(kSwigluThreads), 0, stream,
                           a);
    else
        hipLaunchKernelGGL((moedisp_swiglu<kBf16, false>), dim3((unsigned)blocks), dim3(kSwigluThreads), 0, stream, a);
    return hipGetLastError();
}
hipError_t launch_swiglu_backward(const SwigluArgs& a, int scale_fmt, hipStream_t stream) {
    return launch<true>(a, scale_fmt, stream);
}

}  // namespace moedisp
