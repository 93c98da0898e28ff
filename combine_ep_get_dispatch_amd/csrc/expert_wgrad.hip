// Weight gradient of the experts' product:
//     dw[e][n][k] (+)= sum over e's rows r of dy[r][n] * sx[r][k/128] * x[r][k]
//
// Precision.  The scales belong to rows, over which is summed, so they cannot
// wait until after a matrix instruction: x becomes bf16, scale times code
// rounded once (by 2^-8 of itself at most; exact for powers of two), and the
// products are those of the bf16 instruction, added in binary32.  bf16
// results, rounded as much themselves, take that.  fp32 results of FP32 scales
// keep binary32's error, over micro-batches too: x becomes a sum of three bf16
// terms, exact to binary32, and each has its product.
//
// What bounds it.  Many rows (32768 over 8 experts, 4096 x 4096): 1.07 ms, 1.0
// PFLOP/s; products alone 0.78 ms, loads and LDS alone 0.91 ms.  Few rows (7782
// over 64 experts, 7168 x 2048, fp32): the 3.8 GB of results, 0.94 ms, 4.1 TB/s.
// Three terms: the products, 3.3 and 1.65 ms at these sizes.  An expert's rows
// are not split, so that a few small experts, or one much longer than the
// others, leave units without work.
//
// How.  A workgroup computes one tile over all rows of its expert, 32 rows a
// step, three steps of loads under way.  Both operands are contracted over
// rows, which is across the way they lie: LDS holds them by rows and the
// transposing reads of the matrix operands turn them (registers that gather 8
// rows a lane before LDS took 1.59 ms).  x passes through registers to be
// widened, once per tile, between the products.
#include "experts_common.h"

namespace moedisp {
namespace {

constexpr int kStep = 32;    // rows per step: the contraction of one matrix instruction
constexpr int kStages = 4;   // steps under way or in use

// Terms of scale times code: one, but three for fp32 results of FP32 scales.
constexpr int wgrad_terms(int fmt, bool f32) { return fmt == MOEDISP_SCALE_FP32 && f32 ? 3 : 1; }

// Two values as pairs of bf16 terms of eight bits each, cut off one after the
// other, so that every step is exact and three terms hold binary32's 24 bits.
template <int TERMS>
__device__ inline void bf16_terms(float v0, float v1, uint32_t o[TERMS]) {
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
        const uint32_t b0 = __float_as_uint(v0), b1 = __float_as_uint(v1);
        o[t] = (b0 >> 16) | (b1 & 0xFFFF0000u);
        // infinity and NaN are their first term alone
        v0 = t > 0 || fabsf(v0) < INFINITY ? v0 - __uint_as_float(b0 & 0xFFFF0000u) : 0.0f;
        v1 = t > 0 || fabsf(v1) < INFINITY ? v1 - __uint_as_float(b1 & 0xFFFF0000u) : 0.0f;
    }
}

// Tile of TN columns of dy by TK channels of x; WN x WK waves; x as a sum of
// TERMS bf16 values.
template <int TN, int TK, int WN, int WK, int TERMS>
struct WTile {
    static constexpr int kWaves = WN * WK;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int kNT = TN / WN / 16;   // 16-wide tiles of a wave
    static constexpr int kKT = TK / WK / 16;
    static constexpr int kDyRow = TN * 2;      // bytes
    static constexpr int kXRow = TK * 2;
    static constexpr int kDyStage = kStep * kDyRow;
    static constexpr int kXStage = kStep * kXRow;
    static constexpr int kDyLoads = kDyStage / 1024 / kWaves;  // of a wave and step
    static constexpr int kXLanes = TK / 16;                    // lanes of a row, 16 channels each
    static constexpr int kXRows = 64 / kXLanes;                // rows of a wave and step
    static constexpr int kOps = kDyLoads + 2;                  // loads of a wave and step
    static constexpr int kXRaw = 1024 + 256;                   // a wave's codes and scales of a step
    static constexpr int kLds = kStages * (kDyStage + kWaves * kXRaw) + 2 * TERMS * kXStage;
    static_assert(kKT >= 4 && kKT % 2 == 0 && kXRows * kWaves == kStep && kDyRow >= 256 && kXRow >= 256, "tile shape");
};

template <int TN, int TK, int WN, int WK, int FMT, bool F32, bool ADD>
__global__ __launch_bounds__(64 * WN * WK) void moedisp_expert_wgrad(ExpertWgradArgs a) {
    constexpr int TERMS = wgrad_terms(FMT, F32);
    using T = WTile<TN, TK, WN, WK, TERMS>;
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    int incl, own;
    if (expert_tiles<1>(a.r, &incl, &own) < 0) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(&a.hdr->status, (uint32_t)MOEDISP_DEV_BAD_LAYOUT);
        return;
    }
    // XCD x (consecutive workgroups go round the XCDs) takes every 8th run of
    // kRun tiles, neighbours of kGroup column tiles by kRun / kGroup channel
    // tiles that share their rows in its L2.  Short runs: experts' rows are
    // uneven, and so is the work of a run.
    constexpr int kRun = 32, kGroup = 4;
    const int local = blockIdx.x / kXcds;
    const long long item = ((long long)(local / kRun) * kXcds + blockIdx.x % kXcds) * kRun + local % kRun;
    const int per_expert = a.nt * a.kt;
    if (item >= (long long)a.r.E * per_expert) return;
    const int e = (int)(item / per_expert);
    const int rest = (int)(item - (long long)e * per_expert);
    const int grp = rest / (kGroup * a.kt);
    const int gn = min(kGroup, a.nt - grp * kGroup);
    const int in_grp = rest - grp * kGroup * a.kt;
    const int n0 = (grp * kGroup + in_grp % gn) * TN, k0 = (in_grp / gn) * TK;
    int first, rows;
    expert_rows(a.r, e, a.r.bounds[e], a.r.bounds[a.r.stride > 0 ? e : e + 1], &first, &rows);
    first = __builtin_amdgcn_readfirstlane(first);
    rows = __builtin_amdgcn_readfirstlane(rows);
    const int steps = (rows + kStep - 1) / kStep;

    // dy: rows as they are, straight into LDS.  Load i of the wave brings
    // 1 KiB; rows past the expert's last are read as its last, and count
    // nothing as x is zero there.
    int dy_row[T::kDyLoads], dy_col[T::kDyLoads];
#pragma unroll
    for (int i = 0; i < T::kDyLoads; ++i) {
        const int at = (wave * T::kDyLoads + i) * 1024 + lane * 16;
        dy_row[i] = at / T::kDyRow;
        const int chunk = (at % T::kDyRow / 16) ^ (unit_swizzle(dy_row[i]) << 1);
        dy_col[i] = min(chunk * 16, (a.n - n0) * 2 - 16);
    }
    auto load_dy = [&](int step, int buf) {
        const int r0 = min(step * kStep, rows - 1);
        const char* base = (const char*)a.dy + (((size_t)first + r0) * a.n + n0) * 2;
#pragma unroll
        for (int i = 0; i < T::kDyLoads; ++i)
            load_to_lds_unseen<16>(base, lds + buf * T::kDyStage + (wave * T::kDyLoads + i) * 1024,
                                   min(dy_row[i], rows - 1 - r0) * (a.n * 2) + dy_col[i]);
    };
    // x: 16 channels of a row and their scale per lane, to a place of the
    // wave's own; from there they become bf16 (scale times code, rounded
    // once), zero past the expert's last row
    constexpr int SB = FMT == MOEDISP_SCALE_FP32 ? 4 : 1;
    char* const raw = lds + kStages * T::kDyStage + 2 * TERMS * T::kXStage + wave * (kStages * T::kXRaw);
    const int x_row = wave * T::kXRows + lane / T::kXLanes;
    const int x_ch = min(k0 + lane % T::kXLanes * 16, a.k - 16);
    auto load_x = [&](int step, int u) {
        const int r0 = min(step * kStep, rows - 1);
        const int row = min(x_row, rows - 1 - r0);
        load_to_lds_unseen<16>(a.x + ((size_t)first + r0) * a.k, raw + u * T::kXRaw, row * a.k + x_ch);
        load_to_lds_unseen<SB>((const char*)a.x_scales + ((size_t)first + r0) * a.kb * SB, raw + u * T::kXRaw + 1024,
                               (row * a.kb + x_ch / kScaleBlock) * SB);
    };
    // bf16 results: unit 2p holds channels 0-3, 8-11, 16-19, 24-27 of 32 and
    // unit 2p + 1 the others, so that two products give a lane 8 neighbours,
    // 16 bytes to store (4 lanes 64 bytes; in order it would be 32)
    constexpr bool kPairs = !F32;
    char* const x_lds = lds + kStages * T::kDyStage;
    const int x_unit = lane % T::kXLanes, x_sw = unit_swizzle(x_row);
    const int x_at[2] = {
        x_row * T::kXRow + (kPairs ? ((x_unit & ~1) ^ x_sw) * 32 + (x_unit & 1) * 16 : (x_unit ^ x_sw) * 32),
        x_row * T::kXRow + (kPairs ? ((x_unit | 1) ^ x_sw) * 32 + (x_unit & 1) * 16 : (x_unit ^ x_sw) * 32 + 16)};
    const bool x_half = lane & 8;  // which 16 bytes first: 16 neighbours fill different banks
    auto stage_x = [&](int step, int u) {
        const v4u xr = *reinterpret_cast<const v4u*>(raw + u * T::kXRaw + lane * 16);
        const int xs = *reinterpret_cast<const int*>(raw + u * T::kXRaw + 1024 + lane * 4);
        const float s = FMT == MOEDISP_SCALE_FP32 ? __int_as_float(xs) : ue8m0_value((uint32_t)xs);
        const uint32_t on = step * kStep + x_row < rows ? 0xFFFFFFFFu : 0u;
        if constexpr (TERMS == 1) {
            v4u o[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)xr[i], false);
                const v2f hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)xr[i], true);
                o[i >> 1][2 * (i & 1)] = pack_bf16x2(lo.x * s, lo.y * s) & on;
                o[i >> 1][2 * (i & 1) + 1] = pack_bf16x2(hi.x * s, hi.y * s) & on;
            }
            if (kPairs) {
                const v4u t = {o[0][0], o[0][1], o[1][0], o[1][1]};
                o[1] = v4u{o[0][2], o[0][3], o[1][2], o[1][3]};
                o[0] = t;
            }
            char* to = x_lds + (step & 1) * T::kXStage;
            *reinterpret_cast<v4u*>(to + (x_half ? x_at[1] : x_at[0])) = x_half ? o[1] : o[0];
            *reinterpret_cast<v4u*>(to + (x_half ? x_at[0] : x_at[1])) = x_half ? o[0] : o[1];
        } else {
            v4u o[TERMS][2];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const v2f v = i & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)xr[i >> 1], true)
                                    : __builtin_amdgcn_cvt_pk_f32_fp8((int)xr[i >> 1], false);
                uint32_t a[TERMS];
                bf16_terms<TERMS>(v.x * s, v.y * s, a);
#pragma unroll
                for (int t = 0; t < TERMS; ++t) o[t][i >> 2][i & 3] = a[t] & on;
            }
#pragma unroll
            for (int t = 0; t < TERMS; ++t) {
                char* to = x_lds + ((step & 1) * TERMS + t) * T::kXStage;
                *reinterpret_cast<v4u*>(to + (x_half ? x_at[1] : x_at[0])) = x_half ? o[t][1] : o[t][0];
                *reinterpret_cast<v4u*>(to + (x_half ? x_at[0] : x_at[1])) = x_half ? o[t][0] : o[t][1];
            }
        }
    };

    const int wk = wave % WK * (TK / WK), wn = wave / WK * (TN / WN);
    v4f acc[T::kKT][T::kNT];
#pragma unroll
    for (int i = 0; i < T::kKT; ++i)
#pragma unroll
        for (int j = 0; j < T::kNT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int q = lane >> 4, c = lane & 15;
    // the lane's place in the transposing reads of rows 8q + c/4 (and + 4)
    const int tr_row = q * 8 + (c >> 2);
    const int tr_sw = unit_swizzle(tr_row);  // the same 4 rows below
    // 8 rows of column (or channel) c of unit u
    auto operand = [&](const char* st, int row_bytes, int u) {
        const char* p = st + tr_row * row_bytes + ((u ^ tr_sw) << 5) + ((c & 3) << 3);
        const v4s lo = read_transposed(p);
        const v4s hi = read_transposed(p + 4 * row_bytes);
        return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };

    if (steps > 0) {
#pragma unroll
        for (int p = 0; p < kStages - 1; ++p) {
            load_x(p, p);
            load_dy(p, p);
        }
        wait_own_loads<(kStages - 2) * T::kOps>();
        stage_x(0, 0);
        wait_loads_and_sync<(kStages - 2) * T::kOps>();
        for (int s0 = 0; s0 < steps; s0 += kStages) {
#pragma unroll
            for (int h = 0; h < kStages; ++h) {
                const int s = s0 + h;
                if (s >= steps) break;
                const char* ds = lds + h * T::kDyStage;
                const char* xst = x_lds + (h & 1) * TERMS * T::kXStage;
                v8bf b[T::kNT], av[2][TERMS];
#pragma unroll
                for (int j = 0; j < T::kNT; ++j) b[j] = operand(ds, T::kDyRow, wn / 16 + j);
                av[0][0] = operand(xst, T::kXRow, wk / 16);
#pragma unroll
                for (int t = 1; t < TERMS; ++t) av[0][t] = operand(xst + t * T::kXStage, T::kXRow, wk / 16);
#pragma unroll
                for (int i = 0; i < T::kKT; ++i) {
                    if (i + 1 < T::kKT) av[(i + 1) & 1][0] = operand(xst, T::kXRow, wk / 16 + i + 1);
#pragma unroll
                    for (int t = 1; t < TERMS; ++t)
                        if (i + 1 < T::kKT)
                            av[(i + 1) & 1][t] = operand(xst + t * T::kXStage, T::kXRow, wk / 16 + i + 1);
#pragma unroll
                    for (int j = 0; j < T::kNT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[i & 1][0], b[j], acc[i][j], 0, 0, 0);
#pragma unroll
                    for (int t = 1; t < TERMS; ++t)
#pragma unroll
                        for (int j = 0; j < T::kNT; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[i & 1][t], b[j], acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    // behind the products: step s + 3 into the place of step
                    // s - 1, which all waves have read; x of step s + 1
                    if (i == 0) load_x(s + kStages - 1, (h + kStages - 1) % kStages);
                    if (i == 1) load_dy(s + kStages - 1, (h + kStages - 1) % kStages);
                    if (i == 2) {
                        wait_own_loads<(kStages - 2) * T::kOps>();
                        stage_x(s + 1, (h + 1) % kStages);
                    }
                    if (i < 3) __builtin_amdgcn_sched_barrier(0);
                }
                wait_loads_and_sync<(kStages - 2) * T::kOps>();
            }
        }
        wait_loads_and_sync<0>();  // no load may reach LDS after the workgroup's end
    }

#pragma unroll
    for (int j = 0; j < T::kNT; ++j) {
        const int n = n0 + wn + j * 16 + c;
        if (n >= a.n) continue;
        if (F32) {
#pragma unroll
            for (int i = 0; i < T::kKT; ++i) {
                const int k = k0 + wk + i * 16 + q * 4;
                if (k >= a.k) continue;
                v4f* o = reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.dw) + ((size_t)e * a.n + n) * a.k + k);
                *o = ADD ? acc[i][j] + *o : acc[i][j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < T::kKT; i += 2) {
                const int k = k0 + wk + i * 16 + q * 8;
                if (k >= a.k) continue;
                const v4f lo = acc[i][j], hi = acc[i + 1][j];
                *reinterpret_cast<v4u*>(reinterpret_cast<uint16_t*>(a.dw) + ((size_t)e * a.n + n) * a.k + k) =
                    v4u{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]),
                        pack_bf16x2(hi[2], hi[3])};
            }
        }
    }
}

template <int TN, int TK, int WN, int WK, int FMT, bool F32, bool ADD>
hipError_t launch_one(ExpertWgradArgs a, hipStream_t stream) {
    using T = WTile<TN, TK, WN, WK, wgrad_terms(FMT, F32)>;
    a.nt = (a.n + TN - 1) / TN;
    a.kt = (a.k + TK - 1) / TK;
    const long long blocks = ((long long)a.r.E * a.nt * a.kt + 255) / 256 * 256;  // whole runs of 32 on each XCD
    if (!grid_fits(blocks, T::kThreads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((moedisp_expert_wgrad<TN, TK, WN, WK, FMT, F32, ADD>), dim3((unsigned)blocks),
                       dim3(T::kThreads), T::kLds, stream, a);
    return hipGetLastError();
}

template <int FMT, bool F32, bool ADD>
hipError_t launch_tiles(const ExpertWgradArgs& a, hipStream_t stream) {
    const bool large = expert_wgrad_tile(a.r.E, a.n, a.k, FMT, F32).a == 256;
    if constexpr (wgrad_terms(FMT, F32) == 1) {
        if (large) return launch_one<256, 256, 4, 2, FMT, F32, ADD>(a, stream);
    } else {
        if (large) return launch_one<256, 128, 2, 2, FMT, F32, ADD>(a, stream);
    }
    return launch_one<128, 128, 2, 2, FMT, F32, ADD>(a, stream);
}

template <int FMT>
hipError_t launch_fmt(const ExpertWgradArgs& a, bool f32_out, bool accumulate, hipStream_t stream) {
    if (!f32_out) return launch_tiles<FMT, false, false>(a, stream);
    return accumulate ? launch_tiles<FMT, true, true>(a, stream) : launch_tiles<FMT, true, false>(a, stream);
}

}  // namespace

// Tiles of 256 x 256 move the fewest bytes per product (8 experts of 4096 x
// 4096 and 4096 rows each: 1069 us against 1459 with 128 x 128).  Tiles of 128 x
// 128 (two workgroups to a unit) where large ones, in whole rounds of one for
// each unit, cover a fifth more than small ones do: 8 experts of 512 x 512 and
// 1024 rows each 24 us against 47, 52 of 2008 x 128 26 against 33, 13 of 1048
// x 3328 42 against 51; not 35 of 3264 x 1536 (1.03 times as much), 164 against
// 179.
//
// Three terms of x leave LDS no room for 256 x 256, and for one workgroup to a
// unit at either tile: 256 x 128, which a round of takes 1.4 times as long as one
// of 128 x 128, unless the rounds are as many (fp32 results of FP32 scales, 8
// experts of 4096 x 4096 and 4096 rows each: 3.29 ms against 4.75; 24 of 1000 x 640,
// 88 rows: 43 us against 50; but 8 of 512 x 512 and 1024 rows: 65 us against 48).
TileShape expert_wgrad_tile(int E, int n, int k, int scale_fmt, bool f32_out) {
    const long long small = (long long)E * ((n + 127) / 128) * ((k + 127) / 128);
    if (wgrad_terms(scale_fmt, f32_out) > 1) {
        const long long half = (long long)E * ((n + 255) / 256) * ((k + 127) / 128);
        return (half + kCus - 1) / kCus * 7 <= (small + kCus - 1) / kCus * 5 ? TileShape{256, 128} : TileShape{128, 128};
    }
    const long long large = (long long)E * ((n + 255) / 256) * ((k + 255) / 256);
    const long long rounds = (large + kCus - 1) / kCus * kCus;
    return rounds * 4 * 5 <= small * 6 ? TileShape{256, 256} : TileShape{128, 128};
}

hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, int scale_fmt, bool f32_out, bool accumulate,
                               hipStream_t stream) {
    return scale_fmt == MOEDISP_SCALE_UE8M0 ? launch_fmt<MOEDISP_SCALE_UE8M0>(a, f32_out, accumulate, stream)
                                            : launch_fmt<MOEDISP_SCALE_FP32>(a, f32_out, accumulate, stream);
}

}  // namespace moedisp
