// Weight gradient of the experts' bf16 product:
//     dw[e][n][k] (+)= sum over e's rows r of dy[r][n] * x[r][k]
//
// Products are exact and sums are binary32; bf16 results are rounded once.
//
// What bounds it.  Many rows (32768 over 8 experts, 4096 x 4096): 0.90 ms, 1.22
// PFLOP/s, products with the transposing reads beside them (matrix units 0.6 of
// the time).  Few rows (7782 over 64, 7168 x 2048, fp32): the writes, 3.8 GB in
// 0.86 ms, 4.4 TB/s (7176 x 1992, tiles cut at both edges: 0.92 ms).  An expert's
// rows are not split.
//
// How.  A workgroup computes one tile over all rows of its expert, 32 rows a
// step, two or three steps of loads under way.  Both operands are contracted over
// rows, which is across the way they lie: they go straight into LDS by rows
// and the transposing reads of the matrix operands turn them.  Rows past the
// expert's last are zeros in both (their loads lie past the descriptor's end).
#include "experts_common.h"

namespace moedisp {
namespace {

constexpr int kStep = 32;   // rows per step: the contraction of one matrix instruction

// Tile of TN columns of dy by TK channels of x; WN x WK waves; NS steps under
// way or in use.
template <int TN, int TK, int WN, int WK, int NS>
struct WTile {
    static constexpr int kStages = NS;
    static constexpr int kWaves = WN * WK;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int kNT = TN / WN / 16;  // 16-wide tiles of a wave
    static constexpr int kKT = TK / WK / 16;
    static constexpr int kDyRow = TN * 2;     // bytes
    static constexpr int kXRow = TK * 2;
    static constexpr int kDyStage = kStep * kDyRow;
    static constexpr int kXStage = kStep * kXRow;
    static constexpr int kDyLoads = kDyStage / 1024 / kWaves;  // of a wave and step
    static constexpr int kXLoads = kXStage / 1024 / kWaves;
    static constexpr int kOps = kDyLoads + kXLoads;
    static constexpr int kLds = kStages * (kDyStage + kXStage);
    static_assert(kKT >= 4 && kKT % 2 == 0 && kDyRow >= 256 && kXRow >= 256 && kDyLoads > 0 && kXLoads > 0,
                  "tile shape");
};

template <int TN, int TK, int WN, int WK, int NS, bool F32, bool ADD>
__global__ __launch_bounds__(64 * WN * WK) void moedisp_expert_wgrad_bf16(ExpertBf16Args a) {
    using T = WTile<TN, TK, WN, WK, NS>;
    constexpr int kStages = NS;
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

    // load i of the wave brings 1 KiB: whole rows, or two parts of one
    int dy_off[T::kDyLoads], x_off[T::kXLoads];
#pragma unroll
    for (int i = 0; i < T::kDyLoads; ++i) {
        const int at = (wave * T::kDyLoads + i) * 1024 + lane * 16;
        const int row = at / T::kDyRow;
        const int chunk = (at % T::kDyRow / 16) ^ (unit_swizzle(row) << 1);
        dy_off[i] = row * a.n * 2 + min(chunk * 16, (a.n - n0) * 2 - 16);
    }
#pragma unroll
    for (int i = 0; i < T::kXLoads; ++i) {
        const int at = (wave * T::kXLoads + i) * 1024 + lane * 16;
        const int row = at / T::kXRow;
        const int chunk = (at % T::kXRow / 16) ^ (unit_swizzle(row) << 1);
        x_off[i] = row * a.k * 2 + min(chunk * 16, (a.k - k0) * 2 - 16);
    }
    char* const x_lds = lds + kStages * T::kDyStage;
    auto load_dy = [&](int step, int buf) {
        const int r0 = min(step * kStep, rows);
        const int left = min(rows - r0, kStep);
        const uint16_t* base = a.dy + ((size_t)first + r0) * a.n + n0;
#pragma unroll
        for (int i = 0; i < T::kDyLoads; ++i)
            load_to_lds_unseen<16>(base, lds + buf * T::kDyStage + (wave * T::kDyLoads + i) * 1024, dy_off[i],
                                   max(left * a.n - n0, 0) * 2);
    };
    auto load_x = [&](int step, int buf) {
        const int r0 = min(step * kStep, rows);
        const int left = min(rows - r0, kStep);
        const uint16_t* base = a.x + ((size_t)first + r0) * a.k + k0;
#pragma unroll
        for (int i = 0; i < T::kXLoads; ++i)
            load_to_lds_unseen<16>(base, x_lds + buf * T::kXStage + (wave * T::kXLoads + i) * 1024, x_off[i],
                                   max(left * a.k - k0, 0) * 2);
    };

    const int wk = wave % WK * (TK / WK), wn = wave / WK * (TN / WN);
    v4f acc[T::kKT][T::kNT];
#pragma unroll
    for (int i = 0; i < T::kKT; ++i)
#pragma unroll
        for (int j = 0; j < T::kNT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int q = lane >> 4, c = lane & 15;
    // the lane's place in the transposing reads: row 8q + c/4 (and + 4), piece
    // c%4 of 4 columns
    const int tr_row = q * 8 + (c >> 2);
    const int tr_sw = unit_swizzle(tr_row);  // the same 4 rows below
    const int piece = c & 3;
    auto turned = [&](const char* p, int row_bytes) {
        const v4s lo = read_transposed(p);
        const v4s hi = read_transposed(p + 4 * row_bytes);
        return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto dy_at = [&](const char* st, int j) {
        return turned(st + tr_row * T::kDyRow + (((wn / 16 + j) ^ tr_sw) << 5) + piece * 8, T::kDyRow);
    };
    // bf16 results: products 2p and 2p + 1 take the channels 0-3, 8-11, 16-19,
    // 24-27 of 32 and the others, so that they give a lane 8 neighbours, 16
    // bytes to store
    auto x_at = [&](const char* st, int i) {
        const int unit = wk / 16 + (F32 ? i : (i & ~1) + (piece >> 1));
        const int in_unit = F32 ? piece * 8 : (piece & 1) * 16 + (i & 1) * 8;
        return turned(st + tr_row * T::kXRow + ((unit ^ tr_sw) << 5) + in_unit, T::kXRow);
    };

    if (steps > 0) {
#pragma unroll
        for (int p = 0; p < kStages - 1; ++p) {
            load_x(p, p);
            load_dy(p, p);
        }
        wait_loads_and_sync<(kStages - 2) * T::kOps>();
        int buf = 0;
        for (int s = 0; s < steps; ++s) {
            const char* ds = lds + buf * T::kDyStage;
            const char* xs = x_lds + buf * T::kXStage;
            v8bf b[T::kNT], av[2];
#pragma unroll
            for (int j = 0; j < T::kNT; ++j) b[j] = dy_at(ds, j);
            av[0] = x_at(xs, 0);
            const int next = (buf + kStages - 1) % kStages;
#pragma unroll
            for (int i = 0; i < T::kKT; ++i) {
                if (i + 1 < T::kKT) av[(i + 1) & 1] = x_at(xs, i + 1);
#pragma unroll
                for (int j = 0; j < T::kNT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[i & 1], b[j], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                // behind the products: step s + kStages - 1 into the place of
                // step s - 1, which all waves have read
                if (i == 0) load_x(s + kStages - 1, next);
                if (i == 1) load_dy(s + kStages - 1, next);
                if (i < 2) __builtin_amdgcn_sched_barrier(0);
            }
            wait_loads_and_sync<(kStages - 2) * T::kOps>();
            buf = (buf + 1) % kStages;
        }
        wait_loads_and_sync<0>();  // no load may reach LDS after the workgroup's end
    }

    // Results by way of LDS, a wave's 16 columns at a time in a place of its
    // own, so that rows of dw are written in runs of a wave's channels (64 experts
    // of 7176 x 1992, fp32: 984 -> 927 us).
    constexpr int kEl = F32 ? 4 : 2;
    constexpr int kRunBytes = TK / WK * kEl;   // bytes
    constexpr int kPitch = kRunBytes + 16;     // rows of 16 lanes start at different banks
    constexpr int kLanes = kRunBytes / 16;  // lanes of a run
    constexpr int kRows = 64 / kLanes;      // runs of a store
    constexpr int kStores = 16 / kRows;
    static_assert(16 * kPitch * T::kWaves <= T::kLds && 64 % kLanes == 0, "results fit LDS");
    char* const mine = lds + wave * (16 * kPitch);
#pragma unroll
    for (int j = 0; j < T::kNT; ++j) {
#pragma unroll
        for (int i = 0; i < T::kKT; i += F32 ? 1 : 2) {
            char* const to = mine + c * kPitch + (i * 16 + q * (F32 ? 4 : 8)) * kEl;
            if (F32) {
                *reinterpret_cast<v4f*>(to) = acc[i][j];
            } else {
                const v4f lo = acc[i][j], hi = acc[i + 1][j];
                *reinterpret_cast<v4u*>(to) = v4u{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                                                  pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])};
            }
        }
        own_lds_done();
        v4u v[kStores];
#pragma unroll
        for (int r = 0; r < kStores; ++r)
            v[r] = *reinterpret_cast<const v4u*>(mine + (r * kRows + lane / kLanes) * kPitch + lane % kLanes * 16);
        const int k = k0 + wk + lane % kLanes * (16 / kEl);
#pragma unroll
        for (int r = 0; r < kStores; ++r) {
            const int n = n0 + wn + j * 16 + r * kRows + lane / kLanes;
            if (n >= a.n || k >= a.k) continue;
            v4u* const o = reinterpret_cast<v4u*>(static_cast<char*>(a.y) + (((size_t)e * a.n + n) * a.k + k) * kEl);
            if (ADD) v[r] = __builtin_bit_cast(v4u, __builtin_bit_cast(v4f, v[r]) + __builtin_bit_cast(v4f, *o));
            *o = v[r];
        }
        own_lds_done();
    }
}

template <int TN, int TK, int WN, int WK, int NS, bool F32, bool ADD>
hipError_t launch_one(ExpertBf16Args a, hipStream_t stream) {
    using T = WTile<TN, TK, WN, WK, NS>;
    a.nt = (a.n + TN - 1) / TN;
    a.kt = (a.k + TK - 1) / TK;
    const long long blocks = ((long long)a.r.E * a.nt * a.kt + 255) / 256 * 256;  // whole runs of 32 on each XCD
    if (!grid_fits(blocks, T::kThreads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((moedisp_expert_wgrad_bf16<TN, TK, WN, WK, NS, F32, ADD>), dim3((unsigned)blocks),
                       dim3(T::kThreads), T::kLds, stream, a);
    return hipGetLastError();
}

template <bool F32, bool ADD>
hipError_t launch_tiles(const ExpertBf16Args& a, hipStream_t stream) {
    if (expert_wgrad_bf16_tile(a.r.E, a.n, a.k).a == 256) return launch_one<256, 256, 4, 2, 4, F32, ADD>(a, stream);
    return launch_one<128, 128, 2, 2, 3, F32, ADD>(a, stream);
}

}  // namespace

// Tiles of 256 x 256 move the fewest bytes per product (8 experts of 4096 x
// 4096 and 4096 rows each: 869 us against 1054 with 128 x 128; 64 of 7168 x
// 2048 and 122 rows, fp32: 858 against 975).  Tiles of 128 x
// 128, three workgroups to a unit, where large ones, in whole rounds of one for
// each unit, cover a fifth more than small ones do.
TileShape expert_wgrad_bf16_tile(int E, int n, int k) {
    const long long small = (long long)E * ((n + 127) / 128) * ((k + 127) / 128);
    const long long large = (long long)E * ((n + 255) / 256) * ((k + 255) / 256);
    const long long rounds = (large + kCus - 1) / kCus * kCus;
    return rounds * 4 * 5 <= small * 6 ? TileShape{256, 256} : TileShape{128, 128};
}

hipError_t launch_expert_wgrad_bf16(const ExpertBf16Args& a, bool f32_out, bool accumulate, hipStream_t stream) {
    if (!f32_out) return launch_tiles<false, false>(a, stream);
    return accumulate ? launch_tiles<true, true>(a, stream) : launch_tiles<true, false>(a, stream);
}

}  // namespace moedisp
