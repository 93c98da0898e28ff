// Product of the experts' bf16 rows with their bf16 weights:
//     NK:  y[r][n] = sum_k x[r][k] * w[e][n][k]
//     KN:  y[r][n] = sum_k x[r][k] * w[e][k][n]
// The second is the first's gradient of x from the weights as they lie.
//
// Products are exact and sums are binary32; a result is rounded once.
//
// What bounds it.  128 rows an expert (256 experts, 7168 -> 4096): the weights
// from HBM, 15.7 GB in 2.80 ms, 5.6 TB/s (loads alone 2.83 ms, products alone
// 1.42).  4096 rows (8 experts, 4096 -> 8192): 1.76 ms, 1.25 PFLOP/s; products
// alone take 1.29 ms and loads alone 1.23, which do not overlap fully.  KN at 122
// rows, skewed (256 experts, 7168 -> 2048): 1.74 ms, loads alone 1.68.
//
// How.  A workgroup computes a tile of BM rows by BN columns, 64 channels after
// 64.  Both operands go straight into LDS.  NK: 128 bytes of 8 rows per load,
// 16-byte chunks swizzled so that operand reads have no bank conflicts.  KN:
// rows of channels by columns, which the transposing reads turn.  Channels past
// the last one are zeros in both operands: lanes that would load them point
// behind their buffer descriptor.  The weights are the matrix instruction's
// rows and the tokens its columns, so that a lane's results are neighbours of
// one row of y; bf16 results' columns are dealt to the instruction so that two
// of them make 8 neighbours, one 16-byte store.  Workgroups stay and take tile
// after tile.
//
// A step's loads go out one by one between the products (all at once: 1776 us
// where 1728 were taken); the rows' as soon as the step's rows are in registers, so
// that they have nearly two steps to arrive (1910 -> 1801 us), the weights' three
// steps ahead.  Steps of 32 channels, five in LDS, took longer (2018 us): lines
// of 128 bytes are read in two halves, each at the price of one.
#include "experts_common.h"

namespace moedisp {
namespace {

constexpr int kBlk = 64;                     // channels of a step: 128 bytes
constexpr long long kLdsBytes = 160 * 1024;  // of a CU
constexpr int kOutside = (int)0x80000000u;   // an offset past every descriptor's end

template <int BM, int BN, int WM, int WN, int WS, int XS>
struct Tile {
    static constexpr int kWaves = WM * WN;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int kM = BM / WM;          // rows of a wave
    static constexpr int kN = BN / WN;          // columns of a wave
    static constexpr int kMT = kM / 16;
    static constexpr int kNT = kN / 16;
    static constexpr int kWLoads = BN / 8 / kWaves;  // 1 KiB loads of a wave and step
    static constexpr int kXLoads = (BM / 8 + kWaves - 1) / kWaves;
    // Loads of a wave and step kb, in this order: the rows of step kb + XS, as
    // soon as those of step kb are in registers; the weights of step kb + WS,
    // behind the last of step kb.  Before step kb + 1 its own have to be there;
    // younger ones may be under way.
    static constexpr int kLoads = kWLoads + kXLoads;
    static constexpr int kYounger = (XS - 1) * kXLoads + (WS - 2) * kWLoads;
    static constexpr int kXBytes = kXLoads * kWaves * 1024;
    static constexpr int kWStage = BN * 2 * kBlk;
    static constexpr int kLds = WS * kWStage + XS * kXBytes;
    static_assert(WS >= XS && XS >= 2 && WS - XS <= 1 && (WS + XS) * kLoads < 64, "stages");
    static_assert(kNT % 2 == 0 && kM % 16 == 0 && kN % 32 == 0 && BN % (8 * kWaves) == 0 && BN >= 128, "tile shape");
    static_assert(kLds <= kLdsBytes, "LDS");
};

// Both halves of a lane's 16 channels of a step: those of two products.
struct Frag {
    v8bf lo, hi;
};

template <int BM, int BN, int WM, int WN, int WS, int XS, bool KN, bool F32>
__global__ __launch_bounds__(64 * WM * WN) void moedisp_expert_gemm_bf16(ExpertBf16Args a) {
    using T = Tile<BM, BN, WM, WN, WS, XS>;
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    int incl, own;
    const int tiles = expert_tiles<BM>(a.r, &incl, &own);
    if (tiles < 0) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(&a.hdr->status, (uint32_t)MOEDISP_DEV_BAD_LAYOUT);
        return;
    }
    const int steps = (a.k + kBlk - 1) / kBlk;
    const int tail = a.k - (steps - 1) * kBlk;  // channels of the last step
    // XCD x (consecutive workgroups go round the XCDs) takes the x-th run of
    // the tiles, its workgroups every (gridDim / 8)-th of them
    const int total = tiles * a.nt;
    const int per = (total + kXcds - 1) / kXcds;
    const int end = min(total, ((int)(blockIdx.x % kXcds) + 1) * per);
    for (int item = (blockIdx.x % kXcds) * per + blockIdx.x / kXcds; item < end; item += gridDim.x / kXcds) {
        const ExpertTile t = expert_tile<BM, BN>(a.r, item, a.nt, a.n, incl, own);
        const char* const xp = reinterpret_cast<const char*>(a.x + t.row0 * a.k);
        const char* const wp = reinterpret_cast<const char*>(
            a.w + (KN ? (size_t)t.e * a.k * a.n + t.n0 : ((size_t)t.e * a.n + t.n0) * a.k));

        // offsets of the wave's loads in a step, and the same in the last one
        int woff[T::kWLoads], xoff[T::kXLoads];
        uint32_t w_out = 0, x_out = 0;  // bit i: load i lies past the last channel
#pragma unroll
        for (int i = 0; i < T::kWLoads; ++i) {
            if (KN) {
                constexpr int kRow = BN * 2;
                const int at = (wave * T::kWLoads + i) * 1024 + lane * 16;
                const int ch = at / kRow;
                const int chunk = (at % kRow / 16) ^ (unit_swizzle(ch) << 1);
                woff[i] = ch * a.n * 2 + min(chunk * 16, t.cols * 2 - 16);
                w_out |= ch >= tail ? 1u << i : 0u;
            } else {
                const int row = (wave * T::kWLoads + i) * 8 + (lane >> 3);
                const int chunk = (lane & 7) ^ (F32 ? swizzle_x(row) : swizzle_w(row));
                woff[i] = min(row, t.cols - 1) * a.k * 2 + chunk * 16;
                w_out |= chunk * 8 >= tail ? 1u << i : 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < T::kXLoads; ++i) {
            const int row = (wave * T::kXLoads + i) * 8 + (lane >> 3);
            const int chunk = (lane & 7) ^ swizzle_x(row);
            xoff[i] = min(row, t.rows - 1) * a.k * 2 + chunk * 16;
            x_out |= chunk * 8 >= tail ? 1u << i : 0u;
        }
        const int wm = wave % WM, wn = wave / WM;
        char* const x_lds = lds + WS * T::kWStage;

        // load i of step kb; steps past the last load the last one again, to no use
        auto issue_w = [&](int kb, int buf, int i) {
            const int s = min(kb, steps - 1);
            const char* const base = wp + (KN ? (size_t)s * kBlk * a.n * 2 : (size_t)s * kBlk * 2);
            const uint32_t out = s == steps - 1 ? w_out : 0u;
            load_to_lds_unseen<16>(base, lds + buf * T::kWStage + (wave * T::kWLoads + i) * 1024,
                                   out >> i & 1 ? kOutside : woff[i]);
        };
        auto issue_x = [&](int kb, int buf, int i) {
            const int s = min(kb, steps - 1);
            const char* const base = xp + (size_t)s * kBlk * 2;
            const uint32_t out = s == steps - 1 ? x_out : 0u;
            load_to_lds_unseen<16>(base, x_lds + buf * T::kXBytes + (wave * T::kXLoads + i) * 1024,
                                   out >> i & 1 ? kOutside : xoff[i]);
        };

        v4f acc[T::kNT][T::kMT];
#pragma unroll
        for (int i = 0; i < T::kNT; ++i)
#pragma unroll
            for (int j = 0; j < T::kMT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
        for (int p = 0; p < WS; ++p) {
#pragma unroll
            for (int i = 0; i < T::kXLoads; ++i)
                if (p >= WS - XS) issue_x(p - (WS - XS), p - (WS - XS), i);
#pragma unroll
            for (int i = 0; i < T::kWLoads; ++i) issue_w(p, p, i);
            __builtin_amdgcn_sched_barrier(0);
        }

        const int q = lane >> 4, c = lane & 15;
        const int xrow = wm * T::kM + c, xsw = swizzle_x(xrow);
        // columns of products 2t and 2t + 1 that a lane gets: bf16 results 8
        // neighbours, fp32 results 4 of each, 16 bytes to store either way
        const int wrow = wn * T::kN + (F32 ? c : (c >> 2) * 8 + (c & 3));
        const int wsw = F32 ? swizzle_x(wrow) : swizzle_w(wrow);
        // KN: channel 8q + c/4 (and + 4) of a half step, piece c%4 of 4 columns
        const int tr_row = q * 8 + (c >> 2), tr_sw = unit_swizzle(tr_row);
        auto read_rows = [&](const char* row, int sw) {
            const int lo_at = (q ^ sw) << 4;
            return Frag{*reinterpret_cast<const v8bf*>(row + lo_at), *reinterpret_cast<const v8bf*>(row + (lo_at ^ 64))};
        };
        auto w_at = [&](const char* st, int i) {
            if constexpr (KN) {
                constexpr int kRow = BN * 2;
                const int piece = c & 3;
                const int unit = wn * T::kN / 16 + (F32 ? i : (i & ~1) + (piece >> 1));
                const int in_unit = F32 ? piece * 8 : (piece & 1) * 16 + (i & 1) * 8;
                const char* p = st + tr_row * kRow + ((unit ^ tr_sw) << 5) + in_unit;
                auto half = [&](const char* h) {
                    const v4s lo = read_transposed(h), hi = read_transposed(h + 4 * kRow);
                    return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                };
                return Frag{half(p), half(p + 32 * kRow)};
            } else {
                return read_rows(st + (wrow + (F32 ? i * 16 : (i >> 1) * 32 + (i & 1) * 4)) * 128, wsw);
            }
        };
        auto x_at = [&](const char* st, int j) { return read_rows(st + (xrow + j * 16) * 128, xsw); };

        Frag b[T::kMT], wf[2];
        wait_loads_and_sync<(XS - 1) * T::kXLoads + (WS - 1) * T::kWLoads>();
        wf[0] = w_at(lds, 0);
#pragma unroll
        for (int j = 0; j < T::kMT; ++j) b[j] = x_at(x_lds, j);
        // Step kb: its rows' operands and the first of the weights' are in
        // registers.  Behind the first products the waves meet, as all have read
        // the rows, whose place is filled; before the last ones again, for the
        // weights; the next step's operands are read behind the last products.
        int wbuf = 0, xbuf = 0;
        for (int kb = 0; kb < steps; ++kb) {
            const char* st = lds + wbuf * T::kWStage;
            const int nwbuf = wbuf + 1 == WS ? 0 : wbuf + 1;
            const int nxbuf = xbuf + 1 == XS ? 0 : xbuf + 1;
            const char* nst = lds + nwbuf * T::kWStage;
            const char* nxt = x_lds + nxbuf * T::kXBytes;
#pragma unroll
            for (int i = 0; i < T::kNT; ++i) {
                if (i + 1 < T::kNT) wf[(i + 1) & 1] = w_at(st, i + 1);
                if (i == T::kNT - 1) {
                    wait_loads_and_sync<T::kYounger>();
                    wf[0] = w_at(nst, 0);
                }
#pragma unroll
                for (int j = 0; j < T::kMT; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i & 1].lo, b[j].lo, acc[i][j], 0, 0, 0);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i & 1].hi, b[j].hi, acc[i][j], 0, 0, 0);
                    if (i == T::kNT - 1) b[j] = x_at(nxt, j);
                    __builtin_amdgcn_sched_barrier(0);
                    // the loads one by one between the products
                    constexpr int kPlaces = (T::kNT - 2) * T::kMT;
                    if (i > 0 && i < T::kNT - 1) {
                        const int place = (i - 1) * T::kMT + j;
#pragma unroll
                        for (int l = 0; l < T::kXLoads; ++l)
                            if (l * kPlaces / T::kXLoads == place) issue_x(kb + XS, xbuf, l);
                    }
                    if (i == T::kNT - 1) {
#pragma unroll
                        for (int l = 0; l < T::kWLoads; ++l)
                            if (l * T::kMT / T::kWLoads == j) issue_w(kb + WS, wbuf, l);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (i == 0) {
                    reads_done_and_sync();
#pragma unroll
                    for (int l = 0; l < T::kXLoads; ++l)
                        if (T::kNT == 2) issue_x(kb + XS, xbuf, l);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            wbuf = nwbuf;
            xbuf = nxbuf;
        }
        // all loads into LDS have arrived and all reads are done: the next tile
        // may fill it, and none arrives after the workgroup's end
        wait_loads_and_sync<0>();

#pragma unroll
        for (int j = 0; j < T::kMT; ++j) {
            const int m = wm * T::kM + j * 16 + c;
            if (m >= t.rows) continue;
#pragma unroll
            for (int i = 0; i < T::kNT; i += F32 ? 1 : 2) {
                const int n = wn * T::kN + i * 16 + q * (F32 ? 4 : 8);
                if (n >= t.cols) continue;
                const size_t at = (t.row0 + m) * a.n + t.n0 + n;
                if (F32) {
                    *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.y) + at) = acc[i][j];
                } else {
                    const v4f lo = acc[i][j], hi = acc[i + 1][j];
                    const v4u v = {pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]),
                                   pack_bf16x2(hi[2], hi[3])};
                    *reinterpret_cast<v4u*>(reinterpret_cast<uint16_t*>(a.y) + at) = v;
                }
            }
        }
    }
}

template <int BM, int BN, int WM, int WN, int WS, int XS, bool KN, bool F32>
hipError_t launch_tile(ExpertBf16Args a, hipStream_t stream) {
    using T = Tile<BM, BN, WM, WN, WS, XS>;
    a.nt = (a.n + BN - 1) / BN;
    const long long tiles = (long long)a.r.max_rows / BM + a.r.E;  // at least the tiles of any bounds
    if (tiles * a.nt > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    long long blocks = (tiles * a.nt + kXcds - 1) / kXcds * kXcds;
    const long long resident = kCus * (kLdsBytes / T::kLds);
    if (blocks > resident) blocks = resident;
    hipLaunchKernelGGL((moedisp_expert_gemm_bf16<BM, BN, WM, WN, WS, XS, KN, F32>), dim3((unsigned)blocks),
                       dim3(T::kThreads), T::kLds, stream, a);
    return hipGetLastError();
}

template <bool KN, bool F32>
hipError_t launch_variant(const ExpertBf16Args& a, int mean_rows, hipStream_t stream) {
    const TileShape t = expert_gemm_bf16_tile(a.r.E, a.n, mean_rows);
    if (t.a == 32) return launch_tile<32, 128, 1, 4, 3, 3, KN, F32>(a, stream);
    if (t.a == 64) return launch_tile<64, 256, 2, 4, 3, 3, KN, F32>(a, stream);
    if (t.a == 96) return launch_tile<96, 256, 2, 4, 3, 2, KN, F32>(a, stream);
    if (t.a == 128) return launch_tile<128, 256, 2, 4, 3, 2, KN, F32>(a, stream);
    if (t.a == 160) return launch_tile<160, 256, 2, 4, 3, 2, KN, F32>(a, stream);
    return launch_tile<256, 256, 4, 2, 2, 2, KN, F32>(a, stream);
}

}  // namespace

// Times of a round of all compute units for 4096 channels, whose weights other
// workgroups read as well.  Experts, usual rows, K, n, us (NK):
//                              32x128  64x256  96x256  128x256  160x256  256x256
//       8,   16, 4096, 8192       110     121     122      121      123      130
//       8,   64, 4096, 8192       146     142     129      130      132      140
//      64,   62, 2048, 4096       279     229     198      199      204      249
//     256,  128, 7168, 4096      5934    3972    3529     3872     2882     3467
//      16,  250, 2048, 2000        69      60      52       57       41       48
//      30,  400, 1024, 2048       119      82      74       71       67       64
//       8, 4096, 4096, 8192      5580    3030    2389     2074     2008     1728
TileShape expert_gemm_bf16_tile(int E, int n, int mean_rows) {
    static const TileTime kinds[] = {{32, 128, 2, 44}, {64, 256, 1, 47},  {96, 256, 1, 56},
                                     {128, 256, 1, 65}, {160, 256, 1, 78}, {256, 256, 1, 112}};
    return tile_by_rounds(kinds, 6, E, n, mean_rows);
}

hipError_t launch_expert_gemm_bf16(const ExpertBf16Args& a, int mean_rows, bool kn, bool f32_out,
                                   hipStream_t stream) {
    if (kn)
        return f32_out ? launch_variant<true, true>(a, mean_rows, stream)
                       : launch_variant<true, false>(a, mean_rows, stream);
    return f32_out ? launch_variant<false, true>(a, mean_rows, stream)
                   : launch_variant<false, false>(a, mean_rows, stream);
}

}  // namespace moedisp
