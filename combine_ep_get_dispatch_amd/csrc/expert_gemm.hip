// Product of the experts' rows with their weights, both E4M3 with a scale per
// block of 128 channels:
//     y[r][n] = sum_b sx[r][b] * sw[e][n/128][b] * (x[r][128b..] . w[e][n][128b..])
//
// Precision.  A block's dot product is one E4M3 matrix instruction (16 x 16 x
// 128).  It drops what lies 16 bits below the largest products that it adds:
// 1.4e-5 of a result of normal rows, whatever the instruction's shape and
// whether blocks are chained or added apart.  bf16 results (rounded by 2^-8)
// take it; fp32 results widen the codes to bf16, whose products and sums are
// good to binary32, at half the matrix rate.  Block sums are scaled and added
// in binary32 (UE8M0 scales of bf16 results: inside the instruction).
//
// What bounds it.  Few rows: the weights from HBM (decode, 128 tokens top-8 of
// 256 experts, 7168 -> 4096: 7.4 GB in 1.20 ms, 6.2 TB/s).  128 rows an expert
// (prefill): the same bytes, 1.64 ms, 4.9 TB/s and 1.2 PFLOP/s.  4096 rows
// (16384 tokens top-2 of 8, 4096 -> 8192): 1.08 ms, 2.0 PFLOP/s; the products
// alone would take 0.85 ms and the loads alone 0.97 ms: one block's loads, 64
// KiB per compute unit, take 2 us to arrive (why so long is not known) and there
// is LDS for two.
//
// How.  A workgroup computes a tile of BM rows by BN columns, block of 128
// channels after block.  Rows and weights go straight into LDS, 128 bytes of 8
// rows per load; swizzled 16-byte chunks keep the operand reads free of bank
// conflicts (weights that go to registers in operand order cost 4 times the
// load time: 16 rows by 64 bytes do not coalesce).  The weights are the matrix
// instruction's rows, the tokens its columns: a lane's four results then
// belong to one token, whose scale is one factor.  bf16 results' columns are dealt
// to the instruction so that two of them make 8 neighbours, one 16-byte store.
// Workgroups stay and take tile after tile; which expert a tile belongs to
// comes from one scan over the experts' rows, so the host needs no counts.
#include "experts_common.h"

namespace moedisp {
namespace {

constexpr int kBlk = kScaleBlock;
constexpr int kChunk = 8;  // scale blocks of a row loaded at a time
constexpr long long kLdsBytes = 160 * 1024;  // of a CU

// 32 bytes of an operand row: 16-byte chunks q and q + 4 of the row's 8,
// stored at chunk ^ swizzle.
__device__ inline v8i read_frag(const char* row, int sw, int q) {
    const int lo_at = (q ^ sw) << 4;
    const v4i lo = *reinterpret_cast<const v4i*>(row + lo_at);
    const v4i hi = *reinterpret_cast<const v4i*>(row + (lo_at ^ 64));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// 8 E4M3 codes (dwords 2j, 2j+1 of a fragment) as bf16, exactly.
__device__ inline v8bf widen(const v8i& f, int j) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * j], 1.0f, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * j], 1.0f, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * j + 1], 1.0f, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * j + 1], 1.0f, true);
    return v8bf{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// A scale's value from its stored bits (a UE8M0 byte in a dword).
template <int FMT>
__device__ inline float scale_value(int bits) {
    return FMT == MOEDISP_SCALE_FP32 ? __int_as_float(bits) : ue8m0_value((uint32_t)bits);
}

template <int BM, int BN, int WM, int WN, int WS, int XS, int FMT, bool F32>
struct Tile {
    static constexpr int kWaves = WM * WN;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int kM = BM / WM;          // rows of a wave
    static constexpr int kN = BN / WN;          // columns of a wave
    static constexpr int kMT = kM / 16;
    static constexpr int kNT = kN / 16;
    static constexpr int kWLoads = BN / 8 / kWaves;  // 1 KiB loads of a wave and stage
    static constexpr int kXLoads = (BM / 8 + kWaves - 1) / kWaves;
    // Loads of a wave and block, in this order: the rows of block kb + XS, one
    // load of scales, the weights of block kb + WS.  Before block kb + 1 its
    // rows have to be there, and all that is older; what is younger may be
    // under way.
    static constexpr int kLoads = kWLoads + kXLoads + 1;
    static constexpr int kYounger = (WS > XS ? 1 + kWLoads : 0) + (XS - 2) * kLoads;
    static constexpr int kXBytes = kXLoads * kWaves * 1024;
    static constexpr int kWStage = BN * kBlk;
    static constexpr int kStages = WS * kWStage + XS * kXBytes;
    // scales of the rows: chunks of kChunk blocks, two in LDS, [row][block]
    static constexpr int kSGroups = BM / 8;                             // loads of 8 rows by kChunk blocks
    static constexpr int kSTurns = (kSGroups + kWaves - 1) / kWaves;    // blocks in which a chunk is loaded
    static constexpr int kSBytes = 2 * BM * kChunk * 4 + kWaves * 256;  // and what the other blocks load
    static_assert(kSTurns + XS <= kChunk, "a chunk is there before it is read");
    static_assert(WS >= XS && XS >= 2, "stages");
    static constexpr int kSwBlocks = BN >= kBlk ? BN / kBlk : 1;
    static_assert(kNT % 2 == 0 && kM % 16 == 0 && kN % 32 == 0 && kN <= kBlk && BN % (8 * kWaves) == 0, "tile shape");
    static constexpr size_t lds(int kb) { return (size_t)kStages + kSBytes + (size_t)kSwBlocks * kb * 4; }
};

template <int BM, int BN, int WM, int WN, int WS, int XS, int FMT, bool F32>
__global__ __launch_bounds__(64 * WM * WN) void moedisp_expert_gemm(ExpertGemmArgs a) {
    using T = Tile<BM, BN, WM, WN, WS, XS, FMT, F32>;
    constexpr int SB = FMT == MOEDISP_SCALE_FP32 ? 4 : 1;
    extern __shared__ char lds[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    int incl, own;
    const int tiles = expert_tiles<BM>(a.r, &incl, &own);
    if (tiles < 0) {
        if (blockIdx.x == 0 && tid == 0) atomicOr(&a.hdr->status, (uint32_t)MOEDISP_DEV_BAD_LAYOUT);
        return;
    }
    // XCD x (consecutive workgroups go round the XCDs) takes the x-th run of
    // the tiles, its workgroups every (gridDim / 8)-th of them
    const int total = tiles * a.nt;
    const int per = (total + kXcds - 1) / kXcds;
    const int end = min(total, ((int)(blockIdx.x % kXcds) + 1) * per);
    for (int item = (blockIdx.x % kXcds) * per + blockIdx.x / kXcds; item < end; item += gridDim.x / kXcds) {
        const ExpertSpan s = expert_of_tile<BM>(a.r, item / a.nt, incl, own);
        // an expert's tiles: groups of kGroup row tiles, columns, row tiles
        constexpr int kGroup = 8;
        const int mt = (s.count + BM - 1) / BM;
        const int j0 = item - s.tiles_before * a.nt;
        const int g = j0 / (kGroup * a.nt);
        const int gm = min(kGroup, mt - g * kGroup);
        const int jr = j0 - g * kGroup * a.nt;
        const int ni = jr / gm;
        const int n0 = ni * BN;
        const int m0 = (g * kGroup + jr - ni * gm) * BM;
        const int rows = min(BM, s.count - m0);
        const int cols = min(BN, a.n - n0);

        const size_t row0 = (size_t)s.first + m0;
        const uint8_t* wp = a.w + ((size_t)s.e * a.n + n0) * a.k;
        const uint8_t* xp = a.x + row0 * a.k;
        const auto wrs = buffer_of(wp), xrs = buffer_of(xp);
        const auto srs = buffer_of((const char*)a.x_scales + row0 * a.kb * SB);

        int woff[T::kWLoads], xoff[T::kXLoads];
#pragma unroll
        for (int i = 0; i < T::kWLoads; ++i) {
            const int row = (wave * T::kWLoads + i) * 8 + (lane >> 3);
            woff[i] = min(row, cols - 1) * a.k + (((lane & 7) ^ (F32 ? swizzle_x(row) : swizzle_w(row))) << 4);
        }
#pragma unroll
        for (int i = 0; i < T::kXLoads; ++i) {
            const int row = (wave * T::kXLoads + i) * 8 + (lane >> 3);
            xoff[i] = min(row, rows - 1) * a.k + (((lane & 7) ^ swizzle_x(row)) << 4);
        }
        const int wm = wave % WM, wn = wave / WM;
        char* const x_lds = lds + WS * T::kWStage;
        char* const sx_lds = lds + T::kStages;
        // Scales of 8 rows (group g of the tile) and the 8 blocks of chunk ch: 32
        // bytes of each row at a time, as one scale of 64 rows costs a request
        // per lane.
        auto issue_scales = [&](int g, int ch, char* to) {
            const int at = min(g * 8 + (lane >> 3), rows - 1) * a.kb + min(ch * kChunk + (lane & 7), a.kb - 1);
            load_to_lds<SB>(srs, to, at * SB, 0);
        };

        auto issue_w = [&](int kb, int buf) {
#pragma unroll
            for (int i = 0; i < T::kWLoads; ++i)
                load_to_lds<16>(wrs, lds + buf * T::kWStage + (wave * T::kWLoads + i) * 1024, woff[i],
                                min(kb, a.kb - 1) * kBlk);
        };
        auto issue_x = [&](int kb, int buf) {
#pragma unroll
            for (int i = 0; i < T::kXLoads; ++i)
                load_to_lds<16>(xrs, x_lds + buf * T::kXBytes + (wave * T::kXLoads + i) * 1024, xoff[i],
                                min(kb, a.kb - 1) * kBlk);
        };
        char* const unused = sx_lds + 2 * BM * kChunk * 4 + wave * 256;

        // the weights' scales of the tile, all of k
        int* sw = reinterpret_cast<int*>(sx_lds + T::kSBytes);
        for (int i = tid; i < T::kSwBlocks * a.kb; i += T::kThreads) {
            const int b = i / a.kb;
            const size_t at = ((size_t)s.e * a.nb + min(n0 / kBlk + b, a.nb - 1)) * a.kb + (i - b * a.kb);
            sw[i] = FMT == MOEDISP_SCALE_FP32 ? reinterpret_cast<const int*>(a.w_scales)[at]
                                              : (int)reinterpret_cast<const uint8_t*>(a.w_scales)[at];
        }
        const int* swp = sw + (T::kSwBlocks > 1 ? (wn * T::kN / kBlk) * a.kb : 0);

        v4f acc[T::kNT][T::kMT];
#pragma unroll
        for (int i = 0; i < T::kNT; ++i)
#pragma unroll
            for (int j = 0; j < T::kMT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
        for (int t = 0; t < T::kSTurns; ++t)
            if (t * T::kWaves + wave < T::kSGroups)
                issue_scales(t * T::kWaves + wave, 0, sx_lds + (t * T::kWaves + wave) * 256);
#pragma unroll
        for (int p = 0; p < WS; ++p) {
            if (p >= WS - XS) {
                issue_x(p - (WS - XS), p - (WS - XS));
                issue_scales(0, 0, unused);  // as many loads as a later block has
            }
            issue_w(p, p);
            __builtin_amdgcn_sched_barrier(0);
        }

        const int q = lane >> 4, c = lane & 15;
        // columns of products 2t and 2t + 1 that a lane gets: bf16 results 8
        // neighbours, fp32 results 4 of each, 16 bytes to store either way
        const int wrow = wn * T::kN + (F32 ? c : (c >> 2) * 8 + (c & 3));
        const int xrow = wm * T::kM + c;
        const int wsw = F32 ? swizzle_x(wrow) : swizzle_w(wrow), xsw = swizzle_x(xrow);
        // scale of the block's partial sums; the power-of-two scales of bf16
        // results go into the matrix instruction
        constexpr bool PROMOTE = FMT == MOEDISP_SCALE_FP32 || F32;
        v8i b[T::kMT], wf[2];
        int sxv[T::kMT];
        auto w_at = [&](const char* st, int i) {
            return read_frag(st + (wrow + (F32 ? i * 16 : (i >> 1) * 32 + (i & 1) * 4)) * kBlk, wsw, q);
        };
        auto x_at = [&](const char* st, int kb, int j) {
            sxv[j] = reinterpret_cast<const int*>(
                sx_lds)[(((kb / kChunk) & 1) * BM + wm * T::kM + j * 16 + c) * kChunk + kb % kChunk];
            return read_frag(st + (xrow + j * 16) * kBlk, xsw, q);
        };
        wait_loads_and_sync<T::kYounger + T::kLoads>();
        wf[0] = w_at(lds, 0);
#pragma unroll
        for (int j = 0; j < T::kMT; ++j) b[j] = x_at(x_lds, 0, j);
        // Block kb: its rows' operands and the first of the weights' are in
        // registers.  Product u = (i, j) is followed by the scaled add of the
        // product LAG before it, so that the matrix unit need not finish one
        // first; sched_barrier keeps this order.  Before the last i the block's
        // LDS has been read: the waves meet, its place is filled with the block
        // stages later, and the next block's operands are read behind the last
        // products.
        int wbuf = 0, xbuf = 0;
        for (int kb = 0; kb < a.kb; ++kb) {
            const char* st = lds + wbuf * T::kWStage;
            const int nwbuf = wbuf + 1 == WS ? 0 : wbuf + 1;
            const int nxbuf = xbuf + 1 == XS ? 0 : xbuf + 1;
            const char* nst = lds + nwbuf * T::kWStage;
            const char* nxt = x_lds + nxbuf * T::kXBytes;
            const int swv = swp[kb];
            float f[T::kMT];
            if (PROMOTE) {
#pragma unroll
                for (int j = 0; j < T::kMT; ++j) f[j] = scale_value<FMT>(sxv[j]) * scale_value<FMT>(swv);
            }
            constexpr int LAG = 2;
            constexpr int U = T::kNT * T::kMT;
            v4f p[LAG + 1];
#pragma unroll
            for (int u = 0; u < U + LAG; ++u) {
                const int i = u / T::kMT, j = u % T::kMT;
                if (u < U) {
                    if (j == 0 && i + 1 < T::kNT) wf[(i + 1) & 1] = w_at(st, i + 1);
                    if (u == U - T::kMT) {
                        wait_loads_and_sync<T::kYounger>();
                        issue_x(kb + XS, xbuf);
                        // the next chunk of the rows' scales, in the first blocks
                        // of this one; later blocks load to a place of no use, so
                        // that every block has as many loads to wait for
                        const int g = kb % kChunk * T::kWaves + wave;
                        char* const next = sx_lds + (kb / kChunk + 1) % 2 * BM * kChunk * 4;
                        issue_scales(min(g, T::kSGroups - 1), kb / kChunk + 1,
                                     g < T::kSGroups ? next + g * 256 : unused);
                        issue_w(kb + WS, wbuf);
                        __builtin_amdgcn_sched_barrier(0);
                        wf[0] = w_at(nst, 0);
                    }
                    if (!PROMOTE) {
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[i & 1], b[j], acc[i][j], 0, 0,
                                                                                     0, swv, 0, sxv[j]);
                    } else if (F32) {
                        v4f r = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int h = 0; h < 4; ++h)
                            r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(wf[i & 1], h), widen(b[j], h), r, 0,
                                                                        0, 0);
                        p[u % (LAG + 1)] = r;
                    } else {
                        p[u % (LAG + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wf[i & 1], b[j], v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
                    }
                    if (u >= U - T::kMT) b[j] = x_at(nxt, kb + 1, j);
                }
                if (PROMOTE && u >= LAG) {
                    const int io = (u - LAG) / T::kMT, jo = (u - LAG) % T::kMT;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[io][jo][v] = __builtin_fmaf(p[(u - LAG) % (LAG + 1)][v], f[jo], acc[io][jo][v]);
                }
                __builtin_amdgcn_sched_barrier(0);
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
            if (m >= rows) continue;
#pragma unroll
            for (int t = 0; t < T::kNT; t += F32 ? 1 : 2) {
                const int n = wn * T::kN + t * 16 + q * (F32 ? 4 : 8);
                if (n >= cols) continue;
                const size_t at = (row0 + m) * a.n + n0 + n;
                if (F32) {
                    *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.y) + at) = acc[t][j];
                } else {
                    const v4f lo = acc[t][j], hi = acc[t + 1][j];
                    const v4u v = {pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]),
                                   pack_bf16x2(hi[2], hi[3])};
                    *reinterpret_cast<v4u*>(reinterpret_cast<uint16_t*>(a.y) + at) = v;
                }
            }
        }
    }
}

template <int BM, int BN, int WM, int WN, int WS, int XS, int FMT, bool F32>
hipError_t launch_tile(ExpertGemmArgs a, hipStream_t stream) {
    using T = Tile<BM, BN, WM, WN, WS, XS, FMT, F32>;
    a.nt = (a.n + BN - 1) / BN;
    const long long tiles = (long long)a.r.max_rows / BM + a.r.E;  // at least the tiles of any bounds
    if (tiles * a.nt > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    static_assert(T::lds(512) <= kLdsBytes, "65536 channels");
    const size_t lds = T::lds(a.kb);
    long long blocks = (tiles * a.nt + kXcds - 1) / kXcds * kXcds;
    const long long resident = kCus * (kLdsBytes / (long long)lds);
    if (blocks > resident) blocks = resident;
    hipLaunchKernelGGL((moedisp_expert_gemm<BM, BN, WM, WN, WS, XS, FMT, F32>), dim3((unsigned)blocks),
                       dim3(T::kThreads), lds, stream, a);
    return hipGetLastError();
}

template <int FMT, bool F32>
hipError_t launch_variant(const ExpertGemmArgs& a, int mean_rows, hipStream_t stream) {
    const TileShape t = expert_gemm_tile(a.r.E, a.n, mean_rows, F32);
    if (t.a == 32) return launch_tile<32, 128, 1, 4, 3, 3, FMT, F32>(a, stream);
    if (t.a == 64) return launch_tile<64, 256, 2, 4, 3, 3, FMT, F32>(a, stream);
    if (t.a == 96) return launch_tile<96, 256, 2, 4, 3, 2, FMT, F32>(a, stream);
    if constexpr (!F32) {  // larger tiles' widened operands leave the registers
        if (t.a == 160) return launch_tile<160, 256, 2, 4, 3, 2, FMT, F32>(a, stream);
        if (t.a == 256) return launch_tile<256, 256, 4, 2, 2, 2, FMT, F32>(a, stream);
    }
    return launch_tile<128, 256, 2, 4, 3, 2, FMT, F32>(a, stream);
}

}  // namespace

// Tile by the rows an expert usually has.  Every weight is read once per row
// tile, so the tile holds the rows of a usual expert with some to spare, and
// is no higher: the rows' loads take LDS from the weights' that come from HBM
// (three blocks of weights and two of rows lie there).  Many rows: the tile
// whose loads per product are fewest.  64 experts, K = N = 4096, us (fp32
// scales, uniform routing):
//     rows     32x128  64x256  96x256  128x256  160x256  256x256
//       8       178      178     184     195      226      278
//      24       199      185     187     196      226      275
//      48       252      218     192     198      225      277
//      96       362      249     255     217      239      285
//     128        -       304     331     282      247      291
//     192        -       393     377     371      464      299
// Where the whole product is few tiles, small ones spread it over the device:
// the smallest while they are resident at once (two to a unit), those of 64 x
// 256 for as much again if experts fill more than half of them (33 experts of
// 64 rows, K = 4096, N = 1656, fp32 results: 45 us against 59 with 32 x 128; 24
// of 125 rows, K = 640, N = 1000, fp32 results: 14 us against 14.6, and 18.8
// with 128 x 256).  Many rows, but tiles of 256 x 256 in whole rounds
// of one for each unit cover half as much again as those of 128 x 256 do: those
// (12 experts of 206 rows, K = 2816, N = 2216: 30 us against 40; 15 of 784 rows,
// K = 1408, N = 1200: 33 against 47; not 9 of 335 rows, K = 3584, N = 3536, with
// 1.35 times as much: 61 against 52).
TileShape expert_gemm_tile(int E, int n, int mean_rows, bool f32_out) {
    const long long small = (long long)E * (((long long)mean_rows + 31) / 32) * ((n + 127) / 128);
    if (mean_rows <= 16 || small <= 2 * kCus || (mean_rows <= 32 && small <= 4 * kCus)) return {32, 128};
    if (mean_rows <= 32 || small <= 4 * kCus) return {64, 256};
    if (mean_rows <= 72) return {96, 256};
    if (f32_out || mean_rows <= 112) return {128, 256};
    if (mean_rows <= 144) return {160, 256};
    const long long nt = (n + 255) / 256;
    const long long large = E * (((long long)mean_rows + 255) / 256) * nt;
    const long long half = E * (((long long)mean_rows + 127) / 128) * nt;
    const long long rounds = (large + kCus - 1) / kCus * kCus;
    if (rounds * 4 > half * 3) return {128, 256};
    return {256, 256};
}

hipError_t launch_expert_gemm(const ExpertGemmArgs& a, int mean_rows, int scale_fmt, bool f32_out,
                              hipStream_t stream) {
    if (scale_fmt == MOEDISP_SCALE_UE8M0)
        return f32_out ? launch_variant<MOEDISP_SCALE_UE8M0, true>(a, mean_rows, stream)
                       : launch_variant<MOEDISP_SCALE_UE8M0, false>(a, mean_rows, stream);
    return f32_out ? launch_variant<MOEDISP_SCALE_FP32, true>(a, mean_rows, stream)
                   : launch_variant<MOEDISP_SCALE_FP32, false>(a, mean_rows, stream);
}

}  // namespace moedisp
