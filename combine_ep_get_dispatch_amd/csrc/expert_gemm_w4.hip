// Product of the experts' bf16 rows with weights of 4 bits and a scale per
// group of channels:
//     y[r][n] = sum_k x[r][k] * s[e][k/g][n] * c[e][n][k]
// c an E2M1 number with a power-of-two scale per 32 channels, or an integer of
// -8 .. 7 with a bf16 scale per 128.
//
// Precision.  E2M1: a weight times its scale is a bf16 number, made by the
// conversion instruction; products are exact and sums binary32.  Integers:
// codes 0 .. 15 become bf16 numbers, whose products with x are exact; a group's
// sum starts at -8 times that of x, from matrix instructions with constant
// weights; the scale comes last, in binary32.  A group's 256 terms have
// magnitudes (q + 8) |x| <= 23 |x|, whatever the size of the weights: its sum is
// off by at most 516 u of theirs (u = 2^-24), and weights of zero may leave that
// instead of zero.
//
// What bounds it.  Few rows: the codes from HBM (128 tokens top-8 of 256
// experts, 7168 -> 4096, E2M1: 3.9 GB in 0.67 ms, 5.9 TB/s; one token, 125 MB in
// 26 us, of which 5 are the launch, the search for the experts and the first
// loads).  Many rows: the conversions, done again for each wave that shares the
// weights, beside the products (8 experts of 1024 rows, 4096 -> 8192: 0.47 ms,
// 1.17 PFLOP/s; integers, with a fifth more products and the scaled sums, 0.61).
//
// How.  A workgroup computes a tile of BM rows by BN columns, KS channels a
// stage; codes, rows and scales go straight into LDS.  A lane of the matrix
// operand of the weights reads 16 bytes, 32 channels of one column, for four
// products: product d takes the dword d of all four lanes of a column, so that
// its channels are 32 (lane / 16) + 8 d .. + 7, and the rows' operands are read
// to match.  A lane's 32 channels are one group of E2M1 weights, the four
// lanes' 128 one of the integers.
#include "experts_common.h"

namespace moedisp {
namespace {

constexpr long long kLdsBytes = 160 * 1024;  // of a CU
constexpr int kOutside = (int)0x80000000u;   // an offset past every descriptor's end

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

template <int BM, int BN, int WM, int WN, int KS, int WS, int FMT>
struct Tile {
    static constexpr bool kE2m1 = FMT == MOEDISP_W4_E2M1;
    static constexpr int kWaves = WM * WN;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int kM = BM / WM;
    static constexpr int kN = BN / WN;
    static constexpr int kMT = kM / 16;
    static constexpr int kNT = kN / 16;
    static constexpr int kH = KS / 128;            // runs of 128 channels in a stage
    static constexpr int kWRow = KS / 2;           // bytes
    static constexpr int kXRow = KS * 2;
    static constexpr int kWLoads = BN * kWRow / 1024 / kWaves;
    static constexpr int kXLoads = (BM * kXRow + 1024 * kWaves - 1) / 1024 / kWaves;
    static constexpr int kLoads = kWLoads + kXLoads + 1;  // and one of scales
    static constexpr int kWStage = BN * kWRow;
    static constexpr int kXStage = kXLoads * kWaves * 1024;
    static constexpr int kStage = kWStage + kXStage + kWaves * 256;
    static constexpr int kLds = WS * kStage;
    // scales: a wave's own columns, 4 bytes a lane
    static constexpr int kSBytes = kE2m1 ? 1 : 2;
    static constexpr int kSGroups = KS / (kE2m1 ? 32 : 128);  // rows of scales in a stage
    static constexpr int kSLanes = kN * kSBytes / 4;          // lanes of such a row
    static_assert(kSGroups * kSLanes <= 64, "one load of scales");
    static_assert(kNT % 2 == 0 && kM % 16 == 0 && kWLoads > 0 && BN * kWRow % (1024 * kWaves) == 0, "tile shape");
    static_assert((KS == 128 || KS == 256) && WS >= 2 && kLds <= kLdsBytes, "stages");
};

// Where a row's 16-byte chunk lies in LDS (the loads put chunk p of a row at p
// ^ swizzle): reads of 16 bytes go in groups of 16 lanes ({0-3, 12-15, 20-27}
// and its like) over 64 banks, and each group's chunks are on different ones.
template <int KS, bool F32>
__device__ inline int w_swizzle(int row) {
    if (KS == 256) return F32 ? swizzle_x(row) : swizzle_w(row);
    return (0 - (row >> (F32 ? 2 : 3))) & 3;
}
__device__ inline int x_swizzle(int row) { return (row & 15) ^ (((row >> 2) ^ (row >> 3)) & 1) << 2; }

// 8 E2M1 codes times 2^(s - 127).
__device__ inline v8bf widen_e2m1(uint32_t v, float s) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 0);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 1);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 2);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, s, 3);
    return v8bf{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
// 8 codes q = 0 .. 15 as numbers: E4M3 codes 0 .. 15 are q 2^-9, its smallest
// numbers.
__device__ inline v8bf widen_int4(uint32_t v) {
    const uint32_t even = v & 0x0F0F0F0Fu, odd = (v >> 4) & 0x0F0F0F0Fu;
    const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u), hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
    return v8bf{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

template <int BM, int BN, int WM, int WN, int KS, int WS, int FMT, bool F32>
__global__ __launch_bounds__(64 * WM * WN) void moedisp_expert_gemm_w4(ExpertW4Args a) {
    using T = Tile<BM, BN, WM, WN, KS, WS, FMT>;
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
    const int steps = (a.k + KS - 1) / KS;
    const int tail = a.k - (steps - 1) * KS;       // channels of the last stage
    constexpr int kGroup = T::kE2m1 ? 32 : 128;    // channels of a scale
    const int wm = wave % WM, wn = wave / WM;
    const int q = lane >> 4, c = lane & 15;
    // XCD x (consecutive workgroups go round the XCDs) takes the x-th run of
    // the tiles, its workgroups every (gridDim / 8)-th of them
    const int total = tiles * a.nt;
    const int per = (total + kXcds - 1) / kXcds;
    const int end = min(total, ((int)(blockIdx.x % kXcds) + 1) * per);
    for (int item = (blockIdx.x % kXcds) * per + blockIdx.x / kXcds; item < end; item += gridDim.x / kXcds) {
        const ExpertTile t = expert_tile<BM, BN>(a.r, item, a.nt, a.n, incl, own);
        const uint8_t* const wp = a.w + ((size_t)t.e * a.n + t.n0) * (a.k / 2);
        const uint16_t* const xp = a.x + t.row0 * a.k;
        const uint8_t* const sp = reinterpret_cast<const uint8_t*>(a.w_scales) +
                                  ((size_t)t.e * (a.k / kGroup) * a.n + t.n0) * T::kSBytes;

        // offsets of the wave's loads in a stage, and which of them lie past
        // the last channel in the last one: zeros (a code 0 of an integer meets
        // an x of zero)
        int woff[T::kWLoads], xoff[T::kXLoads], soff;
        uint32_t out_w = 0, out_x = 0, out_s;
#pragma unroll
        for (int i = 0; i < T::kWLoads; ++i) {
            const int at = (wave * T::kWLoads + i) * 1024 + lane * 16;
            const int row = at / T::kWRow;
            const int chunk = (at % T::kWRow / 16) ^ w_swizzle<KS, F32>(row);
            woff[i] = min(row, t.cols - 1) * (a.k / 2) + chunk * 16;
            out_w |= chunk * 32 >= tail ? 1u << i : 0u;
        }
#pragma unroll
        for (int i = 0; i < T::kXLoads; ++i) {
            const int at = (wave * T::kXLoads + i) * 1024 + lane * 16;
            const int row = at / T::kXRow;
            const int chunk = (at % T::kXRow / 16) ^ x_swizzle(row);
            xoff[i] = min(row, t.rows - 1) * a.k * 2 + chunk * 16;
            out_x |= chunk * 8 >= tail ? 1u << i : 0u;
        }
        {
            const int g = min(lane / T::kSLanes, T::kSGroups - 1);
            const int at = wn * T::kN * T::kSBytes + lane % T::kSLanes * 4;
            soff = g * a.n * T::kSBytes + min(at, t.cols * T::kSBytes - 4);
            out_s = g * kGroup >= tail;
        }
        char* const x_lds = lds + WS * T::kWStage;
        char* const s_lds = x_lds + WS * T::kXStage + wave * 256;

        // stages past the last load the last one again, to no use
        auto issue = [&](int kb, int buf) {
            const int s = min(kb, steps - 1);
            const bool last = s == steps - 1;
            const uint32_t ow = last ? out_w : 0u, ox = last ? out_x : 0u;
#pragma unroll
            for (int i = 0; i < T::kXLoads; ++i)
                load_to_lds_unseen<16>(xp + (size_t)s * KS, x_lds + buf * T::kXStage + (wave * T::kXLoads + i) * 1024,
                                       ox >> i & 1 ? kOutside : xoff[i]);
            load_to_lds_unseen<4>(sp + (size_t)s * T::kSGroups * a.n * T::kSBytes, s_lds + buf * T::kWaves * 256,
                                  last && out_s ? kOutside : soff);
#pragma unroll
            for (int i = 0; i < T::kWLoads; ++i)
                load_to_lds_unseen<16>(wp + (size_t)s * (KS / 2), lds + buf * T::kWStage + (wave * T::kWLoads + i) * 1024,
                                       ow >> i & 1 ? kOutside : woff[i]);
        };

        v4f acc[T::kNT][T::kMT];
#pragma unroll
        for (int i = 0; i < T::kNT; ++i)
#pragma unroll
            for (int j = 0; j < T::kMT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
        for (int p = 0; p < WS - 1; ++p) issue(p, p);

        // columns of products 2t and 2t + 1 that a lane gets: bf16 results 8
        // neighbours, fp32 results 4 of each, 16 bytes to store either way
        const int col = F32 ? c : (c >> 2) * 8 + (c & 3);
        auto col_of = [&](int i) { return F32 ? i * 16 : (i >> 1) * 32 + (i & 1) * 4; };
        const int wsw = w_swizzle<KS, F32>(wn * T::kN + col);
        const int xrow = wm * T::kM + c, xsw = x_swizzle(xrow);
        int buf = 0;
        for (int kb = 0; kb < steps; ++kb) {
            // stage kb is there, and all waves have read the one before, whose
            // place the next load takes
            wait_loads_and_sync<(WS - 2) * T::kLoads>();
            issue(kb + WS - 1, buf == 0 ? WS - 1 : buf - 1);
            const char* st = lds + buf * T::kWStage + (wn * T::kN + col) * T::kWRow;
            const char* xt = x_lds + buf * T::kXStage + xrow * T::kXRow;
            const char* sc = s_lds + buf * T::kWaves * 256;
#pragma unroll
            for (int h = 0; h < T::kH; ++h) {
                v4u wf[T::kNT];
#pragma unroll
                for (int i = 0; i < T::kNT; ++i)
                    wf[i] = *reinterpret_cast<const v4u*>(st + col_of(i) * T::kWRow + (((q + 4 * h) ^ wsw) << 4));
                auto x_at = [&](int j, int d) {
                    const int chunk = ((q + 4 * h) * 4 + d) ^ xsw;
                    return *reinterpret_cast<const v8bf*>(xt + j * 16 * T::kXRow + (chunk << 4));
                };
                if constexpr (T::kE2m1) {
                    float s[T::kNT];
#pragma unroll
                    for (int i = 0; i < T::kNT; ++i)
                        s[i] = __uint_as_float(
                            (uint32_t) * reinterpret_cast<const uint8_t*>(sc + (q + 4 * h) * T::kN + col + col_of(i))
                            << 23);
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        v8bf w[T::kNT];
#pragma unroll
                        for (int i = 0; i < T::kNT; ++i) w[i] = widen_e2m1(wf[i][d], s[i]);
#pragma unroll
                        for (int j = 0; j < T::kMT; ++j) {
                            const v8bf x = x_at(j, d);
#pragma unroll
                            for (int i = 0; i < T::kNT; ++i)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], x, acc[i][j], 0, 0, 0);
                        }
                    }
                } else {
                    // the scales of the lane's four columns
                    float s[T::kNT][4];
                    v8bf w[T::kNT][4];
#pragma unroll
                    for (int i = 0; i < T::kNT; ++i) {
                        const v2i sv = *reinterpret_cast<const v2i*>(
                            sc + (h * T::kN + q * (F32 ? 4 : 8) + col_of(i)) * 2);
                        s[i][0] = bf16_low((uint32_t)sv.x);
                        s[i][1] = bf16_high((uint32_t)sv.x);
                        s[i][2] = bf16_low((uint32_t)sv.y);
                        s[i][3] = bf16_high((uint32_t)sv.y);
#pragma unroll
                        for (int d = 0; d < 4; ++d) w[i][d] = widen_int4(wf[i][d]);
                    }
                    const v4u k8 = {0xC100C100u, 0xC100C100u, 0xC100C100u, 0xC100C100u};  // -8
                    const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < T::kMT; ++j) {
                        v8bf x[4];
                        v4f base, part[T::kNT];
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            x[d] = x_at(j, d);
                            base = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, k8), x[d],
                                                                           d ? base : zero, 0, 0, 0);
                        }
#pragma unroll
                        for (int d = 0; d < 4; ++d)
#pragma unroll
                            for (int i = 0; i < T::kNT; ++i)
                                part[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i][d], x[d], d ? part[i] : base, 0, 0,
                                                                                  0);
#pragma unroll
                        for (int i = 0; i < T::kNT; ++i)
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                acc[i][j][v] = __builtin_fmaf(s[i][v], part[i][v], acc[i][j][v]);
                    }
                }
            }
            buf = buf + 1 == WS ? 0 : buf + 1;
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

template <int BM, int BN, int WM, int WN, int KS, int WS, int FMT, bool F32>
hipError_t launch_tile(ExpertW4Args a, hipStream_t stream) {
    using T = Tile<BM, BN, WM, WN, KS, WS, FMT>;
    a.nt = (a.n + BN - 1) / BN;
    const long long tiles = (long long)a.r.max_rows / BM + a.r.E;  // at least the tiles of any bounds
    if (tiles * a.nt > 0x7FFFFFFFll) return hipErrorInvalidConfiguration;
    long long blocks = (tiles * a.nt + kXcds - 1) / kXcds * kXcds;
    const long long resident = kCus * (kLdsBytes / T::kLds);
    if (blocks > resident) blocks = resident;
    hipLaunchKernelGGL((moedisp_expert_gemm_w4<BM, BN, WM, WN, KS, WS, FMT, F32>), dim3((unsigned)blocks),
                       dim3(T::kThreads), T::kLds, stream, a);
    return hipGetLastError();
}

template <int FMT, bool F32>
hipError_t launch_variant(const ExpertW4Args& a, int mean_rows, hipStream_t stream) {
    const TileShape t = expert_gemm_w4_tile(a.r.E, a.n, mean_rows, FMT);
    if (t.a == 16) return launch_tile<16, 128, 1, 4, 256, 3, FMT, F32>(a, stream);
    if (t.a == 32) return launch_tile<32, 256, 1, 4, 128, 3, FMT, F32>(a, stream);
    if (t.a == 64) return launch_tile<64, 128, 2, 2, 128, 2, FMT, F32>(a, stream);
    if (t.a == 96) return launch_tile<96, 256, 2, 4, 128, 3, FMT, F32>(a, stream);
    return launch_tile<160, 256, 2, 4, 128, 2, FMT, F32>(a, stream);
}

}  // namespace

// Times of a round of all compute units for 4096 channels.  8 experts, K =
// 4096, integers, us for usual rows (columns):
//     rows (n)    16x128  32x256  64x128  96x256  160x256
//       16 (8192)     39      38      52      62       87
//       32 (8192)     53      53      52      62       87
//       64 (8192)     93      70      76      64       89
//      125 (8192)    177     118     118     121       91
//      125 (8208)    190     117     117     175      171
//     1024 (8192)   1343     804     802     709      607
TileShape expert_gemm_w4_tile(int E, int n, int mean_rows, int w4_fmt) {
    static const TileTime e2m1[] = {{16, 128, 2, 22}, {32, 256, 2, 48}, {64, 128, 2, 38}, {96, 256, 1, 48},
                                    {160, 256, 1, 69}};
    static const TileTime int4[] = {{16, 128, 2, 24}, {32, 256, 2, 56}, {64, 128, 2, 52}, {96, 256, 1, 63},
                                    {160, 256, 1, 90}};
    return tile_by_rounds(w4_fmt == MOEDISP_W4_INT4 ? int4 : e2m1, 5, E, n, mean_rows);
}

hipError_t launch_expert_gemm_w4(const ExpertW4Args& a, int mean_rows, int w4_fmt, bool f32_out, hipStream_t stream) {
    if (w4_fmt == MOEDISP_W4_INT4)
        return f32_out ? launch_variant<MOEDISP_W4_INT4, true>(a, mean_rows, stream)
                       : launch_variant<MOEDISP_W4_INT4, false>(a, mean_rows, stream);
    return f32_out ? launch_variant<MOEDISP_W4_E2M1, true>(a, mean_rows, stream)
                   : launch_variant<MOEDISP_W4_E2M1, false>(a, mean_rows, stream);
}

}  // namespace moedisp
