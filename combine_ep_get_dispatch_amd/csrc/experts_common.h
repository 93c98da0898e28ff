// Which rows belong to which expert, and the tiling of the experts' products
// over them (gfx950, wave64).  Shared by the kernels between dispatch and
// combine.
#pragma once

#include <math.h>

#include "kernels_common.h"

namespace moedisp {

constexpr int kCus = 256;          // compute units
constexpr int kScaleBlock = 128;  // channels per scale

// moedisp_rows for the device.
struct RowsArg {
    int E;
    int max_rows;
    int stride;  // 0: contiguous
    int cap;
    int base;
    const int32_t* bounds;
};

struct ExpertGemmArgs {
    RowsArg r;
    int n, k;
    int kb;  // scale blocks of a row (k / 128)
    int nb;  // scale blocks of the columns (ceil(n / 128))
    int nt;  // column tiles
    const uint8_t* x;
    const void* x_scales;
    const uint8_t* w;
    const void* w_scales;
    void* y;
    WsHeader* hdr;
};

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));

__device__ inline uint32_t pack_bf16x2(float lo, float hi) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}
// The binary32 value of a UE8M0 byte: 2^(b - 127), 255 is NaN.
__device__ inline float ue8m0_value(uint32_t b) {
    return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23);
}
__device__ inline float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Loads of `SIZE` bytes per lane straight into LDS at `lds` + lane * max(4, SIZE).
template <int SIZE>
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t rs, char* lds, int voff, int soff) {
    auto* to = (__attribute__((address_space(3))) void*)lds;
    if constexpr (SIZE == 16)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 16, voff, soff, 0, 0);
    else if constexpr (SIZE == 4)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 4, voff, soff, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 1, voff, soff, 0, 0);
}

__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, 0x7FFFFFFF, kRawBufferWord3);
}

// LDS reads of 16 bytes go in groups of 16 lanes ({0-3, 12-15, 20-27} and its
// like) over 64 banks.  Rows of an operand read: 0-3, 8-11, 16-19, 24-27 for
// the weights of bf16 results (see the columns' order), else 0-15.
__device__ inline int swizzle_w(int row) { return ((row >> 1) & 1) | (((row >> 3) & 3) << 1); }
__device__ inline int swizzle_x(int row) { return (row >> 1) & 7; }

// In LDS both operands lie by rows, in bf16, as units of 32 bytes (16 columns
// or channels); unit u of row r is stored at u ^ unit_swizzle(r).  An operand
// read takes the same unit of 4 rows for each of 4 groups of 16 lanes (rows r,
// r + 8, r + 16, r + 24): the swizzle puts 8 of these 16 on different banks,
// as many as 64 banks hold.
__device__ inline int unit_swizzle(int r) { return (r & 3) | ((r >> 1) & 4); }

// Lane 4m + i of 16 reads 8 bytes of row m of four; lane c gets column c of
// the 16 that the four rows' pieces make up, a row each.
__device__ inline v4s read_transposed(const char* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
}

// load_to_lds by an instruction that the compiler does not
// see into: with the builtin it waits for every load into LDS before a
// transposing read, and nothing could be loaded ahead (1372 us against 1182
// for 4096 x 4096 weights and 32768 rows).  There is no result register; the
// waits are wait_loads_and_sync's and wait_own_loads'.  Lanes whose offset lies
// at or past `records` bytes leave zeros in LDS.  The s_nop covers the new m0
// and a descriptor that a vector instruction has just written (five wait
// states).
//
// The clobber of m0 is what makes the compiler set it anew for a load of its
// own.  It warns that reserved registers may not be preserved, as none is here.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int SIZE>
__device__ inline void load_to_lds_unseen(const void* base, const char* lds, int voff, int records = 0x7FFFFFFF) {
    const uint32_t to = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)lds;
    const v4i rs = {__builtin_amdgcn_readfirstlane((int)(uintptr_t)base),
                    __builtin_amdgcn_readfirstlane((int)((uintptr_t)base >> 32) & 0xFFFF),
                    __builtin_amdgcn_readfirstlane(records), kRawBufferWord3};
    if constexpr (SIZE == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to),
                     "v"(voff), "s"(rs)
                     : "memory", "m0");
    else if constexpr (SIZE == 4)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to),
                     "v"(voff), "s"(rs)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_ubyte %1, %2, 0 offen lds" ::"s"(to),
                     "v"(voff), "s"(rs)
                     : "memory", "m0");
}
#pragma clang diagnostic pop

// Waits until at most N of the wave's loads are under way and its LDS accesses
// are done, then for the workgroup.  (A plain barrier would wait for all loads.)
template <int N>
__device__ inline void wait_loads_and_sync() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The workgroup's LDS reads are done; loads may be under way.
__device__ inline void reads_done_and_sync() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The wave's own LDS accesses are done.
__device__ inline void own_lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// At most N of the wave's own loads are under way.
template <int N>
__device__ inline void wait_own_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int CTRL>
__device__ inline float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// op over a row's LPR lanes (aligned), every lane gets it: exchanges by
// register moves, no LDS.  After steps 1 and 2 the lanes of 4 agree, so
// mirroring 8 and then 16 lanes meets the other half.
template <int LPR, class OP>
__device__ inline float row_reduce(float v, OP op) {
    if (LPR > 1) v = op(v, dpp<0xB1>(v));
    if (LPR > 2) v = op(v, dpp<0x4E>(v));
    if (LPR > 4) v = op(v, dpp<0x141>(v));
    if (LPR > 8) v = op(v, dpp<0x140>(v));
    if (LPR > 16) {  // both 16-lane rows' values, in the same order for both
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    if (LPR > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}
template <int LPR>
__device__ inline float lanes_sum(float v) {
    return row_reduce<LPR>(v, [](float x, float y) { return x + y; });
}
template <int LPR>
__device__ inline float lanes_max(float v) {
    return row_reduce<LPR>(v, [](float x, float y) { return fmaxf(x, y); });
}

constexpr long long kCacheBytes = 256ll << 20;  // of the memory-side cache

// First row and number of rows of expert e, from its bounds (b1 is not used
// in the padded layout); false if they break the rules.
__device__ inline bool expert_rows(const RowsArg& r, int e, int b0, int b1, int* first, int* count) {
    if (r.stride > 0) {
        *first = e * r.stride + r.base;
        *count = max(0, min(b0, r.cap));
        return b0 >= 0;
    }
    const bool ok = b0 >= 0 && b1 >= b0 && b1 <= r.max_rows;
    *first = ok ? b0 : 0;
    *count = ok ? b1 - b0 : 0;
    return ok;
}

// One expert of the tiling below: its first row, rows, and the tiles of the
// experts before it.
struct ExpertSpan {
    int e, first, count, tiles_before;
};

// A tile of BM rows by BN columns, and whose it is.
struct ExpertTile {
    int e;
    size_t row0;      // first row of the row buffers
    int n0;           // first column
    int rows, cols;   // that are the expert's and inside n
};

// Tiles of BM rows over all experts (an expert's last one may be shorter),
// counted by one wave on its own: lane l sums the tiles of E/64 experts, one
// scan over the lanes gives the running totals.  Returns the total, -1 if any
// expert's bounds break the rules (then nothing may be computed).  *incl is
// the lane's running total.
template <int BM>
__device__ inline int expert_tiles(const RowsArg& r, int* incl, int* own) {
    const int lane = threadIdx.x & 63;
    const int per = (r.E + 63) >> 6;
    const int lo = min(r.E, lane * per), hi = min(r.E, lo + per);
    int tiles = 0;
    bool ok = true;
    const int up = r.stride > 0 ? 0 : 1;
    for (int e0 = lo; e0 < hi; e0 += 4) {
        int b[5];  // 4 experts' loads in flight
#pragma unroll
        for (int q = 0; q < 5; ++q) b[q] = r.bounds[min(e0 + q, hi - 1 + up)];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            int first, count;
            ok &= e0 + q >= hi || expert_rows(r, e0 + q, b[q], b[q + 1], &first, &count);
            tiles += e0 + q < hi ? (count + BM - 1) / BM : 0;
        }
    }
    if (__ballot(!ok)) return -1;
    *own = tiles;
    *incl = wave_inclusive_scan_dpp(tiles);
    return __builtin_amdgcn_readlane(*incl, 63);
}

// The expert whose tiles hold tile `at` (0 <= at < the total), from the
// running totals of expert_tiles<BM>; uniform over the wave.
template <int BM>
__device__ inline ExpertSpan expert_of_tile(const RowsArg& r, int at, int incl, int own) {
    const int lane = threadIdx.x & 63;
    const int per = (r.E + 63) >> 6;
    const int lo = min(r.E, lane * per), hi = min(r.E, lo + per);
    const int src = __ffsll((unsigned long long)__ballot(incl > at)) - 1;
    ExpertSpan s = {0, 0, 0, 0};
    int before = incl - own;
    if (lane == src) {
        for (int e = lo; e < hi; ++e) {
            int first, count;
            expert_rows(r, e, r.bounds[e], r.bounds[r.stride > 0 ? e : e + 1], &first, &count);
            const int t = (count + BM - 1) / BM;
            if (at >= before && at < before + t) {
                s.e = e;
                s.first = first;
                s.count = count;
                s.tiles_before = before;
            }
            before += t;
        }
    }
    s.e = __builtin_amdgcn_readlane(s.e, src);
    s.first = __builtin_amdgcn_readlane(s.first, src);
    s.count = __builtin_amdgcn_readlane(s.count, src);
    s.tiles_before = __builtin_amdgcn_readlane(s.tiles_before, src);
    return s;
}

// Tile `item` of all experts' tiles of BM x BN (nt column tiles): an expert's
// go by groups of kGroup row tiles, columns, row tiles, so that neighbours
// share rows and weights in an XCD's L2.
template <int BM, int BN>
__device__ inline ExpertTile expert_tile(const RowsArg& r, int item, int nt, int n, int incl, int own) {
    constexpr int kGroup = 8;
    const ExpertSpan s = expert_of_tile<BM>(r, item / nt, incl, own);
    const int mt = (s.count + BM - 1) / BM;
    const int j0 = item - s.tiles_before * nt;
    const int g = j0 / (kGroup * nt);
    const int gm = min(kGroup, mt - g * kGroup);
    const int jr = j0 - g * kGroup * nt;
    const int ni = jr / gm;
    const int m0 = (g * kGroup + jr - ni * gm) * BM;
    return {s.e, (size_t)s.first + m0, ni * BN, min(BM, s.count - m0), min(BN, n - ni * BN)};
}

struct ExpertWgradArgs {
    RowsArg r;
    int n, k;
    int kb;
    int nt, kt;  // tiles of the columns and of the channels
    const uint8_t* x;
    const void* x_scales;
    const uint16_t* dy;
    void* dw;
    WsHeader* hdr;
};

// The bf16 product and its weight gradient.
struct ExpertBf16Args {
    RowsArg r;
    int n, k;
    int nt, kt;  // tiles of the columns, and (weight gradient) of the channels
    const uint16_t* x;
    const uint16_t* w;   // product
    const uint16_t* dy;  // weight gradient
    void* y;             // or dw
    WsHeader* hdr;
};

// The product with 4-bit weights.
struct ExpertW4Args {
    RowsArg r;
    int n, k;
    int nt;  // column tiles
    const uint16_t* x;
    const uint8_t* w;
    const void* w_scales;
    void* y;
    WsHeader* hdr;
};

struct SwigluArgs {
    RowsArg r;
    int inner;
    int blocks;  // scale blocks of h's row (inner / 128)
    const uint16_t* gu;
    const uint16_t* dh;   // backward
    uint16_t* dgu;        // backward: bf16 gradient, may be null
    uint16_t* h;          // forward in bf16
    uint8_t* q;           // codes of h, or of the gradient (may be null)
    void* q_scales;
    WsHeader* hdr;
};

struct RouterArgs {
    int T, E, k;
    int groups, topk_groups, per_group, group_best;
    int group_lanes;   // neighbouring lanes that share a group
    bool sigmoid, normalise;
    bool vec;          // rows of whole 16-byte (8-byte) pieces
    float scale;
    const void* logits;
    const float* bias;      // may be null
    const uint8_t* live;    // may be null
    int32_t* topk_idx;      // backward: read
    float* weights;         // backward: the gradient of the weights, read
    void* d_logits;
    WsHeader* hdr;
};

struct BalanceArgs {
    int S, L, E, k;
    int tile_tokens;   // tokens of a workgroup's tile, inside one sequence
    int tiles;         // tiles per sequence
    float coef;
    int sigmoid;
    const void* logits;
    const int32_t* topk_idx;
    float* loss;
    int32_t* tokens_per_expert;
    int32_t* tokens_per_seq;
    float* psum;       // [S * tiles][E]
    int32_t* count;    // [S * tiles][E]
    int32_t* tokens;   // [S * tiles]
    double* part;      // [S][ceil(E / 64)]: parts of the loss
    int32_t* some;     // [S]: whether the sequence has tokens
    const float* d_loss;
    void* d_logits;
    WsHeader* hdr;
};

// Lanes that share a row of E logits, 8 experts each (more beyond 512).
inline int balance_lanes(int E) {
    int lanes = 1;
    while (lanes < 64 && lanes * 8 < E) lanes *= 2;
    return lanes;
}

// Tile of rows by columns (product), of columns by channels (weight gradient).
struct TileShape {
    int a, b;
};
// A tile and the time of a round of its workgroups on all compute units, so
// many to a unit (any unit of time).
struct TileTime {
    int rows, cols, per_cu;
    double time;
};
// The tile whose rounds take the least time, the first of equal ones.
// Experts' rows are taken to scatter round the usual number as random choices
// do, by its square root.  Workgroups that share a unit go on into the next
// round; those alone there start together.
inline TileShape tile_by_rounds(const TileTime* kinds, int count, int E, int n, int mean_rows) {
    const double mean = mean_rows, spread = 2.0 * sqrt(mean);
    TileShape best = {kinds[0].rows, kinds[0].cols};
    double least = 0.0;
    for (int i = 0; i < count; ++i) {
        const TileTime& k = kinds[i];
        // row tiles of an expert: one more for each multiple of the tile that is exceeded
        const double whole = floor(fmax(mean - spread, 0.0) / k.rows);
        double row_tiles = 1.0 + whole;
        for (double m = whole + 1.0; m * k.rows < mean + spread; m += 1.0)
            row_tiles += fmin(1.0, fmax(0.0, (mean - m * k.rows) / spread + 0.5));
        double rounds = row_tiles * E * (((long long)n + k.cols - 1) / k.cols) / (k.per_cu * kCus);
        rounds = k.per_cu > 1 ? fmax(rounds, 1.0) : ceil(rounds);
        if (i == 0 || rounds * k.time < least) {
            best = {k.rows, k.cols};
            least = rounds * k.time;
        }
    }
    return best;
}
TileShape expert_gemm_tile(int E, int n, int mean_rows, bool f32_out);
// How the router's choice lies in a wave: lanes of a row, experts of a lane.
struct RouterShape {
    int lanes, per_lane;
};
RouterShape router_shape(int T, int E);
TileShape expert_gemm_bf16_tile(int E, int n, int mean_rows);
TileShape expert_gemm_w4_tile(int E, int n, int mean_rows, int w4_fmt);
TileShape expert_wgrad_bf16_tile(int E, int n, int k);
TileShape expert_wgrad_tile(int E, int n, int k, int scale_fmt, bool f32_out);
long long swiglu_rows_at_once(int blocks);
long long swiglu_blocks(int max_rows, int blocks, bool backward);

// Workgroups of the balance loss's backward pass over so many tiles.
inline long long balance_backward_blocks(long long tiles) { return tiles <= 4096 ? tiles : 2048; }

hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, int scale_fmt, bool f32_out, bool accumulate,
                               hipStream_t stream);
hipError_t launch_router(const RouterArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_router_backward(const RouterArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_expert_gemm_bf16(const ExpertBf16Args& a, int mean_rows, bool kn, bool f32_out,
                                   hipStream_t stream);
hipError_t launch_expert_gemm_w4(const ExpertW4Args& a, int mean_rows, int w4_fmt, bool f32_out, hipStream_t stream);
hipError_t launch_expert_wgrad_bf16(const ExpertBf16Args& a, bool f32_out, bool accumulate, hipStream_t stream);
hipError_t launch_swiglu_bf16(const SwigluArgs& a, hipStream_t stream);
hipError_t launch_swiglu(const SwigluArgs& a, int scale_fmt, hipStream_t stream);
hipError_t launch_swiglu_backward(const SwigluArgs& a, int scale_fmt, hipStream_t stream);
hipError_t launch_balance(const BalanceArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_balance_backward(const BalanceArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_expert_gemm(const ExpertGemmArgs& a, int mean_rows, int scale_fmt, bool f32_out,
                              hipStream_t stream);

}  // namespace moedisp
