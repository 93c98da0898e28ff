// Which rows belong to which expert, and the tiling of the experts' products
// over them (gfx950, wave64).  Shared by the kernels between dispatch and
// combine.
#pragma once

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

// Waits until at most N of the wave's loads are under way and its LDS accesses
// are done, then for the workgroup.  (A plain barrier would wait for all loads.)
template <int N>
__device__ inline void wait_loads_and_sync() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

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

struct SwigluArgs {
    RowsArg r;
    int inner;
    int blocks;  // scale blocks of h's row (inner / 128)
    const uint16_t* gu;
    const uint16_t* dh;   // backward
    uint16_t* dgu;        // backward: bf16 gradient, may be null
    uint8_t* q;           // codes of h, or of the gradient (may be null)
    void* q_scales;
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
TileShape expert_gemm_tile(int E, int n, int mean_rows, bool f32_out);
TileShape expert_wgrad_tile(int E, int n, int k, int scale_fmt, bool f32_out);
long long swiglu_rows_at_once(int blocks);
long long swiglu_blocks(int max_rows, int blocks, bool backward);

// Workgroups of the balance loss's backward pass over so many tiles.
inline long long balance_backward_blocks(long long tiles) { return tiles <= 4096 ? tiles : 2048; }

hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, int scale_fmt, bool f32_out, bool accumulate,
                               hipStream_t stream);
hipError_t launch_swiglu(const SwigluArgs& a, int scale_fmt, hipStream_t stream);
hipError_t launch_swiglu_backward(const SwigluArgs& a, int scale_fmt, hipStream_t stream);
hipError_t launch_balance(const BalanceArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_balance_backward(const BalanceArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_expert_gemm(const ExpertGemmArgs& a, int mean_rows, int scale_fmt, bool f32_out,
                              hipStream_t stream);

}  // namespace moedisp
