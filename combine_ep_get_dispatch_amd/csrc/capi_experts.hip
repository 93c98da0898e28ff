// C ABI of the experts' products, the gated activation and the balance loss:
// argument checks on the host, then launches on the caller's stream.  As in
// capi.hip, a rejected call touches no device and enqueues nothing.
#include <math.h>
#include <stddef.h>
#include <string.h>

#include "moedisp_tools.h"
#include "experts_common.h"

namespace moedisp {
namespace {

bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int status_of(hipError_t e) {
    if (e == hipSuccess) return MOEDISP_OK;
    return e == hipErrorInvalidConfiguration ? MOEDISP_ERR_UNSUPPORTED : MOEDISP_ERR_HIP;
}

constexpr int kMaxChannels = 65536;     // the scales of a weight tile's rows lie in LDS
constexpr int kMaxColumns = 1 << 20;

int check_rows(const moedisp_rows* r, const int32_t* bounds) {
    if (!r || !bounds) return MOEDISP_ERR_INVALID_ARG;
    if (r->num_experts < 1 || r->max_rows < 0 || r->expert_stride < 0 || r->expected_rows < 0)
        return MOEDISP_ERR_INVALID_ARG;
    if (r->expert_stride > 0) {
        if (r->expert_capacity < 0 || r->row_base < 0 ||
            (long long)r->row_base + r->expert_capacity > r->expert_stride)
            return MOEDISP_ERR_INVALID_ARG;
        if ((long long)r->num_experts * r->expert_stride != r->max_rows) return MOEDISP_ERR_INVALID_ARG;
    } else if (r->expert_capacity != 0 || r->row_base != 0) {
        return MOEDISP_ERR_INVALID_ARG;
    }
    if (r->num_experts > kMaxExperts || r->max_rows >= (1 << 30)) return MOEDISP_ERR_UNSUPPORTED;
    if (!aligned_to(bounds, 4)) return MOEDISP_ERR_MISALIGNED;
    return MOEDISP_OK;
}

RowsArg rows_arg(const moedisp_rows& r, const int32_t* bounds) {
    RowsArg a;
    a.E = r.num_experts;
    a.max_rows = r.max_rows;
    a.stride = r.expert_stride;
    a.cap = r.expert_capacity;
    a.base = r.row_base;
    a.bounds = bounds;
    return a;
}

int mean_rows(const moedisp_rows& r) {
    if (r.expected_rows > 0) return r.expected_rows;
    return r.expert_stride > 0 ? r.expert_capacity : (r.max_rows + r.num_experts - 1) / r.num_experts;
}

int check_header(void* ws, size_t ws_bytes) {
    if (!ws) return MOEDISP_ERR_INVALID_ARG;
    if (!aligned_to(ws, 256)) return MOEDISP_ERR_MISALIGNED;
    if (ws_bytes < sizeof(WsHeader)) return MOEDISP_ERR_WORKSPACE_TOO_SMALL;
    return MOEDISP_OK;
}

int check_scale_fmt(int fmt) {
    return fmt == MOEDISP_SCALE_FP32 || fmt == MOEDISP_SCALE_UE8M0 ? MOEDISP_OK : MOEDISP_ERR_UNSUPPORTED;
}
bool scales_aligned(const void* p, int fmt) { return fmt == MOEDISP_SCALE_UE8M0 || aligned_to(p, 4); }

// Columns, channels and types of the two products.
int check_product(int n, int k, int scale_fmt, int out_dtype) {
    if (n <= 0 || k <= 0) return MOEDISP_ERR_INVALID_ARG;
    if (k % kScaleBlock != 0 || n % 8 != 0) return MOEDISP_ERR_UNSUPPORTED;
    if (n > kMaxColumns || k > kMaxChannels) return MOEDISP_ERR_UNSUPPORTED;
    if (out_dtype != MOEDISP_BF16 && out_dtype != MOEDISP_FP32) return MOEDISP_ERR_UNSUPPORTED;
    return check_scale_fmt(scale_fmt);
}

int check_inner(int inner, int scale_fmt) {
    if (inner <= 0) return MOEDISP_ERR_INVALID_ARG;
    if (inner % kScaleBlock != 0 || inner > kMaxChannels) return MOEDISP_ERR_UNSUPPORTED;
    return check_scale_fmt(scale_fmt);
}

int check_balance(const moedisp_balance* b) {
    if (!b) return MOEDISP_ERR_INVALID_ARG;
    if (b->num_seqs < 0 || b->seq_len < 0 || b->num_experts < 1 || b->topk < 1 || b->topk > b->num_experts)
        return MOEDISP_ERR_INVALID_ARG;
    if (!isfinite(b->coef)) return MOEDISP_ERR_INVALID_ARG;
    if (b->num_experts > kMaxExperts || b->topk > kMaxTopk) return MOEDISP_ERR_UNSUPPORTED;
    if (b->score != MOEDISP_SCORE_SOFTMAX && b->score != MOEDISP_SCORE_SIGMOID) return MOEDISP_ERR_UNSUPPORTED;
    if (b->logits_dtype != MOEDISP_BF16 && b->logits_dtype != MOEDISP_FP32) return MOEDISP_ERR_UNSUPPORTED;
    if ((long long)b->num_seqs * b->seq_len >= (1ll << 30) / b->topk) return MOEDISP_ERR_UNSUPPORTED;
    return MOEDISP_OK;
}

size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }

struct BalancePlan {
    int tile_tokens, tiles;
    size_t psum, count, tokens, part, some, total;
};

constexpr int kBalanceTiles = 2048;
// Tiles of a sequence: about 2048 over all sequences (8 workgroups per
// compute unit: 27 us for 131072 rows of 256 bf16 logits, 30 with 1024), whole passes of the rows that a workgroup takes at once.
BalancePlan plan_balance(const moedisp_balance& b) {
    BalancePlan p;
    const long long S = b.num_seqs, L = b.seq_len, E = b.num_experts;
    const long long once = 256 / balance_lanes(b.num_experts);
    long long want = S > 0 ? (kBalanceTiles + S - 1) / S : 1;
    long long tile = (L + want - 1) / want;
    tile = (tile + once - 1) / once * once;
    if (tile < once) tile = once;
    p.tile_tokens = (int)tile;
    p.tiles = (int)((L + tile - 1) / tile);
    const size_t all = (size_t)S * p.tiles;
    p.psum = sizeof(WsHeader);
    p.count = round256(p.psum + all * E * 4);
    p.tokens = round256(p.count + all * E * 4);
    p.part = round256(p.tokens + all * 4);
    p.some = round256(p.part + (size_t)S * ((E + 63) / 64) * 8);
    p.total = round256(p.some + (size_t)S * 4);
    return p;
}

BalanceArgs balance_args(const moedisp_balance& b, const BalancePlan& p) {
    BalanceArgs a = {};
    a.S = b.num_seqs;
    a.L = b.seq_len;
    a.E = b.num_experts;
    a.k = b.topk;
    a.tile_tokens = p.tile_tokens;
    a.tiles = p.tiles;
    a.coef = b.coef;
    a.sigmoid = b.score == MOEDISP_SCORE_SIGMOID;
    return a;
}

}  // namespace
}  // namespace moedisp

using namespace moedisp;

extern "C" {

int ep_expert_gemm(const moedisp_rows* rows, int32_t n, int32_t k, int32_t scale_fmt, const void* x,
                   const void* x_scales, const void* w, const void* w_scales, const int32_t* row_bounds, void* y,
                   int32_t out_dtype, void* ws, size_t ws_bytes, void* stream) {
    int st = check_rows(rows, row_bounds);
    if (st || (st = check_product(n, k, scale_fmt, out_dtype))) return st;
    if (!w || !w_scales || (rows->max_rows > 0 && (!x || !x_scales || !y))) return MOEDISP_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(y, 16) || !scales_aligned(x_scales, scale_fmt) ||
        !scales_aligned(w_scales, scale_fmt))
        return MOEDISP_ERR_MISALIGNED;
    if ((st = check_header(ws, ws_bytes))) return st;
    ExpertGemmArgs a = {};
    a.r = rows_arg(*rows, row_bounds);
    a.n = n;
    a.k = k;
    a.kb = k / kScaleBlock;
    a.nb = (n + kScaleBlock - 1) / kScaleBlock;
    a.x = (const uint8_t*)x;
    a.x_scales = x_scales;
    a.w = (const uint8_t*)w;
    a.w_scales = w_scales;
    a.y = y;
    a.hdr = (WsHeader*)ws;
    return status_of(
        launch_expert_gemm(a, mean_rows(*rows), scale_fmt, out_dtype == MOEDISP_FP32, (hipStream_t)stream));
}

int ep_expert_wgrad(const moedisp_rows* rows, int32_t n, int32_t k, int32_t scale_fmt, const void* x,
                    const void* x_scales, const void* dy, const int32_t* row_bounds, void* dw, int32_t out_dtype,
                    int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
    int st = check_rows(rows, row_bounds);
    if (st || (st = check_product(n, k, scale_fmt, out_dtype))) return st;
    if (accumulate != 0 && accumulate != 1) return MOEDISP_ERR_INVALID_ARG;
    if (accumulate && out_dtype != MOEDISP_FP32) return MOEDISP_ERR_UNSUPPORTED;
    if (!dw || (rows->max_rows > 0 && (!x || !x_scales || !dy))) return MOEDISP_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(dy, 16) || !aligned_to(dw, 16) || !scales_aligned(x_scales, scale_fmt))
        return MOEDISP_ERR_MISALIGNED;
    if ((st = check_header(ws, ws_bytes))) return st;
    ExpertWgradArgs a = {};
    a.r = rows_arg(*rows, row_bounds);
    a.n = n;
    a.k = k;
    a.kb = k / kScaleBlock;
    a.x = (const uint8_t*)x;
    a.x_scales = x_scales;
    a.dy = (const uint16_t*)dy;
    a.dw = dw;
    a.hdr = (WsHeader*)ws;
    return status_of(
        launch_expert_wgrad(a, scale_fmt, out_dtype == MOEDISP_FP32, accumulate != 0, (hipStream_t)stream));
}

int ep_swiglu_quant(const moedisp_rows* rows, int32_t inner, int32_t scale_fmt, const void* gu,
                    const int32_t* row_bounds, void* h, void* h_scales, void* ws, size_t ws_bytes, void* stream) {
    int st = check_rows(rows, row_bounds);
    if (st || (st = check_inner(inner, scale_fmt))) return st;
    if (rows->max_rows > 0 && (!gu || !h || !h_scales)) return MOEDISP_ERR_INVALID_ARG;
    if (!aligned_to(gu, 16) || !aligned_to(h, 16) || !scales_aligned(h_scales, scale_fmt))
        return MOEDISP_ERR_MISALIGNED;
    if ((st = check_header(ws, ws_bytes))) return st;
    SwigluArgs a = {};
    a.r = rows_arg(*rows, row_bounds);
    a.inner = inner;
    a.blocks = inner / kScaleBlock;
    a.gu = (const uint16_t*)gu;
    a.q = (uint8_t*)h;
    a.q_scales = h_scales;
    a.hdr = (WsHeader*)ws;
    return status_of(launch_swiglu(a, scale_fmt, (hipStream_t)stream));
}

int ep_swiglu_backward(const moedisp_rows* rows, int32_t inner, int32_t scale_fmt, const void* gu, const void* dh,
                       const int32_t* row_bounds, void* dgu, void* dgu_q, void* dgu_scales, void* ws,
                       size_t ws_bytes, void* stream) {
    int st = check_rows(rows, row_bounds);
    if (st || (st = check_inner(inner, scale_fmt))) return st;
    if ((dgu_q == nullptr) != (dgu_scales == nullptr)) return MOEDISP_ERR_INVALID_ARG;
    if (rows->max_rows > 0 && (!gu || !dh || (!dgu && !dgu_q))) return MOEDISP_ERR_INVALID_ARG;
    if (!aligned_to(gu, 16) || !aligned_to(dh, 16) || !aligned_to(dgu, 16) || !aligned_to(dgu_q, 16) ||
        !scales_aligned(dgu_scales, scale_fmt))
        return MOEDISP_ERR_MISALIGNED;
    if ((st = check_header(ws, ws_bytes))) return st;
    SwigluArgs a = {};
    a.r = rows_arg(*rows, row_bounds);
    a.inner = inner;
    a.blocks = inner / kScaleBlock;
    a.gu = (const uint16_t*)gu;
    a.dh = (const uint16_t*)dh;
    a.dgu = (uint16_t*)dgu;
    a.q = (uint8_t*)dgu_q;
    a.q_scales = dgu_scales;
    a.hdr = (WsHeader*)ws;
    return status_of(launch_swiglu_backward(a, scale_fmt, (hipStream_t)stream));
}

size_t ep_balance_workspace_bytes(const moedisp_balance* b) {
    if (check_balance(b) != MOEDISP_OK) return 0;
    return plan_balance(*b).total;
}

int ep_balance_loss(const moedisp_balance* b, const void* logits, const int32_t* topk_idx, float* loss,
                    int32_t* tokens_per_expert, int32_t* tokens_per_seq, void* ws, size_t ws_bytes, void* stream) {
    int st = check_balance(b);
    if (st) return st;
    const bool any = b->num_seqs > 0 && b->seq_len > 0;
    if (!loss || (any && (!logits || !topk_idx)) || (b->num_seqs > 0 && (!tokens_per_expert || !tokens_per_seq)))
        return MOEDISP_ERR_INVALID_ARG;
    if (!aligned_to(logits, 16) || !aligned_to(topk_idx, 4) || !aligned_to(loss, 4) ||
        !aligned_to(tokens_per_expert, 4) || !aligned_to(tokens_per_seq, 4))
        return MOEDISP_ERR_MISALIGNED;
    if ((st = check_header(ws, ws_bytes))) return st;
    const BalancePlan p = plan_balance(*b);
    if (ws_bytes < p.total) return MOEDISP_ERR_WORKSPACE_TOO_SMALL;
    BalanceArgs a = balance_args(*b, p);
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.loss = loss;
    a.tokens_per_expert = tokens_per_expert;
    a.tokens_per_seq = tokens_per_seq;
    a.psum = (float*)((char*)ws + p.psum);
    a.count = (int32_t*)((char*)ws + p.count);
    a.tokens = (int32_t*)((char*)ws + p.tokens);
    a.part = (double*)((char*)ws + p.part);
    a.some = (int32_t*)((char*)ws + p.some);
    a.hdr = (WsHeader*)ws;
    return status_of(launch_balance(a, b->logits_dtype == MOEDISP_BF16, (hipStream_t)stream));
}

int ep_balance_loss_backward(const moedisp_balance* b, const void* logits, const int32_t* topk_idx,
                             const int32_t* tokens_per_expert, const int32_t* tokens_per_seq, const float* d_loss,
                             void* d_logits, void* stream) {
    int st = check_balance(b);
    if (st) return st;
    const bool any = b->num_seqs > 0 && b->seq_len > 0;
    if (!d_loss || (any && (!logits || !topk_idx || !tokens_per_expert || !tokens_per_seq || !d_logits)))
        return MOEDISP_ERR_INVALID_ARG;
    if (!aligned_to(logits, 16) || !aligned_to(d_logits, 16) || !aligned_to(topk_idx, 4) ||
        !aligned_to(tokens_per_expert, 4) || !aligned_to(tokens_per_seq, 4) || !aligned_to(d_loss, 4))
        return MOEDISP_ERR_MISALIGNED;
    BalanceArgs a = balance_args(*b, plan_balance(*b));
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.tokens_per_expert = const_cast<int32_t*>(tokens_per_expert);
    a.tokens_per_seq = const_cast<int32_t*>(tokens_per_seq);
    a.d_loss = d_loss;
    a.d_logits = d_logits;
    return status_of(launch_balance_backward(a, b->logits_dtype == MOEDISP_BF16, (hipStream_t)stream));
}

int ep_expert_plan_query(const moedisp_rows* rows, int32_t n, int32_t k, int32_t scale_fmt, int32_t out_dtype,
                         moedisp_expert_plan_info* info, size_t info_bytes) {
    if (!info || info_bytes != sizeof(moedisp_expert_plan_info)) return MOEDISP_ERR_INVALID_ARG;
    memset(info, 0, sizeof *info);
    static const int32_t some_bounds = 0;  // the query has no bounds; the rows' own rules are checked
    int st = check_rows(rows, &some_bounds);
    if (st || (st = check_product(n, k, scale_fmt, out_dtype))) return st;
    info->struct_bytes = (int64_t)sizeof *info;
    const TileShape g = expert_gemm_tile(rows->num_experts, n, mean_rows(*rows), out_dtype == MOEDISP_FP32);
    info->product_rows = g.a;
    info->product_cols = g.b;
    const TileShape w = expert_wgrad_tile(rows->num_experts, n, k, scale_fmt, out_dtype == MOEDISP_FP32);
    info->wgrad_cols = w.a;
    info->wgrad_channels = w.b;
    const int blocks = k / kScaleBlock;
    info->swiglu_rows = swiglu_rows_at_once(blocks);
    info->swiglu_blocks = swiglu_blocks(rows->max_rows, blocks, false);
    info->swiglu_backward_blocks = swiglu_blocks(rows->max_rows, blocks, true);
    return MOEDISP_OK;
}

int ep_balance_plan_query(const moedisp_balance* b, moedisp_balance_plan_info* info, size_t info_bytes) {
    if (!info || info_bytes != sizeof(moedisp_balance_plan_info)) return MOEDISP_ERR_INVALID_ARG;
    memset(info, 0, sizeof *info);
    const int st = check_balance(b);
    if (st) return st;
    info->struct_bytes = (int64_t)sizeof *info;
    const BalancePlan p = plan_balance(*b);
    info->tile_tokens = p.tile_tokens;
    info->tiles = p.tiles;
    info->lanes = balance_lanes(b->num_experts);
    info->rows_at_once = 256 / info->lanes;
    info->passes = p.tile_tokens / info->rows_at_once;
    info->backward_blocks = balance_backward_blocks((long long)b->num_seqs * p.tiles);
    return MOEDISP_OK;
}

}  // extern "C"
