// C ABI of a decoder layer's operators between its products (declared in include/nvfp4.h): argument checks on the host,
// scratch, launches.
//
// Kernels per call (all on the caller's stream):
//   nvfp4_rotary    : k_rotary
//   nvfp4_kv_append : k_kv_append
//   nvfp4_attention : k_attn_rows [-> k_attn_join, where the blocks go in parts], or k_attn_split -> k_attn_join
//   nvfp4_moe       : [k_moe_route ->] k_moe_product or k_moe_rows (up) -> k_moe_down, or k_moe_product or k_moe_rows (down)
//                     -> k_moe_sum
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "host.hpp"
#include "launch.hpp"

namespace {

using nvfp4::aligned;
using nvfp4::plain_dtype;
using nvfp4::status;
using nvfp4::width;
using nvfp4::with_scratch;

constexpr int64_t kMaxTokens = (int64_t)1 << 23, kMaxHeads = 65535;
constexpr int64_t kMaxGroups = (int64_t)1 << 24;  // work-groups of 256 threads along a grid's dimension

int check_cache(const nvfp4_kv_cache_t *c, const nvfp4_sequences_t *s, int64_t tokens) {
    if (!c || !s || tokens < 0 || c->pages < 0 || c->kv_heads <= 0 || c->dim <= 0 || s->seqs < 0 || s->width < 0)
        return NVFP4_ERR_INVALID_ARG;
    if (c->dim % 16 != 0 || c->dim > nvfp4::kMaxHeadDim || c->kv_heads > kMaxHeads || tokens > kMaxTokens ||
        s->seqs > kMaxTokens || s->width > (1 << 24) || c->pages >= ((int64_t)1 << 31))
        return NVFP4_ERR_SHAPE;
    if (s->seqs == 0 || tokens == 0) return NVFP4_OK;
    if (!s->starts && tokens != s->seqs) return NVFP4_ERR_INVALID_ARG;
    if (!s->lengths || !aligned(s->lengths, 4) || !aligned(s->starts, 4)) return NVFP4_ERR_INVALID_ARG;
    if (!s->table || !aligned(s->table, 4) || s->width == 0 || (s->seqs > 1 && s->ldt < s->width)) return NVFP4_ERR_INVALID_ARG;
    if (c->pages == 0 || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !aligned(c->k_codes, 16) ||
        !aligned(c->v_codes, 16))
        return NVFP4_ERR_INVALID_ARG;
    return NVFP4_OK;
}

nvfp4::SeqArgs sequences(const nvfp4_kv_cache_t *c, const nvfp4_sequences_t *s, int64_t tokens) {
    nvfp4::SeqArgs q = {};
    q.table = s->table, q.lengths = s->lengths, q.starts = s->starts, q.ldt = s->ldt;
    q.seqs = s->seqs, q.width = s->width, q.tokens = (int)tokens, q.pages = (int)c->pages;
    return q;
}

// NVFP4_OK where the grids and the lists of an attention call hold its pieces.
int check_plan(int64_t tokens, int seqs, int w, int heads, int kv_heads, int dim) {
    if (tokens < 0 || seqs < 0 || w < 0 || heads <= 0 || kv_heads <= 0 || dim <= 0 || heads % kv_heads != 0)
        return NVFP4_ERR_INVALID_ARG;
    if (heads > kMaxHeads || dim % 16 != 0 || dim > nvfp4::kMaxHeadDim || tokens > kMaxTokens || seqs > kMaxTokens)
        return NVFP4_ERR_SHAPE;
    // a row's token by a multiplication of 32 bits
    const int64_t group = heads / kv_heads;
    if (tokens * group * group >= ((int64_t)1 << 32)) return NVFP4_ERR_SHAPE;
    const nvfp4::AttnPlan plan = nvfp4::plan_attention(tokens, seqs, w, kv_heads, (int)group, dim);
    if (plan.pieces * kv_heads >= kMaxGroups || plan.pieces * (int64_t)w >= ((int64_t)1 << 31)) return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}

}  // namespace

NVFP4_API int nvfp4_rotary(const nvfp4_rotary_args_t *a) {
    if (!a || !plain_dtype(a->dtype) || a->tokens < 0 || a->heads <= 0 || a->dim <= 0) return NVFP4_ERR_INVALID_ARG;
    if (a->axes < 1 || a->axes > nvfp4::kRotaryAxes || (a->inverse != 0 && a->inverse != 1) ||
        (a->positions64 != 0 && a->positions64 != 1) || !(a->base > 0.0) || !(a->base < INFINITY))
        return NVFP4_ERR_INVALID_ARG;
    if (a->tokens > kMaxTokens || a->heads > kMaxHeads || a->dim > nvfp4::kMaxHeadDim) return NVFP4_ERR_SHAPE;
    nvfp4::RotaryArgs p = {};
    for (int i = 0; i < nvfp4::kRotaryAxes; ++i) {
        if (i < a->axes) {
            if (a->sections[i] < 0 || a->sections[i] > nvfp4::kMaxHeadDim) return NVFP4_ERR_INVALID_ARG;
            p.half += a->sections[i];
        }
        p.end[i] = p.half;
    }
    if (p.half == 0) return NVFP4_ERR_INVALID_ARG;
    if (2 * p.half > a->dim) return NVFP4_ERR_SHAPE;
    // The last axis takes what is left, an axis that is not there nothing.
    for (int i = a->axes - 1; i < nvfp4::kRotaryAxes; ++i) p.end[i] = nvfp4::kMaxHeadDim;
    if (a->tokens == 0) return NVFP4_OK;
    const unsigned w = width(a->dtype);
    if (!a->x || !a->y || !a->positions || !aligned(a->x, w) || !aligned(a->y, w) || !aligned(a->positions, a->positions64 ? 8 : 4))
        return NVFP4_ERR_INVALID_ARG;
    if ((a->heads > 1 && (a->xh < a->dim || a->yh < a->dim)) || (a->tokens > 1 && (a->xs < a->dim || a->ys < a->dim)))
        return NVFP4_ERR_INVALID_ARG;
    p.x = a->x, p.y = a->y, p.pos = a->positions;
    p.xs = a->tokens > 1 ? a->xs : 0, p.ys = a->tokens > 1 ? a->ys : 0;
    p.xh = a->heads > 1 ? a->xh : 0, p.yh = a->heads > 1 ? a->yh : 0;
    if (a->x == a->y && (p.xs != p.ys || p.xh != p.yh)) return NVFP4_ERR_INVALID_ARG;
    p.tokens = a->tokens, p.pos_ld = a->tokens, p.heads = a->heads, p.dim = a->dim;
    p.pass = a->x == a->y ? 0 : (a->dim - 2 * p.half + 7) / 8;
    p.pos64 = a->positions64, p.inverse = a->inverse;
    // log2 of base^(-2/R) in two parts, the first with so few bits that its product with a pair's number is exact.
    const long double c = -log2l((long double)a->base) / p.half;
    double hi = (double)c;
    uint64_t bits;
    __builtin_memcpy(&bits, &hi, 8);
    bits &= ~(uint64_t)0xFF;
    __builtin_memcpy(&hi, &bits, 8);
    p.c_hi = hi, p.c_lo = (double)(c - (long double)hi);
    return status(nvfp4::launch_rotary(p, a->dtype == NVFP4_DTYPE_F32, static_cast<hipStream_t>(a->stream)));
}

NVFP4_API int nvfp4_kv_append(const nvfp4_kv_cache_t *c, const nvfp4_sequences_t *s, const void *k, int64_t k_token,
                              int64_t k_head, const void *v, int64_t v_token, int64_t v_head, int dtype, int64_t tokens,
                              void *stream) {
    if (!plain_dtype(dtype)) return NVFP4_ERR_INVALID_ARG;
    const int e = check_cache(c, s, tokens);
    if (e != NVFP4_OK) return e;
    if (tokens == 0 || s->seqs == 0) return NVFP4_OK;
    if (!k || !v || !aligned(k, width(dtype)) || !aligned(v, width(dtype))) return NVFP4_ERR_INVALID_ARG;
    if (tokens > 1 && (k_token < c->dim || v_token < c->dim)) return NVFP4_ERR_INVALID_ARG;
    if (c->kv_heads > 1 && (k_head < c->dim || v_head < c->dim)) return NVFP4_ERR_INVALID_ARG;
    if (tokens / 64 + 2 * (int64_t)s->seqs >= kMaxGroups) return NVFP4_ERR_SHAPE;
    nvfp4::AppendArgs p = {};
    p.seq = sequences(c, s, tokens);
    p.k = k, p.v = v, p.ks = k_token, p.kh = k_head, p.vs = v_token, p.vh = v_head;
    p.k_codes = c->k_codes, p.v_codes = c->v_codes, p.k_scales = c->k_scales, p.v_scales = c->v_scales;
    p.heads = c->kv_heads, p.dim = c->dim;
    return status(nvfp4::launch_kv_append(p, dtype == NVFP4_DTYPE_F32, static_cast<hipStream_t>(stream)));
}

NVFP4_API size_t nvfp4_attention_workspace_bytes(int64_t tokens, int seqs, int w, int heads, int kv_heads, int dim) {
    if (check_plan(tokens, seqs, w, heads, kv_heads, dim) != NVFP4_OK || tokens == 0 || seqs == 0) return 0;
    const nvfp4::AttnPlan plan = nvfp4::plan_attention(tokens, seqs, w, kv_heads, heads / kv_heads, dim);
    return plan.part_bytes + plan.ml_bytes;
}

NVFP4_API int nvfp4_attention(const nvfp4_kv_cache_t *c, const nvfp4_sequences_t *s, const void *q, int64_t q_token,
                              int64_t q_head, int heads, int64_t tokens, float scale, int causal, void *out, void *workspace,
                              size_t workspace_bytes, void *stream) {
    int e = check_cache(c, s, tokens);
    if (e != NVFP4_OK) return e;
    e = check_plan(tokens, s->seqs, s->width, heads, c->kv_heads, c->dim);
    if (e != NVFP4_OK) return e;
    if ((causal != 0 && causal != 1) || !(fabsf(scale) < 1e30f) || !(fabsf(scale) > 1e-30f) || !aligned(workspace, 256)) return NVFP4_ERR_INVALID_ARG;
    if (tokens == 0 || s->seqs == 0) return NVFP4_OK;
    if (!q || !out || !aligned(q, 2) || !aligned(out, 16)) return NVFP4_ERR_INVALID_ARG;
    if ((tokens > 1 && q_token < c->dim) || (heads > 1 && q_head < c->dim)) return NVFP4_ERR_INVALID_ARG;
    nvfp4::AttnArgs p = {};
    p.seq = sequences(c, s, tokens);
    p.q = static_cast<const uint16_t *>(q), p.qs = q_token, p.qh = q_head;
    p.k_codes = c->k_codes, p.v_codes = c->v_codes, p.k_scales = c->k_scales, p.v_scales = c->v_scales;
    p.out = static_cast<uint16_t *>(out), p.scale2 = (float)(fabs((double)scale) * 1.4426950408889634);
    p.slack = 8.0f / p.scale2, p.flip = scale < 0.0f ? 0x80008000u : 0u;
    p.kv_heads = c->kv_heads, p.group = heads / c->kv_heads, p.dim = c->dim, p.causal = causal;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const nvfp4::AttnPlan plan = nvfp4::plan_attention(tokens, s->seqs, s->width, c->kv_heads, p.group, c->dim);
    return with_scratch(workspace, workspace_bytes, plan.part_bytes + plan.ml_bytes, st,
                        [&](void *ws) { return nvfp4::launch_attention(p, ws, st); });
}

namespace {

constexpr int64_t kMaxSide = (int64_t)1 << 21;  // of an expert's products

int check_experts(int64_t tokens, int64_t width, int64_t inner, int experts, int top_k) {
    if (tokens < 0 || width <= 0 || inner <= 0 || experts <= 0 || top_k <= 0) return NVFP4_ERR_INVALID_ARG;
    if (width % 16 != 0 || inner % 16 != 0 || width > kMaxSide || inner > kMaxSide) return NVFP4_ERR_SHAPE;
    if (experts > nvfp4::kMoeMaxExperts || top_k > nvfp4::kMoeMaxTopK || top_k > experts) return NVFP4_ERR_SHAPE;
    if (tokens > nvfp4::kMoeMaxPairs || tokens * top_k > nvfp4::kMoeMaxPairs) return NVFP4_ERR_SHAPE;
    if (2 * width * inner >= ((int64_t)1 << 31)) return NVFP4_ERR_SHAPE;
    // work-groups of 512 threads: one for 16 rows of each chosen expert
    if ((width > inner ? width : inner) / 16 * (experts + tokens * top_k / 16) >= ((int64_t)1 << 23)) return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}

}  // namespace

NVFP4_API size_t nvfp4_moe_workspace_bytes(int64_t tokens, int64_t width, int64_t inner, int experts, int top_k) {
    if (check_experts(tokens, width, inner, experts, top_k) != NVFP4_OK || tokens == 0) return 0;
    return nvfp4::moe_workspace(tokens, width, inner, experts, top_k);
}

NVFP4_API int nvfp4_moe(const nvfp4_moe_args_t *a) {
    if (!a) return NVFP4_ERR_INVALID_ARG;
    const int c = check_experts(a->tokens, a->width, a->inner, a->experts, a->top_k);
    if (c != NVFP4_OK) return c;
    if (!plain_dtype(a->logits_dtype) || a->activation < NVFP4_ACT_NONE || a->activation > NVFP4_ACT_GELU ||
        (a->gated != 0 && (a->gated != 1 || a->activation == NVFP4_ACT_NONE)) || (a->normalize != 0 && a->normalize != 1) ||
        (a->scoring != NVFP4_SCORE_SOFTMAX && a->scoring != NVFP4_SCORE_SIGMOID) || !aligned(a->workspace, 256))
        return NVFP4_ERR_INVALID_ARG;
    if (a->tokens == 0) return NVFP4_OK;
    if (!a->x || !a->logits || !a->up_codes || !a->up_scales || !a->up_alpha || !a->down_codes || !a->down_scales ||
        !a->down_alpha || !a->y)
        return NVFP4_ERR_INVALID_ARG;
    if (a->tokens > 1 && (a->ldx < a->width || a->ldl < a->experts || (a->residual && a->ldr < a->width)))
        return NVFP4_ERR_INVALID_ARG;
    if (a->tokens > 1 && (a->ldx >= ((int64_t)1 << 31) || a->ldl >= ((int64_t)1 << 31) || (a->residual && a->ldr >= ((int64_t)1 << 31))))
        return NVFP4_ERR_SHAPE;
    if (!aligned(a->x, 2) || !aligned(a->logits, width(a->logits_dtype)) || !aligned(a->up_codes, 8) || !aligned(a->down_codes, 8) ||
        !aligned(a->up_alpha, 4) || !aligned(a->down_alpha, 4) || !aligned(a->residual, 2) || !aligned(a->y, 2))
        return NVFP4_ERR_INVALID_ARG;
    nvfp4::MoeArgs p = {};
    p.x = a->x, p.logits = a->logits, p.logits_f32 = a->logits_dtype == NVFP4_DTYPE_F32;
    p.up = {a->up_codes, a->up_scales, a->up_alpha};
    p.down = {a->down_codes, a->down_scales, a->down_alpha};
    p.res = static_cast<const uint16_t *>(a->residual), p.y = static_cast<uint16_t *>(a->y);
    p.tokens = a->tokens, p.width = a->width, p.inner = a->inner;
    p.ldx = a->tokens > 1 ? a->ldx : a->width, p.ldl = a->tokens > 1 ? a->ldl : a->experts;
    p.ldr = a->tokens > 1 ? a->ldr : a->width;
    p.experts = a->experts, p.top_k = a->top_k, p.act = a->activation, p.gated = a->gated;
    p.sigmoid = a->scoring == NVFP4_SCORE_SIGMOID, p.normalize = a->normalize;
    hipStream_t st = static_cast<hipStream_t>(a->stream);
    return with_scratch(a->workspace, a->workspace_bytes, nvfp4::moe_workspace(p.tokens, p.width, p.inner, p.experts, p.top_k), st,
                        [&](void *ws) { return nvfp4::launch_moe(p, ws, st); });
}
