// gfx950 attention over a paged cache in 8 bits.
//
// For a row (query token i of its sequence's last n, query head h of G to a key/value head) and the tokens t < limit that
// it sees (limit = len - n + i + 1, or len where every query sees every token):
//     s_t = scale (q . k_t),  o = sum_t e^(s_t) v_t / sum_t e^(s_t),  0 where the row sees none.
// q is bf16; k and v are E4M3 codes times a power of two per block of 64 tokens (cache.hpp), exact in bf16. Products
// on v_mfma_f32_16x16x32_bf16 with fp32 sums; maximum, sum and output are fp32, carried from block to block (one
// pass); a probability is rounded to bf16 for the second product, which takes bf16 (half a step, at most 2^-8 of a term,
// independent between terms: of the size of the output's own rounding), and not for the sum. What rounding left as a second
// bf16 operand would take the output's error from 0.0022 of its norm to the 0.0017 of its own rounding, and costs, measured in the
// kernels of few rows: nothing for one sequence, 1 % for 64 (108 -> 109 us), 3 to 7 % for drafts, short tables and heads of 80
// (17.7 -> 18.7 us, 15.9 -> 16.8, 39 -> 42), 14 % for tiles of 32 rows; prompts are bound by the products themselves.
//
// A block of 64 tokens by 16 rows takes no exchange between lanes. Lane l has r = l % 16 and g = l / 16.
//   S^T = K Q^T: slot 4 a + j of key tile t (a = 0..3, t = 0..3) holds token 16 a + 4 t + j, since the rows of an operand
//     may be any rows; a lane ends with the scores of its row r for the 16 tokens 16 g .. + 15.
//   O^T = V^T P^T: the lane's 16 probabilities, packed, are the second operand as they are, with k = 16 g + 8 u + 0..7 in
//     product u; the first has 16 columns of V by the same tokens: 16 neighbouring bytes of a turned page.
//   The lane ends with the columns 16 d + 4 g + j of row r, so the running maximum and sum are its own.
// The maximum that exponents are taken against follows the scores only where one exceeds it by 2^8: then, seldom, the
// lanes of a row agree on the new one and the sums are rescaled. p <= 2^8 has the same relative precision.
//
// A block whose scale byte is 255 (a NaN or an infinity was written) makes NaN of the rows that see any of it,
// and is not multiplied: rows that see none of it are not touched. Codes behind a sequence's end are not trusted: their
// scores are masked, their values zeroed.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "act.hpp"
#include "cache.hpp"
#include "codec.hpp"
#include "launch.hpp"
#include "mx.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4, kAttnThreads = 64 * kWaves;
constexpr float kNegInf = -__builtin_inff();

// Eight codes times a power of two (exact) as an operand.
__device__ __forceinline__ bf16x8 operand8(uint32_t a, uint32_t b, float scale) {
    const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, scale, false);
    const bf16x2 q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, scale, true);
    const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, scale, false);
    const bf16x2 s = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, scale, true);
    return __builtin_bit_cast(bf16x8, u32x4{__builtin_bit_cast(uint32_t, p), __builtin_bit_cast(uint32_t, q),
                                            __builtin_bit_cast(uint32_t, r), __builtin_bit_cast(uint32_t, s)});
}

// Over the four lanes of a row (l % 16 alike), the same result in each.
__device__ __forceinline__ float row_max(float v) {
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    return fmaxf(__uint_as_float(b.x), __uint_as_float(b.y));
}
__device__ __forceinline__ float row_sum(float v) {
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    v = __uint_as_float(a.x) + __uint_as_float(a.y);
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    return __uint_as_float(b.x) + __uint_as_float(b.y);
}

// e^(a - b) in powers of two, 0 for a = -inf whatever b.
__device__ __forceinline__ float weight(float a, float b) { return a == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(a - b); }

// Masks the bytes of the first n of 16 tokens.
__device__ __forceinline__ u32x4 tokens_kept(int n) {
    u32x4 keep;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int k = n - 4 * w;
        keep[w] = k >= 4 ? ~0u : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
    }
    return keep;
}

// What a wave carries for its 16 RT rows: per lane the maximum (of the row), the sum (of the lane's tokens), the output.
template <int KS, int RT>
struct Rows {
    f32x4 o[RT][4 * KS];
    float m[RT], l[RT];
    int lim[RT];  // tokens that the lane's row sees (0: no such row)
};

// The token of a row (among the sequence's new ones): row / group by a multiplication, exact while rows * group stay
// below 2^32 (a work-group of a short call is bound by the way to its blocks, and divisions are the longest steps on it).
__device__ __forceinline__ int token_of(const AttnArgs &p, int row) {
    return p.per_group ? (int)__umulhi((uint32_t)row, p.per_group) : row;
}

// The tokens that a row sees, more for a later one.
__device__ __forceinline__ int seen_by(const AttnArgs &p, const Seq &q, int row) {
    return p.causal ? min(max(q.len - q.n + token_of(p, row) + 1, 0), q.len) : q.len;
}

// The lane's rows row0 + 16 r + l % 16 of the sequence: their queries as operands, and what they see.
template <int KS, int RT, bool FULL>
__device__ __forceinline__ void take_rows(const AttnArgs &p, const Seq &q, int64_t h, int row0, bf16x8 (&Q)[RT][2 * KS], Rows<KS, RT> &R) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = row0 + 16 * r + r16, tok = token_of(p, row), sub = row - tok * p.group;
        const bool in = tok < q.n;
        R.lim[r] = !in ? 0 : p.causal ? min(max(q.len - q.n + tok + 1, 0), q.len) : q.len;
        const uint16_t *x = p.q + (int64_t)(q.first + tok) * p.qs + (h * p.group + sub) * p.qh;
#pragma unroll
        for (int k = 0; k < 2 * KS; ++k) {
            const int c = 64 * (k >> 1) + 16 * g + 8 * (k & 1);
            u32x4 v = {0u, 0u, 0u, 0u};
            if (in && (FULL || c < p.dim)) v = *reinterpret_cast<const u32x4_any *>(x + c);
            v ^= p.flip;  // a negative scale: -q, exact
            // An infinity is read as NaN (exponent of ones: the carry sets the quiet bit). The row is NaN either way where it sees
            // a token, but scores that are all -inf could not be told from masked ones, which give zeros.
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] |= (((v[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u) >> 9;
            Q[r][k] = __builtin_bit_cast(bf16x8, v);
        }
        R.m[r] = kNegInf, R.l[r] = 0.0f;
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d) R.o[r][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
}

// LDS bytes of a wave's block: K's rows with an odd number of 16-byte pieces from one to the next and four pieces more per 16
// rows, so that the sixteen lanes that read one piece of the tokens 16 a + 4 t + j meet no bank twice; V's tiles of 16 columns.
template <int KS>
constexpr int kWaveK = 64 * (64 * KS + 16) + 4 * 64;
template <int KS>
constexpr int kWaveLds = kWaveK<KS> + 4096 * KS;

// KS: head sizes to 64 KS; FULL: 64 KS itself (else what is past dim is read from inside it: K's meet zeros of q, V's
// sums are not stored). RT: tiles of 16 rows. The wave takes blocks b0, b0 + step, ... below b1 of sequence s. `safe`:
// the tokens that every row of the wave sees (blocks below need no mask). `wl`: the wave's kWaveLds bytes.
//
// A block's codes are read whole, 1 KB a load: lanes that read an operand's pieces where they lie are rows apart, which takes
// four times the address cycles. They are turned in LDS, where only the wave itself writes and reads, and the next
// block's loads are in flight meanwhile.
template <int KS, int RT, bool FULL>
__device__ __forceinline__ void attend(const AttnArgs &p, const Seq &q, int s, int64_t h, int row0, int b0, int b1, int step,
                                       Rows<KS, RT> &R, uint8_t *wl) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int dim = FULL ? 64 * KS : p.dim, per = dim / 16;  // 16-byte pieces of a token; loads of a block's K, and of its V
    const int count = b1 > b0 ? (b1 - b0 + step - 1) / step : 0;
    const int safe = seen_by(p, q, row0);  // blocks below need no mask
    const int pitch = dim + (per & 1 ? 0 : 16);
    uint8_t *const wv = wl + kWaveK<KS>;
    // Pages and scales of 64 of the wave's blocks, one a lane.
    int page = -1;
    uint32_t scales = 0u;
    auto look_up = [&](int i0) __attribute__((always_inline)) {
        page = -1, scales = 0u;
        if (i0 + lane < count) page = page_of(p.seq, s, b0 + (i0 + lane) * step);
        if (page >= 0) {
            const int64_t at = (int64_t)page * p.kv_heads + h;
            scales = (uint32_t)p.k_scales[at] | (uint32_t)p.v_scales[at] << 8;
        }
    };
    // Page i; a page that is not there, or one of NaNs, is read as page 0 and left out.
    auto base_of = [&](int i) __attribute__((always_inline)) {
        const int pg = __builtin_amdgcn_readlane(page, i & 63);
        return ((int64_t)max(pg, 0) * p.kv_heads + h) * (kPage * dim);
    };
    u32x4 kc[4 * KS], vc[4 * KS];
    const uint32_t loff = 16u * (uint32_t)lane;
    auto load_k = [&](int64_t base) __attribute__((always_inline)) {
        const uint8_t *c = p.k_codes + base;
#pragma unroll
        for (int i = 0; i < 4 * KS; ++i) kc[i] = *reinterpret_cast<const u32x4 *>(c + 1024 * (FULL ? i : min(i, per - 1)) + loff);
    };
    auto load_v = [&](int64_t base) __attribute__((always_inline)) {
        const uint8_t *c = p.v_codes + base;
#pragma unroll
        for (int i = 0; i < 4 * KS; ++i) vc[i] = *reinterpret_cast<const u32x4 *>(c + 1024 * (FULL ? i : min(i, per - 1)) + loff);
    };
    auto k_place = [&](int token, int c) __attribute__((always_inline)) { return token * pitch + 64 * (token >> 4) + 16 * c; };
    look_up(0);
    bf16x8 Q[RT][2 * KS];
    take_rows<KS, RT, FULL>(p, q, h, row0, Q, R);
    if (count == 0) return;
    int64_t base = base_of(0);
    load_k(base);
    load_v(base);
    int poison = 0x7FFFFFFF;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        const int t0 = (b0 + i * step) * kPage;
        const int pg = __builtin_amdgcn_readlane(page, i & 63);
        const uint32_t sc = (uint32_t)__builtin_amdgcn_readlane((int)scales, i & 63);
        const uint32_t ke = sc & 255u, ve = sc >> 8;
        const bool nan = pg >= 0 && (ke == 255u || ve == 255u), live = pg >= 0 && !nan;
        if (nan) poison = min(poison, t0);
        if (((i + 1) & 63) == 0) look_up(i + 1);
        const int64_t next = base_of(i + 1 < count ? i + 1 : i);
        const float kscale = mx_scale_value(ke), vscale = live ? mx_scale_value(ve) : 1.0f;
        wave_handover();
#pragma unroll
        for (int k = 0; k < 4 * KS; ++k) {
            const int e = 64 * (FULL ? k : min(k, per - 1)) + lane;
            *reinterpret_cast<u32x4 *>(wl + k_place(e / per, e % per)) = kc[k];
        }
        load_k(next);
        wave_handover();
        f32x4 S[RT][4] = {};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            __builtin_amdgcn_sched_barrier(0);  // tile by tile: operands of all tiles at once take more registers than there are
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int piece = FULL ? 4 * k + g : min(4 * k + g, per - 1);
                const u32x4 c = *reinterpret_cast<const u32x4 *>(wl + k_place(16 * (r16 >> 2) + 4 * t + (r16 & 3), piece));
                const bf16x8 a = operand8(c.x, c.y, kscale), b = operand8(c.z, c.w, kscale);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    S[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, Q[r][2 * k], S[r][t], 0, 0, 0);
                    S[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, Q[r][2 * k + 1], S[r][t], 0, 0, 0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (t0 + kPage > q.len || !live) {  // codes behind the end may be any bytes
            const u32x4 keep = tokens_kept(live ? q.len - t0 - 16 * (lane & 3) : 0);
#pragma unroll
            for (int d = 0; d < 4 * KS; ++d) vc[d] &= keep;
        }
        // Piece u of column d of a tile at u ^ (d / 4 % 4).
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d) *reinterpret_cast<u32x4 *>(wv + 1024 * d + (lane >> 2) * 64 + 16 * ((lane ^ (lane >> 4)) & 3)) = vc[d];
        load_v(next);
        const bool mask = t0 + kPage > safe || !live;
        bool more = false;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float top = kNegInf;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v = S[r][t][j];
                    if (mask) v = live && t0 + 16 * g + 4 * t + j < R.lim[r] ? v : kNegInf;
                    S[r][t][j] = v;
                    top = fmaxf(top, v);
                }
            more |= top > R.m[r] + p.slack;
        }
        if (__any(more)) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                float top = kNegInf;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) top = fmaxf(top, S[r][t][j]);
                const float m = row_max(fmaxf(top, R.m[r]));
                const float w = R.m[r] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((R.m[r] - m) * p.scale2);
                R.m[r] = m;
                R.l[r] *= w;
#pragma unroll
                for (int d = 0; d < 4 * KS; ++d) R.o[r][d] *= w;
            }
        }
        bf16x8 P[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float m = (R.m[r] == kNegInf ? 0.0f : -R.m[r]) * p.scale2;
            uint32_t w[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[r][t][j], p.scale2, m));
                    R.l[r] += e[j];
                }
                w[2 * t] = pack_bf16(e[0], e[1]);
                w[2 * t + 1] = pack_bf16(e[2], e[3]);
            }
            P[r][0] = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
            P[r][1] = __builtin_bit_cast(bf16x8, u32x4{w[4], w[5], w[6], w[7]});
        }
        wave_handover();
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d) {
            if (d % 2 == 0) __builtin_amdgcn_sched_barrier(0);
            const u32x4 c = *reinterpret_cast<const u32x4 *>(wv + 1024 * d + r16 * 64 + 16 * ((g ^ (r16 >> 2)) & 3));
            const bf16x8 a = operand8(c.x, c.y, vscale), b = operand8(c.z, c.w, vscale);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                R.o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, P[r][0], R.o[r][d], 0, 0, 0);
                R.o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, P[r][1], R.o[r][d], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
        if (R.lim[r] > poison) R.l[r] = __builtin_nanf("");
}

__device__ __forceinline__ uint16_t *out_row(const AttnArgs &p, const Seq &q, int64_t h, int row) {
    const int tok = token_of(p, row);
    return p.out + ((int64_t)(q.first + tok) * p.kv_heads * p.group + h * p.group + (row - tok * p.group)) * p.dim;
}

// LDS bytes of a work-group whose waves share the blocks: each wave's block, afterwards each wave's sums.
template <int KS>
constexpr int kSumsLds = kWaves * 16 * (64 * KS + 4) * 4;
template <int KS>
constexpr int kBlocksLds = kWaves * kWaveLds<KS> > kSumsLds<KS> ? kWaves * kWaveLds<KS> : kSumsLds<KS>;

// The sums of a work-group's waves over `rows` rows of a tile from row0 on, in wave order: the output, where they are `whole`, or
// a part of it, at the rows `at` of the scratch.
template <int KS, int RT>
__device__ __forceinline__ void join_waves(const AttnArgs &p, const Seq &q, int64_t h, int row0, int rows, const Rows<KS, RT> &R, bool whole,
                                           int64_t at, uint8_t *lds, float (*lds_ml)[kWaves][16]) {
    constexpr int kDim = 64 * KS;
    float (*const lds_o)[16][kDim + 4] = reinterpret_cast<float (*)[16][kDim + 4]>(lds);
    float (*const lds_m)[16] = lds_ml[0], (*const lds_l)[16] = lds_ml[1];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const float l = row_sum(R.l[r]);
        if (16 * r >= rows) break;
        __syncthreads();  // the blocks, or the tile before, have been read
        if (g == 0) lds_m[wave][r16] = R.m[r] * p.scale2, lds_l[wave][r16] = l;
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d) *reinterpret_cast<f32x4 *>(&lds_o[wave][r16][16 * d + 4 * g]) = R.o[r][d];
        __syncthreads();
        // 16 threads a row, each four columns of every 64
        const int row = tid >> 4, c0 = 4 * (tid & 15);
        if (16 * r + row < rows) {
            float m = kNegInf;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) m = fmaxf(m, lds_m[w][row]);
            float f[kWaves], sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                f[w] = weight(lds_m[w][row], m);
                sum += lds_l[w][row] == 0.0f ? 0.0f : f[w] * lds_l[w][row];
            }
            const float inv = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
            float *po = p.part + (at + 16 * r + row) * p.dim;
            uint16_t *o = out_row(p, q, h, row0 + 16 * r + row);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int c = 64 * k + c0;
                if (c >= p.dim) break;
                f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < kWaves; ++w) v += *reinterpret_cast<const f32x4 *>(&lds_o[w][row][c]) * f[w];
                v *= inv;
                if (whole)
                    *reinterpret_cast<uint2 *>(o + c) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                else
                    *reinterpret_cast<f32x4 *>(po + c) = v;
            }
            if (!whole && c0 == 0) {
                float *ml = p.part_ml + (at + 16 * r + row) * 2;
                ml[0] = m, ml[1] = sum;
            }
        }
    }
}

// Rows over the waves, for prompts: a work-group takes 64 RT rows of a sequence and head, a wave 16 RT of them, over the
// blocks that they see, or over one of gridDim.y parts of these (k_attn_join adds the parts). Bound by the matrix cores and
// the exponentials, so a block's codes are decoded once per work-group, into LDS in the order of the operands (every read is 1
// KB in lane order), each block in one of two buffers while the block before is computed. Two work-groups a CU, so that
// one's exponentials run beside the other's products: 32 rows a wave in 256 registers. Prompts of 8800 tokens, 32 heads of 128:
// 530 us, 1.05 PFLOP/s; 64 rows a wave, one work-group a CU: 1105 us (sums move between the two register files); eight
// waves a work-group: 618; each wave decoding for itself: 2010. Decoding and LDS stores take some 90 of them, the
// exponentials 78.
//
// Slot m of key tile t holds token 16 t + m; a lane then ends with the scores of the tokens 16 t + 4 g + j, and V's
// operand u takes tokens 32 u + 4 g + j and 32 u + 16 + 4 g + j, j = 0..3, as k = 8 g .. + 7.
//
// A piece of at most 32 rows, as of a single token beside prompts, takes the way of few rows instead, 16 at a time with the
// blocks over the waves (a prompt of 2048 tokens and 16 single ones over 32000 each: 639 -> 211 us, 16 of six tokens, 24 rows, 620 -> 399;
// 63 single ones over 8000: 318 -> 231).
template <int KS>
constexpr int kRowsLds = 4 * 64 * 64 * KS * 2 > kBlocksLds<KS> ? 4 * 64 * 64 * KS * 2 : kBlocksLds<KS>;

template <int KS, int RT, bool FULL>
__global__ __launch_bounds__(kAttnThreads, KS <= 2 ? 2 : 1) void k_attn_rows(AttnArgs p) {
    constexpr int kRows = 16 * RT * kWaves, kHalf = 64 * 64 * KS * 2;  // LDS bytes of a block's K or V
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ float lds_ml[2][kWaves][16];
    uint8_t *const lds_k = lds, *const lds_v = lds + 2 * kHalf;
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // The heads run fastest over the grid, so that a head's blocks stay in one XCD's L2; the last pieces of a
    // sequence, which see the most, go first.
    const int64_t h = blockIdx.x % p.kv_heads;
    const int piece = p.pieces - 1 - (int)(blockIdx.x / p.kv_heads);
    const int s = piece_sequence(p.seq, piece, p.group, log2_of(kRows), 1);
    const Seq q = sequence(p.seq, s);
    const int first = (piece - piece_base(p.seq, s, p.group, log2_of(kRows), 1)) * kRows;
    if (first >= q.n * p.group || first < 0) return;
    // The blocks that some row of the work-group sees, or this part of them.
    const int in_piece = min(kRows, q.n * p.group - first);
    const int reach = seen_by(p, q, first + in_piece - 1), all = (reach + kPage - 1) / kPage;
    const int start = (int)((int64_t)all * blockIdx.y / gridDim.y), count = (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y);
    const int64_t part = ((h * p.pieces + piece) * gridDim.y + blockIdx.y) * kRows;
    if (in_piece <= 32) {
#pragma unroll 1
        for (int t = 0; t < in_piece; t += 16) {
            Rows<KS, 1> F;
            if (t) __syncthreads();  // the tile before has been read
            attend<KS, 1, FULL>(p, q, s, h, first + t, start + wave, count, kWaves, F, lds + wave * kWaveLds<KS>);
            join_waves<KS, 1>(p, q, h, first + t, min(16, in_piece - t), F, gridDim.y == 1, part + t, lds, lds_ml);
        }
        return;
    }
    const int row0 = first + 16 * RT * wave, dim = FULL ? 64 * KS : p.dim;
    bf16x8 Q[RT][2 * KS];
    Rows<KS, RT> R;
    const int safe = seen_by(p, q, row0);
    take_rows<KS, RT, FULL>(p, q, h, row0, Q, R);

    // Pages and scales of 64 blocks, one a lane.
    int page = -1;
    uint32_t scales = 0u;
    auto look_up = [&](int i0) __attribute__((always_inline)) {
        page = -1, scales = 0u;
        if (i0 + lane < count) page = page_of(p.seq, s, i0 + lane);
        if (page >= 0) {
            const int64_t at = (int64_t)page * p.kv_heads + h;
            scales = (uint32_t)p.k_scales[at] | (uint32_t)p.v_scales[at] << 8;
        }
    };
    // What the wave knows of a block: whether it is there, and its scales (looked up 64 at a time, from `ahead` on).
    struct Block {
        int64_t base;
        float ks, vs;
        int live;
    };
    int poison = 0x7FFFFFFF, ahead = start;
    auto block_of = [&](int b) __attribute__((always_inline)) {
        if (b >= ahead && b < count) look_up(b), ahead = b + 64;  // b == ahead
        const int pg = __builtin_amdgcn_readlane(page, (b - start) & 63);
        const uint32_t sc = (uint32_t)__builtin_amdgcn_readlane((int)scales, (b - start) & 63);
        const bool nan = (sc & 255u) == 255u || (sc >> 8) == 255u;
        Block B;
        B.live = b < count && pg >= 0 && !nan;
        if (b < count && nan) poison = min(poison, b * kPage);
        B.base = ((int64_t)max(pg, 0) * p.kv_heads + h) * (kPage * dim);
        B.ks = B.live ? mx_scale_value(sc & 255u) : 1.0f, B.vs = B.live ? mx_scale_value(sc >> 8) : 1.0f;
        return B;
    };
    // A thread's codes of a block: KS pieces of 16 of K (row e / (dim / 16)) and of V (row e / 4), e = tid + 256 i.
    const int per = dim / 16, pieces = kPage * per;
    u32x4 kraw[KS], vraw[KS];
    Block kb, vb;  // of the raw pieces
    auto load_k = [&](int b) __attribute__((always_inline)) {
        kb = block_of(b);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const int e = tid + kAttnThreads * i;
            kraw[i] = *reinterpret_cast<const u32x4 *>(p.k_codes + kb.base + 16u * (uint32_t)(FULL ? e : min(e, pieces - 1)));
        }
    };
    auto load_v = [&]() __attribute__((always_inline)) {
        vb = kb;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const int e = tid + kAttnThreads * i;
            vraw[i] = *reinterpret_cast<const u32x4 *>(p.v_codes + vb.base + 16u * (uint32_t)(FULL ? e : min(e, pieces - 1)));
        }
    };
    // Piece c = 4 i + g of a token: k = 64 i + 16 g .. + 15, the operands 2 i and 2 i + 1 of the token's tile, at lane
    // (token % 16) ^ c within the sixteen of g: the eight pieces of a row meet no bank twice.
    auto store_k = [&](int b) __attribute__((always_inline)) {
        uint8_t *const to = lds_k + (b & 1) * kHalf;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const int e = tid + kAttnThreads * i, token = e / per, c = e % per;
            if (!FULL && e >= pieces) continue;
            uint8_t *at = to + ((((token >> 4) * 2 * KS + 2 * (c >> 2)) * 64) + 16 * (c & 3) + ((token & 15) ^ c)) * 16;
            *reinterpret_cast<bf16x8 *>(at) = operand8(kraw[i].x, kraw[i].y, kb.ks);
            *reinterpret_cast<bf16x8 *>(at + 1024) = operand8(kraw[i].z, kraw[i].w, kb.ks);
        }
    };
    auto store_v = [&](int b) __attribute__((always_inline)) {
        uint8_t *const to = lds_v + (b & 1) * kHalf;
        if ((b + 1) * kPage > q.len || !vb.live) {  // codes behind the end, and of no page, may be any bytes
            const u32x4 keep = tokens_kept(vb.live ? q.len - b * kPage - 16 * (tid & 3) : 0);
#pragma unroll
            for (int i = 0; i < KS; ++i) vraw[i] &= keep;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const int e = tid + kAttnThreads * i, d = e >> 2, c = e & 3;  // column; 16 tokens
            if (!FULL && e >= pieces) continue;
            uint8_t *at = to + (((d >> 4) * 2 + (c >> 1)) * 64 + (d & 15)) * 16 + 8 * (c & 1);
            const u32x4 a = __builtin_bit_cast(u32x4, operand8(vraw[i].x, vraw[i].y, vb.vs));
            const u32x4 b4 = __builtin_bit_cast(u32x4, operand8(vraw[i].z, vraw[i].w, vb.vs));
            *reinterpret_cast<u32x2 *>(at) = u32x2{a.x, a.y};
            *reinterpret_cast<u32x2 *>(at + 256) = u32x2{a.z, a.w};
            *reinterpret_cast<u32x2 *>(at + 512) = u32x2{b4.x, b4.y};
            *reinterpret_cast<u32x2 *>(at + 768) = u32x2{b4.z, b4.w};
        }
    };
    auto scores = [&](int b, f32x4 (&S)[RT][4]) __attribute__((always_inline)) {
        const uint8_t *const from = lds_k + (b & 1) * kHalf;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < 4; ++t) S[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 2 * KS; ++k) {
            const int c = 4 * (k >> 1) + g;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const bf16x8 a = *reinterpret_cast<const bf16x8 *>(from + ((t * 2 * KS + k) * 64 + 16 * g + (r16 ^ c)) * 16);
#pragma unroll
                for (int r = 0; r < RT; ++r) S[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, Q[r][k], S[r][t], 0, 0, 0);
            }
        }
    };
    if (!FULL) {  // columns past dim: zeros that no block overwrites
        for (int e = tid; e < 4 * kHalf / 16; e += kAttnThreads) reinterpret_cast<u32x4 *>(lds)[e] = u32x4{0u, 0u, 0u, 0u};
        __syncthreads();
    }
    int live = 0;  // of the block that is computed
    if (start < count) {
        load_k(start);
        load_v();
        live = kb.live;
        store_k(start);
        store_v(start);
        load_k(start + 1);
        load_v();
        lds_barrier();
    }
#pragma unroll 1
    for (int b = start; b < count; ++b) {
        const int t0 = b * kPage;
        f32x4 S[RT][4];
        scores(b, S);
        store_k(b + 1);
        store_v(b + 1);
        const int next_live = kb.live;
        load_k(b + 2);
        load_v();
        if (t0 + kPage > safe || !live) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        S[r][t][j] = live && t0 + 16 * t + 4 * g + j < R.lim[r] ? S[r][t][j] : kNegInf;
        }
        // The maximum that exponents are taken against, raised where a score is far above it.
        bool more = false;
        float top[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            top[r] = kNegInf;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) top[r] = fmaxf(top[r], S[r][t][j]);
            more |= top[r] > R.m[r] + p.slack;
        }
        if (__any(more)) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float m = row_max(fmaxf(top[r], R.m[r]));
                const float w = R.m[r] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((R.m[r] - m) * p.scale2);
                R.m[r] = m;
                R.l[r] *= w;
#pragma unroll
                for (int d = 0; d < 4 * KS; ++d) R.o[r][d] *= w;
            }
        }
        bf16x8 P[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float m = (R.m[r] == kNegInf ? 0.0f : -R.m[r]) * p.scale2;
            uint32_t w[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[r][t][j], p.scale2, m));
                    R.l[r] += e[j];
                }
                w[2 * t] = pack_bf16(e[0], e[1]);
                w[2 * t + 1] = pack_bf16(e[2], e[3]);
            }
            P[r][0] = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
            P[r][1] = __builtin_bit_cast(bf16x8, u32x4{w[4], w[5], w[6], w[7]});
        }
        const uint8_t *const from = lds_v + (b & 1) * kHalf;
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bf16x8 a = *reinterpret_cast<const bf16x8 *>(from + ((d * 2 + u) * 64 + lane) * 16);
#pragma unroll
                for (int r = 0; r < RT; ++r) R.o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, P[r][u], R.o[r][d], 0, 0, 0);
            }
        live = next_live;
        lds_barrier();
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const float l = row_sum(R.lim[r] > poison ? __builtin_nanf("") : R.l[r]);
        const int row = row0 + 16 * r + r16;
        if (row >= q.n * p.group) continue;
        if (gridDim.y > 1) {  // a part: k_attn_join adds them
            const int64_t at = part + (row - first);
            if (g == 0) p.part_ml[2 * at] = R.m[r] * p.scale2, p.part_ml[2 * at + 1] = l;
#pragma unroll
            for (int d = 0; d < 4 * KS; ++d)
                if (FULL || 16 * d < p.dim) *reinterpret_cast<f32x4 *>(p.part + at * dim + 16 * d + 4 * g) = R.o[r][d];
            continue;
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t *o = out_row(p, q, h, row) + 4 * g;
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d)
            if (FULL || 16 * d < p.dim) {
                const f32x4 v = R.o[r][d] * inv;
                *reinterpret_cast<uint2 *>(o + 16 * d) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            }
    }
}

// ------------------------------------------------------------------------- blocks over work-groups

// Few rows: the blocks of all sequences, in order, are one list per head that is cut into equal shares, one per
// work-group, whatever the lengths; bound by reading the cache once. A work-group goes through the pieces of its
// share (a piece: blocks of one tile of 16 RT rows of a sequence), its waves taking every fourth block; their results
// are joined in LDS in wave order. A tile that lies in one share is finished there, else its parts go to scratch and
// k_attn_join adds them in order of the shares.
//
// Where there are at least two work-groups for each tile, a tile's blocks are padded to whole shares in the list, so that no
// work-group has two pieces, one after the other: short calls are bound by the way through one (16 sequences of 500 to 5000
// tokens, 21 to 42 rows: 14.3 -> 11.8 us).
struct Share {
    uint32_t total, groups;  // blocks of the head's list; work-groups that share them
    uint32_t unit, more;     // blocks of a share; the first `more` shares have one more
    __device__ __forceinline__ uint32_t begin(uint32_t j) const { return j * unit + min(j, more); }
    __device__ __forceinline__ uint32_t owner(uint32_t u) const {
        const uint32_t longer = more * (unit + 1u);
        return u < longer ? u / (unit + 1u) : more + (u - longer) / unit;
    }
    // of a tile's blocks in the list
    bool whole;
    __device__ __forceinline__ uint32_t padded(uint32_t blocks) const { return whole ? (blocks + unit - 1) / unit * unit : blocks; }
};

__device__ __forceinline__ int tiles_of(const AttnArgs &p, const Seq &q, int size) { return (q.n * p.group + size - 1) >> log2_of(size); }
__device__ __forceinline__ int blocks_of(const Seq &q) { return (q.len + kPage - 1) / kPage; }

// 64 sequences, one a lane, with the blocks (of all their tiles) in front of them in the list. By whole waves.
struct Window {
    int s0;
    Seq q;
    uint32_t mine, upto, before;  // the lane's blocks; those of the window up to and with it; those before the window
    __device__ __forceinline__ void load(const AttnArgs &p, int size, int from, uint32_t front) {
        const int lane = threadIdx.x & 63;
        s0 = from, before = front, mine = 0u, q = Seq{0, 0, 0};
        if (s0 + lane < p.seq.seqs) {
            q = sequence(p.seq, s0 + lane);
            mine = (uint32_t)(tiles_of(p, q, size) * blocks_of(q));
        }
        upto = sums_to(mine);
    }
    __device__ __forceinline__ uint32_t total() const { return before + (uint32_t)__builtin_amdgcn_readlane((int)upto, 63); }
    __device__ __forceinline__ Seq seq(int s) const {
        return Seq{__builtin_amdgcn_readlane(q.first, s - s0), __builtin_amdgcn_readlane(q.n, s - s0), __builtin_amdgcn_readlane(q.len, s - s0)};
    }
    __device__ __forceinline__ uint32_t begin(int s) const {
        return before + (uint32_t)__builtin_amdgcn_readlane((int)(upto - mine), s - s0);
    }
};

// The first window, and the list's length.
__device__ __forceinline__ uint32_t list_total(const AttnArgs &p, int size, Window &w) {
    w.load(p, size, 0, 0u);
    uint32_t sum = w.total();
    for (int s0 = 64; s0 < p.seq.seqs; s0 += 64) {
        Window v;
        v.load(p, size, s0, sum);
        sum = v.total();
    }
    return sum;
}

// The shares, and the first window of the list as they are cut.
__device__ __forceinline__ Share share_of(const AttnArgs &p, int size, Window &w) {
    Share sh;
    sh.total = list_total(p, size, w), sh.whole = false, sh.more = 0u;
    // Long shares go to half as many work-groups, one a CU: parts and pieces are fewer (64 sequences of 300 to 16000 tokens:
    // 110 -> 98 us), where short ones lack loads in flight.
    uint32_t groups = (uint32_t)p.groups;
    if (sh.total >= groups * (kWaves * 8u)) groups = (groups + 1u) / 2u;
    if (p.seq.seqs > 1 && p.seq.seqs <= 64) {
        const bool any = w.mine != 0u;
        const uint32_t tiles = wave_sum(any ? (uint32_t)tiles_of(p, w.q, size) : 0u);
        if (tiles > 1u && 2u * tiles <= groups) {
            const uint32_t least = (sh.total + groups - tiles - 1u) / (groups - tiles);
            sh.unit = (least + kWaves - 1u) / kWaves * kWaves, sh.whole = true;  // a block for each wave
            if (any) w.mine = (uint32_t)tiles_of(p, w.q, size) * sh.padded((uint32_t)blocks_of(w.q));
            w.upto = sums_to(w.mine);
            sh.total = w.total(), sh.groups = groups;  // (of which the last may have none)
            return sh;
        }
    }
    // Not less than a block for each wave of a work-group.
    sh.groups = max(1u, min(groups, (sh.total + kWaves - 1) / kWaves));
    sh.unit = sh.total / sh.groups, sh.more = sh.total - sh.unit * sh.groups;
    return sh;
}

// Where share j's part of a tile lies: a share has at most two that it does not finish, the end of a tile that an earlier
// share begins (an even place) and the beginning of one (`first`, an odd place).
__device__ __forceinline__ int64_t part_place(const AttnArgs &p, int64_t h, uint32_t j, bool first) {
    return (h * p.groups + j) * 2 + (first ? 1 : 0);
}

template <int KS, int RT, bool FULL>
__global__ __launch_bounds__(kAttnThreads, RT * KS <= 2 ? 2 : 1) void k_attn_split(AttnArgs p) {
    constexpr int kRows = 16 * RT;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kBlocksLds<KS>];
    __shared__ float lds_ml[2][kWaves][16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t h = blockIdx.x % p.kv_heads;
    const uint32_t j = blockIdx.x / p.kv_heads;
    Window w;
    const Share sh = share_of(p, kRows, w);
    if (j >= sh.groups || sh.total == 0u) return;
    uint32_t u = sh.begin(j);
    const uint32_t end = min(sh.begin(j + 1), sh.total);
    while (u < end) {
        while (u >= w.total()) w.load(p, kRows, w.s0 + 64, w.total());
        const int s = w.s0 + __ffsll((unsigned long long)__ballot(w.before + w.upto > u)) - 1;
        const Seq q = w.seq(s);
        const uint32_t nb = (uint32_t)blocks_of(q), in_list = sh.padded(nb), at = w.begin(s);
        const int tile = (int)((u - at) / in_list), b0 = (int)((u - at) % in_list), b1 = (int)min(nb, b0 + (end - u));
        u += min(in_list - b0, end - u);
        const int row0 = tile * kRows, rows = min(kRows, q.n * p.group - row0);
        Rows<KS, RT> R;
        attend<KS, RT, FULL>(p, q, s, h, row0, b0 + wave, b1, kWaves, R, lds + wave * kWaveLds<KS>);
        join_waves<KS, RT>(p, q, h, row0, rows, R, b0 == 0 && b1 == (int)nb, part_place(p, h, j, b0 == 0) * kRows, lds, lds_ml);
        __syncthreads();  // LDS is free for the next piece
    }
}

// The tiles whose blocks lie in several shares, and the rows of sequences of no tokens (zeros). TOGETHER: a work-group takes a
// row, its waves every fourth part, joined in wave order; else a wave takes a row.
template <bool TOGETHER>
__global__ __launch_bounds__(kAttnThreads) void k_attn_join(AttnArgs p, int size) {
    constexpr int kShare = TOGETHER ? kWaves : 1;
    __shared__ float lds_o[TOGETHER ? kWaves : 1][TOGETHER ? kMaxHeadDim : 1], lds_l[kWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t h = blockIdx.x % p.kv_heads;
    const int piece = (int)(blockIdx.x / p.kv_heads), row = TOGETHER ? (int)blockIdx.y : (int)blockIdx.y * kWaves + wave;  // of the tile
    const int turn = TOGETHER ? wave : 0;
    if (row >= size) return;
    Window w;
    const Share sh = share_of(p, size, w);
    const int s = piece_sequence(p.seq, piece, p.group, log2_of(size), 1);
    while (s >= w.s0 + 64) w.load(p, size, w.s0 + 64, w.total());
    const Seq q = w.seq(s);
    const int tile = piece - piece_base(p.seq, s, p.group, log2_of(size), 1);
    if (tile < 0 || tile >= tiles_of(p, q, size) || tile * size + row >= q.n * p.group) return;
    uint16_t *o = out_row(p, q, h, tile * size + row);
    const int c = 4 * lane;
    const uint32_t nb = (uint32_t)blocks_of(q);
    if (nb == 0u) {
        if (turn == 0 && c < p.dim) *reinterpret_cast<uint2 *>(o + c) = make_uint2(0u, 0u);
        return;
    }
    int parts = p.parts, apart = 1;  // of k_attn_rows: all tiles alike, side by side
    int64_t at = (h * p.pieces + piece) * p.parts;
    if (parts == 0) {
        // Starts that run backwards give sequences the same rows, and a list that may pass 32 bits: a place in it is then past its
        // end, or nothing is left of it, and there are no such parts. (k_attn_split takes places below the end alone.)
        if (sh.total == 0u) return;
        const uint32_t u0 = w.begin(s) + (uint32_t)tile * sh.padded(nb);
        const uint32_t j0 = sh.owner(u0), j1 = sh.owner(u0 + nb - 1);
        if (j0 >= j1 || j1 >= sh.groups) return;
        parts = (int)(j1 - j0 + 1), apart = 2;
        at = part_place(p, h, j0, false);
    }
    // The row in part k.
    auto place = [&](int k) __attribute__((always_inline)) { return (at + (int64_t)k * apart + (k == 0 ? apart - 1 : 0)) * size + row; };
    // The first parts are on their way while their weights are found.
    constexpr int kAhead = 4;
    const float *o4 = p.part + min(c, p.dim - 4);
    f32x4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ahead[i] = *reinterpret_cast<const f32x4 *>(o4 + place(min(kShare * i + turn, parts - 1)) * p.dim);
    float m = kNegInf;
    for (int k = lane; k < parts; k += 64) m = fmaxf(m, p.part_ml[2 * place(k)]);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k));
    float sum = 0.0f;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < parts; k0 += 64 * kShare) {  // 64 parts of the wave, one a lane
        const int k = k0 + kShare * lane + turn;
        float f = 0.0f;
        if (k < parts) {
            const float *ml = p.part_ml + 2 * place(k);
            f = weight(ml[0], m);
            sum += ml[1] == 0.0f ? 0.0f : f * ml[1];
        }
        const int here = min(64, (parts - k0 - turn + kShare - 1) / kShare);
        int i = 0;
        if (k0 == 0) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                if (a < here) v += ahead[a] * __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), a));
            i = kAhead;
        }
        for (; i < here; ++i)
            v += *reinterpret_cast<const f32x4 *>(o4 + place(k0 + kShare * i + turn) * p.dim) *
                 __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), i));
    }
    sum = wave_sum(sum);
    if constexpr (TOGETHER) {
        if (c < p.dim) *reinterpret_cast<f32x4 *>(&lds_o[wave][c]) = v;
        if (lane == 0) lds_l[wave] = sum;
        __syncthreads();
        if (wave != 0) return;
        sum = 0.0f, v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (c < p.dim)
#pragma unroll
            for (int k = 0; k < kWaves; ++k) sum += lds_l[k], v += *reinterpret_cast<const f32x4 *>(&lds_o[k][c]);
    }
    if (c >= p.dim) return;
    v *= sum == 0.0f ? 0.0f : 1.0f / sum;
    *reinterpret_cast<uint2 *>(o + c) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

template <int KS, bool FULL>
void split(const AttnArgs &p, int rt, hipStream_t st) {
    const dim3 grid((unsigned)(p.groups * p.kv_heads)), block(kAttnThreads);
    if constexpr (KS < 4)
        if (rt == 2) {
            hipLaunchKernelGGL((k_attn_split<KS, 2, FULL>), grid, block, 0, st, p);
            return;
        }
    hipLaunchKernelGGL((k_attn_split<KS, 1, FULL>), grid, block, 0, st, p);
}

template <int KS, bool FULL>
void rows(const AttnArgs &p, int rt, hipStream_t st) {
    const dim3 grid((unsigned)((int64_t)p.pieces * p.kv_heads), (unsigned)std::max(1, p.parts)), block(kAttnThreads);
    constexpr size_t lds = kRowsLds<KS>;
    if (rt == 1)
        hipLaunchKernelGGL((k_attn_rows<KS, 1, FULL>), grid, block, lds, st, p);
    else
        hipLaunchKernelGGL((k_attn_rows<KS, 2, FULL>), grid, block, lds, st, p);
}

}  // namespace

AttnPlan plan_attention(int64_t tokens, int seqs, int width, int kv_heads, int group, int dim) {
    AttnPlan plan = {};
    const int64_t all = tokens * group, mean = seqs ? (all + seqs - 1) / seqs : 0;  // rows of a head; of a sequence
    // Rows over the waves from more than 32 rows of a sequence on: 16 sequences of 4000 tokens, 52 rows each: 48 us (blocks over
    // the work-groups: 62); 30 sequences of 500 to 5000, 24 rows: 71 us (53). And where tables are short, or not long with a
    // work-group for each CU: a sequence is then done by one, and nothing is left to join. 8 heads of 128 on 32, one token of each of
    //   16 sequences, tables of 16 blocks 13.2 us (blocks over the work-groups: 15.9), of 32 blocks 15.7 (15.6);
    //   64 sequences, 16 blocks 16.6 (24.3), 64 blocks 34 (38), 128 blocks 57 (55); 256 sequences, 64 blocks 121 (131);
    //   six tokens, 24 rows, of 64 sequences, 32 blocks 44.6 (43.4).
    if (mean > 32 || width <= 16 || (width <= 64 && mean <= 16 && (int64_t)seqs * kv_heads >= 256)) {
        plan.rows = true;
        plan.rt = mean > 64 ? 2 : 1;
        plan.size = 64 * plan.rt;
        plan.pieces = all / plan.size + seqs;
        // Two work-groups a CU, the blocks in parts where the rows make fewer: 1024 rows over 8256 tokens in eight parts 58 us,
        // in one 190. But not less than 16 blocks a part: 4000 rows over 1000 tokens 31 us, in two parts 50.
        const int64_t groups = std::max<int64_t>(1, (all / plan.size + (seqs + 1) / 2) * kv_heads);
        const int64_t parts = mean > 32 ? std::min<int64_t>({512 / groups, (width + 15) / 16, 64}) : 1;
        plan.parts = parts > 1 ? (int)parts : 0;
        if (plan.parts) {
            const int64_t rows = (int64_t)kv_heads * plan.pieces * plan.parts * plan.size;
            plan.part_bytes = ((size_t)rows * dim * 4 + 255) / 256 * 256;
            plan.ml_bytes = (size_t)rows * 8;
        }
        return plan;
    }
    // Tiles of 16 rows, or, from 17 rows on, of 32, which read a block once for all of them, but in one work-group a CU from 65
    // columns on and with more than there are registers from 193 on. `reach`: the blocks of a share where every sequence is as long
    // as its row of the table and has one tile. Below: tables of so many blocks, 32 and 16 rows a tile, us.
    //   16 x 79 over 128 shares (9.9), 24 rows: 64 columns 18.6 and 16.8, 128 columns 28.2 and 21.7, 192 columns 38.8 and 34.0
    //   8 x 126 over 64 (15.8), 32 rows: 27.4 and 28.5, 42.9 and 35.9, 61 and 71;  16 x 126 (31.5): 38 and 44, 64 and 57, 102 and 95
    //   32 x 126 (63): 67 and 77, 119 and 169, 166 and 253;  256 columns: 64 x 126 158 and 121, 16 x 79 over 128 60 and 38
    const int64_t shares = std::max<int64_t>(1, 512 / kv_heads), reach = (int64_t)seqs * width / shares;
    const bool wide = mean > 16 && dim <= 192 && reach >= (dim > 64 && dim <= 128 ? 40 : 12);
    plan.rt = wide ? 2 : 1;
    plan.size = 16 * plan.rt;
    plan.pieces = all / plan.size + seqs;
    // Two work-groups a CU, not more than there can be blocks for.
    const int64_t most = std::max<int64_t>(1, (plan.pieces * (int64_t)width + kWaves - 1) / kWaves);
    plan.groups = (int)std::min<int64_t>(most, shares);
    const int64_t parts = (int64_t)kv_heads * plan.groups * 2 * plan.size;
    plan.part_bytes = ((size_t)parts * dim * 4 + 255) / 256 * 256;
    plan.ml_bytes = (size_t)parts * 8;
    return plan;
}

hipError_t launch_attention(const AttnArgs &a, void *ws, hipStream_t st) {
    AttnArgs p = a;
    const AttnPlan plan = plan_attention(p.seq.tokens, p.seq.seqs, p.seq.width, p.kv_heads, p.group, p.dim);
    p.pieces = (int)plan.pieces, p.groups = plan.groups, p.parts = plan.parts;
    p.per_group = p.group == 1 ? 0u : (uint32_t)(((uint64_t)1 << 32) / (uint32_t)p.group + 1u);
    p.part = static_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + plan.part_bytes);
    // The sizes most heads have, and forms for any other.
    auto run = [&](auto ks, auto full) {
        if (plan.rows)
            rows<ks.value, full.value>(p, plan.rt, st);
        else
            split<ks.value, full.value>(p, plan.rt, st);
    };
    using std::integral_constant;
    using Full = std::true_type;
    using Part = std::false_type;
    switch (p.dim) {
        case 64: run(integral_constant<int, 1>{}, Full{}); break;
        case 128: run(integral_constant<int, 2>{}, Full{}); break;
        case 256: run(integral_constant<int, 4>{}, Full{}); break;
        default:
            if (p.dim < 64) run(integral_constant<int, 1>{}, Part{});
            else if (p.dim < 128) run(integral_constant<int, 2>{}, Part{});
            else if (p.dim <= 192) run(integral_constant<int, 3>{}, Part{});
            else run(integral_constant<int, 4>{}, Part{});
    }
    if (plan.rows && !plan.parts) return hipGetLastError();
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int most = p.seq.starts ? plan.size : std::min(plan.size, p.group);  // rows of a tile
    // Many parts to a tile: a work-group each row (one sequence of 8000 tokens, 31 parts: 4.4 us, 10.6 with a wave a row); else
    // the rows' work is mostly finding their place (64 sequences, 0 to 16 parts: 6.4 us, 9.0 with a work-group a row).
    const unsigned pieces = (unsigned)((int64_t)p.pieces * p.kv_heads);
    if (p.groups >= 8 * (int64_t)p.pieces)
        hipLaunchKernelGGL(k_attn_join<true>, dim3(pieces, (unsigned)most), dim3(kAttnThreads), 0, st, p, plan.size);
    else
        hipLaunchKernelGGL(k_attn_join<false>, dim3(pieces, (unsigned)((most + kWaves - 1) / kWaves)), dim3(kAttnThreads), 0, st, p, plan.size);
    return hipGetLastError();
}

}  // namespace nvfp4
