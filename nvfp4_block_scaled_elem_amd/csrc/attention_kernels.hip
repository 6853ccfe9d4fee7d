// gfx950 attention over a paged cache in 8 bits.
//
// For a row (query token i of its sequence's last n, query head h of G to a key/value head) and the tokens t < limit that
// it sees (limit = len - n + i + 1, or len where every query sees every token):
//     s_t = scale (q . k_t),  o = sum_t e^(s_t) v_t / sum_t e^(s_t),  0 where the row sees none.
// q is bf16; k and v are E4M3 codes times a power of two per block of 64 tokens (cache.hpp), exact in bf16. Products
// on v_mfma_f32_16x16x32_bf16 with fp32 sums; maximum, sum and output are fp32, carried from block to block (one
// pass); a probability is rounded to bf16 for the second product, which takes bf16 (half a step, 2^-9 of a term,
// independent between terms: of the size of the output's own rounding), and not for the sum.
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

// What a wave carries for its 16 RT rows: per lane the maximum (of the row), the sum (of the lane's tokens), the output.
template <int KS, int RT>
struct Rows {
    f32x4 o[RT][4 * KS];
    float m[RT], l[RT];
    int lim[RT];  // tokens that the lane's row sees (0: no such row)
};

// KS: head sizes to 64 KS. RT: tiles of 16 rows. The wave takes blocks b0, b0 + step, ... below b1 of sequence s. `safe`:
// the tokens that every row of the wave sees (blocks below need no mask).
template <int KS, int RT>
__device__ __forceinline__ void attend(const AttnArgs &p, const Seq &q, int s, int64_t h, int b0, int b1, int step, int safe,
                                       const bf16x8 (&Q)[RT][2 * KS], Rows<KS, RT> &R) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int dim = p.dim;
    const int64_t page_bytes = (int64_t)kPage * dim;
    const int count = b1 > b0 ? (b1 - b0 + step - 1) / step : 0;
    if (count == 0) return;
    // byte offsets of the lane's pieces in a (page, head)
    const int koff = (16 * (r16 >> 2) + (r16 & 3)) * dim + 16 * g;  // + 4 t dim + 64 i
    const int voff = r16 * kPage + 16 * g;                          // + 1024 d
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
        return ((int64_t)max(pg, 0) * p.kv_heads + h) * page_bytes;
    };
    uint4 kc[4][KS], vc[4 * KS];
    auto load_k = [&](int64_t base) __attribute__((always_inline)) {
        const uint8_t *c = p.k_codes + base;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < KS; ++i)
                if (64 * i + 16 * g < dim) kc[t][i] = *reinterpret_cast<const uint4 *>(c + koff + 4 * t * dim + 64 * i);
    };
    auto load_v = [&](int64_t base) __attribute__((always_inline)) {
        const uint8_t *c = p.v_codes + base;
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d)
            if (16 * d < dim) vc[d] = *reinterpret_cast<const uint4 *>(c + voff + 1024 * d);
    };
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < KS; ++i) kc[t][i] = make_uint4(0u, 0u, 0u, 0u);  // columns past dim stay zeros
    look_up(0);
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
        if (!live) {
            load_k(next);
            load_v(next);
            continue;
        }
        const float kscale = mx_scale_value(ke), vscale = mx_scale_value(ve);
        f32x4 S[RT][4] = {};
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const bf16x8 a = operand8(kc[t][k].x, kc[t][k].y, kscale), b = operand8(kc[t][k].z, kc[t][k].w, kscale);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    S[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, Q[r][2 * k], S[r][t], 0, 0, 0);
                    S[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, Q[r][2 * k + 1], S[r][t], 0, 0, 0);
                }
            }
        load_k(next);
        const bool mask = t0 + kPage > safe;
        bool more = false;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float top = kNegInf;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v = S[r][t][j] * p.scale2;
                    if (mask) v = t0 + 16 * g + 4 * t + j < R.lim[r] ? v : kNegInf;
                    S[r][t][j] = v;
                    top = fmaxf(top, v);
                }
            more |= top > R.m[r] + 8.0f;
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
                const float w = weight(R.m[r], m);
                R.m[r] = m;
                R.l[r] *= w;
#pragma unroll
                for (int d = 0; d < 4 * KS; ++d) R.o[r][d] *= w;
            }
        }
        if (t0 + kPage > q.len) {  // codes behind the end may be any bytes
            const int n = q.len - t0 - 16 * g;
            uint32_t keep[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int k = n - 4 * w;
                keep[w] = k >= 4 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
            }
#pragma unroll
            for (int d = 0; d < 4 * KS; ++d) vc[d].x &= keep[0], vc[d].y &= keep[1], vc[d].z &= keep[2], vc[d].w &= keep[3];
        }
        bf16x8 P[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float m = R.m[r] == kNegInf ? 0.0f : R.m[r];
            uint32_t w[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float e[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    e[j] = __builtin_amdgcn_exp2f(S[r][t][j] - m);
                    R.l[r] += e[j];
                }
                w[2 * t] = pack_bf16(e[0], e[1]);
                w[2 * t + 1] = pack_bf16(e[2], e[3]);
            }
            P[r][0] = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
            P[r][1] = __builtin_bit_cast(bf16x8, u32x4{w[4], w[5], w[6], w[7]});
        }
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d)
            if (16 * d < dim) {
                const bf16x8 a = operand8(vc[d].x, vc[d].y, vscale), b = operand8(vc[d].z, vc[d].w, vscale);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    R.o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, P[r][0], R.o[r][d], 0, 0, 0);
                    R.o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, P[r][1], R.o[r][d], 0, 0, 0);
                }
            }
        load_v(next);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
        if (R.lim[r] > poison) R.l[r] = __builtin_nanf("");
}

// The lane's rows row0 + 16 r + l % 16 of the sequence: their queries as operands, and what they see. Returns the
// tokens that all of the wave's rows see.
template <int KS, int RT>
__device__ __forceinline__ int take_rows(const AttnArgs &p, const Seq &q, int64_t h, int row0, bf16x8 (&Q)[RT][2 * KS], Rows<KS, RT> &R) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    int safe = 0x7FFFFFFF;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = row0 + 16 * r + r16, tok = row / p.group, sub = row % p.group;
        const bool in = tok < q.n;
        R.lim[r] = !in ? 0 : p.causal ? min(max(q.len - q.n + tok + 1, 0), q.len) : q.len;
        if (in) safe = min(safe, R.lim[r]);
        const uint16_t *x = p.q + (int64_t)(q.first + tok) * p.qs + (h * p.group + sub) * p.qh;
#pragma unroll
        for (int k = 0; k < 2 * KS; ++k) {
            const int c = 64 * (k >> 1) + 16 * g + 8 * (k & 1);
            u32x4 v = {0u, 0u, 0u, 0u};
            if (in && c < p.dim) v = *reinterpret_cast<const u32x4_any *>(x + c);
            Q[r][k] = __builtin_bit_cast(bf16x8, v);
        }
        R.m[r] = kNegInf, R.l[r] = 0.0f;
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d) R.o[r][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) safe = min(safe, __shfl_xor(safe, k));
    return __builtin_amdgcn_readfirstlane(safe);
}

__device__ __forceinline__ uint16_t *out_row(const AttnArgs &p, const Seq &q, int64_t h, int row) {
    return p.out + ((int64_t)(q.first + row / p.group) * p.kv_heads * p.group + h * p.group + row % p.group) * p.dim;
}

// Rows over the waves: a work-group takes 64 RT rows of a sequence and head, a wave 16 RT of them, over all blocks that
// they see. For prompts: bound by the matrix cores and the exponentials. The waves read the same blocks at nearly
// the same time, mostly from the first-level cache.
template <int KS, int RT>
__global__ __launch_bounds__(kAttnThreads) void k_attn_rows(AttnArgs p) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kRows = 16 * RT * kWaves;
    // The heads run fastest over the grid, so that a head's blocks stay in one XCD's L2; the last pieces of a
    // sequence, which see the most, go first.
    const int64_t h = blockIdx.x % p.kv_heads;
    const int piece = p.pieces - 1 - (int)(blockIdx.x / p.kv_heads);
    const int s = piece_sequence(p.seq, piece, p.group, kRows, 1);
    const Seq q = sequence(p.seq, s);
    const int row0 = (piece - piece_base(p.seq, s, p.group, kRows, 1)) * kRows + 16 * RT * wave;
    if (row0 >= q.n * p.group || row0 < 0) return;
    bf16x8 Q[RT][2 * KS];
    Rows<KS, RT> R;
    const int safe = take_rows<KS, RT>(p, q, h, row0, Q, R);
    int most = 0;
#pragma unroll
    for (int r = 0; r < RT; ++r) most = max(most, R.lim[r]);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) most = max(most, __shfl_xor(most, k));
    most = __builtin_amdgcn_readfirstlane(most);
    attend<KS, RT>(p, q, s, h, 0, (most + kPage - 1) / kPage, 1, safe, Q, R);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const float l = row_sum(R.l[r]);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int row = row0 + 16 * r + r16;
        if (row >= q.n * p.group) continue;
        uint16_t *o = out_row(p, q, h, row) + 4 * g;
#pragma unroll
        for (int d = 0; d < 4 * KS; ++d)
            if (16 * d < p.dim) {
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
struct Share {
    uint32_t total, groups;  // blocks of the head's list; work-groups that share them
    __device__ __forceinline__ uint32_t begin(uint32_t j) const { return (uint32_t)((uint64_t)j * total / groups); }
    __device__ __forceinline__ uint32_t owner(uint32_t u) const { return (uint32_t)(((uint64_t)(u + 1) * groups - 1) / total); }
};

__device__ __forceinline__ int tiles_of(const AttnArgs &p, const Seq &q, int size) { return (q.n * p.group + size - 1) / size; }
__device__ __forceinline__ int blocks_of(const Seq &q) { return (q.len + kPage - 1) / kPage; }

// The list's length, and the sequence in whose part block `u` lies, with the part's begin. By whole waves.
__device__ __forceinline__ uint32_t list_total(const AttnArgs &p, int size) {
    const int lane = threadIdx.x & 63;
    uint32_t sum = 0u;
    for (int s = lane; s < p.seq.seqs; s += 64) {
        const Seq q = sequence(p.seq, s);
        sum += (uint32_t)(tiles_of(p, q, size) * blocks_of(q));
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) sum += (uint32_t)__shfl_xor((int)sum, k);
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)sum);
}

__device__ __forceinline__ int list_find(const AttnArgs &p, int size, uint32_t u, uint32_t &begin) {
    const int lane = threadIdx.x & 63;
    uint32_t before = 0u;
    for (int s0 = 0; s0 < p.seq.seqs; s0 += 64) {
        uint32_t mine = 0u;
        if (s0 + lane < p.seq.seqs) {
            const Seq q = sequence(p.seq, s0 + lane);
            mine = (uint32_t)(tiles_of(p, q, size) * blocks_of(q));
        }
        uint32_t upto = mine;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) {
            const uint32_t v = (uint32_t)__shfl_up((int)upto, k);
            if (lane >= k) upto += v;
        }
        const uint64_t past = __ballot(before + upto > u);
        if (past) {
            const int first = __ffsll((unsigned long long)past) - 1;
            begin = before + (uint32_t)__builtin_amdgcn_readlane((int)(upto - mine), first);
            return s0 + first;
        }
        before += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    }
    begin = before;
    return p.seq.seqs;
}

__device__ __forceinline__ Share share_of(const AttnArgs &p, int size) {
    Share sh;
    sh.total = list_total(p, size);
    // Not less than a block for each wave of a work-group.
    sh.groups = max(1u, min((uint32_t)p.groups, (sh.total + kWaves - 1) / kWaves));
    return sh;
}

// Where a tile's part of share j lies: the numbers j + piece ascend along the list.
__device__ __forceinline__ int64_t part_place(const AttnArgs &p, int64_t h, uint32_t j, int piece) {
    return h * (p.groups + p.pieces) + j + piece;
}

template <int KS, int RT>
__global__ __launch_bounds__(kAttnThreads) void k_attn_split(AttnArgs p) {
    constexpr int kRows = 16 * RT, kDim = 64 * KS;
    __shared__ float lds_o[kWaves][16][kDim + 4];
    __shared__ float lds_m[kWaves][16], lds_l[kWaves][16];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t h = blockIdx.x % p.kv_heads;
    const uint32_t j = blockIdx.x / p.kv_heads;
    const Share sh = share_of(p, kRows);
    if (j >= sh.groups || sh.total == 0u) return;
    uint32_t u = sh.begin(j);
    const uint32_t end = sh.begin(j + 1);
    if (u >= end) return;
    uint32_t at;
    int s = list_find(p, kRows, u, at);
    while (u < end && s < p.seq.seqs) {
        const Seq q = sequence(p.seq, s);
        const uint32_t nb = (uint32_t)blocks_of(q), mine = nb * (uint32_t)tiles_of(p, q, kRows);
        if (u >= at + mine) {
            at += mine;
            ++s;
            continue;
        }
        const int tile = (int)((u - at) / nb), b0 = (int)((u - at) % nb), b1 = (int)min(nb, b0 + (end - u));
        u += b1 - b0;
        const int row0 = tile * kRows, rows = min(kRows, q.n * p.group - row0);
        bf16x8 Q[RT][2 * KS];
        Rows<KS, RT> R;
        const int safe = take_rows<KS, RT>(p, q, h, row0, Q, R);
        attend<KS, RT>(p, q, s, h, b0 + wave, b1, kWaves, safe, Q, R);
        const bool whole = b0 == 0 && b1 == (int)nb;
        const int64_t place = part_place(p, h, j, piece_base(p.seq, s, p.group, kRows, 1) + tile);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float l = row_sum(R.l[r]);
            if (16 * r >= rows) break;
            __syncthreads();  // the tile before has been read
            if (g == 0) lds_m[wave][r16] = R.m[r], lds_l[wave][r16] = l;
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
                float *po = p.part + (place * kRows + 16 * r + row) * p.dim;
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
                    float *ml = p.part_ml + (place * kRows + 16 * r + row) * 2;
                    ml[0] = m, ml[1] = sum;
                }
            }
        }
        __syncthreads();  // LDS is free for the next piece
    }
}

// The tiles whose blocks lie in several shares, and the rows of sequences of no tokens (zeros): a wave takes a row.
__global__ __launch_bounds__(kAttnThreads) void k_attn_join(AttnArgs p, int size) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t h = blockIdx.x % p.kv_heads;
    const int piece = (int)(blockIdx.x / p.kv_heads);
    const int s = piece_sequence(p.seq, piece, p.group, size, 1);
    const Seq q = sequence(p.seq, s);
    const int base = piece_base(p.seq, s, p.group, size, 1), tile = piece - base;
    const int row = (int)blockIdx.y * kWaves + wave;  // of the tile
    if (tile < 0 || tile >= tiles_of(p, q, size) || row >= size || tile * size + row >= q.n * p.group) return;
    uint16_t *o = out_row(p, q, h, tile * size + row);
    const int c = 4 * lane;
    const uint32_t nb = (uint32_t)blocks_of(q);
    if (nb == 0u) {
        if (c < p.dim) *reinterpret_cast<uint2 *>(o + c) = make_uint2(0u, 0u);
        return;
    }
    const Share sh = share_of(p, size);
    uint32_t before = 0u;  // blocks of the sequences before s
    for (int i = lane; i < s; i += 64) {
        const Seq e = sequence(p.seq, i);
        before += (uint32_t)(tiles_of(p, e, size) * blocks_of(e));
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) before += (uint32_t)__shfl_xor((int)before, k);
    before = (uint32_t)__builtin_amdgcn_readfirstlane((int)before);
    const uint32_t u0 = before + (uint32_t)tile * nb;
    const uint32_t j0 = sh.owner(u0), j1 = sh.owner(u0 + nb - 1);
    if (j0 == j1) return;
    const int64_t at = part_place(p, h, j0, piece) * size + row;
    float m = kNegInf;
    for (uint32_t j = j0 + lane; j <= j1; j += 64) m = fmaxf(m, p.part_ml[(at + (int64_t)(j - j0) * size) * 2]);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k));
    float sum = 0.0f;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    const int parts = (int)(j1 - j0 + 1);
#pragma unroll 8
    for (int k = 0; k < parts; ++k) {
        const int64_t e = at + (int64_t)k * size;
        const float w = weight(p.part_ml[2 * e], m), l = p.part_ml[2 * e + 1];
        sum += l == 0.0f ? 0.0f : w * l;
        if (c < p.dim) v += *reinterpret_cast<const f32x4 *>(p.part + e * p.dim + c) * w;
    }
    v *= sum == 0.0f ? 0.0f : 1.0f / sum;
    if (c < p.dim) *reinterpret_cast<uint2 *>(o + c) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

template <int KS>
void split(const AttnArgs &p, int rt, hipStream_t st) {
    const dim3 grid((unsigned)(p.groups * p.kv_heads)), block(kAttnThreads);
    if constexpr (KS <= 2)
        if (rt == 4) {
            hipLaunchKernelGGL((k_attn_split<KS, 4>), grid, block, 0, st, p);
            return;
        }
    if (rt >= 2)
        hipLaunchKernelGGL((k_attn_split<KS, 2>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((k_attn_split<KS, 1>), grid, block, 0, st, p);
}

template <int KS>
void rows(const AttnArgs &p, hipStream_t st) {
    const dim3 grid((unsigned)((int64_t)p.pieces * p.kv_heads)), block(kAttnThreads);
    if constexpr (KS <= 2)
        hipLaunchKernelGGL((k_attn_rows<KS, 2>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((k_attn_rows<KS, 1>), grid, block, 0, st, p);
}

int rows_tiles(int ks) { return ks <= 2 ? 2 : 1; }

}  // namespace

AttnPlan plan_attention(int64_t tokens, int seqs, int width, int kv_heads, int group, int dim) {
    AttnPlan plan = {};
    const int ks = (dim + 63) / 64;
    const int64_t all = tokens * group, mean = seqs ? (all + seqs - 1) / seqs : 0;  // rows of a head; of a sequence
    const int big = 64 * rows_tiles(ks);
    // Rows over the waves where that makes work for the whole GPU, else blocks over the work-groups.
    if (mean > 64 && (all / big) * kv_heads >= 512) {
        plan.rows = true;
        plan.size = big;
        plan.pieces = all / big + seqs;
        return plan;
    }
    const int rt = mean <= 16 ? 1 : mean <= 32 || ks > 2 ? 2 : 4;
    plan.rt = rt;
    plan.size = 16 * rt;
    plan.pieces = all / plan.size + seqs;
    // Two work-groups a CU, not more than there can be blocks for.
    const int64_t most = std::max<int64_t>(1, (plan.pieces * (int64_t)width + kWaves - 1) / kWaves);
    plan.groups = (int)std::min<int64_t>(most, std::max<int64_t>(1, 512 / kv_heads));
    const int64_t parts = (int64_t)kv_heads * (plan.groups + plan.pieces) * plan.size;
    plan.part_bytes = ((size_t)parts * dim * 4 + 255) / 256 * 256;
    plan.ml_bytes = (size_t)parts * 8;
    return plan;
}

hipError_t launch_attention(const AttnArgs &a, void *ws, hipStream_t st) {
    AttnArgs p = a;
    const AttnPlan plan = plan_attention(p.seq.tokens, p.seq.seqs, p.seq.width, p.kv_heads, p.group, p.dim);
    p.pieces = (int)plan.pieces, p.groups = plan.groups;
    p.part = static_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + plan.part_bytes);
    const int ks = (p.dim + 63) / 64;
    if (plan.rows) {
        ks == 1 ? rows<1>(p, st) : ks == 2 ? rows<2>(p, st) : ks == 3 ? rows<3>(p, st) : rows<4>(p, st);
        return hipGetLastError();
    }
    ks == 1 ? split<1>(p, plan.rt, st) : ks == 2 ? split<2>(p, plan.rt, st) : ks == 3 ? split<3>(p, plan.rt, st) : split<4>(p, plan.rt, st);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int most = p.seq.starts ? plan.size : std::min(plan.size, p.group);  // rows of a tile
    const dim3 grid((unsigned)((int64_t)p.pieces * p.kv_heads), (unsigned)((most + kWaves - 1) / kWaves));
    hipLaunchKernelGGL(k_attn_join, grid, dim3(kAttnThreads), 0, st, p, plan.size);
    return hipGetLastError();
}

}  // namespace nvfp4
