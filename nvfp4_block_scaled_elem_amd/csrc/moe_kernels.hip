// gfx950 layer of experts with NVFP4 weights, for a few tokens.
//
// For token t with logits l[t][0..E-1]: its top_k largest logits choose experts (equal ones by the lower index; -inf
// never), weighted by p = softmax(l) over all experts or the logistic function s(l), divided by their sum where
// they are normalised:
//     y[t] = residual[t] + sum_j w_j alpha2_e (W2_e h_j),  h_j = act(alpha1_e W1_e x_t)
// (gated: act of the first `inner` rows of W1_e x times the others). Weights are those of the product kernels, e2m1(code)
// e4m3(scale), exact in bf16; x is bf16; sums are fp32 on the matrix cores; h is rounded to bf16, which the second
// product takes (its error, at most 2^-8 of a term and independent between terms, is of the size of y's own rounding: together
// 0.0023 of y's norm, y's own 0.0017), or, for few tokens, kept in two bf16 parts.
//
// Bound by reading the chosen experts' weights, each once however many tokens chose it; a pair is a token and one of its
// choices, and the pairs of an expert are the columns of v_mfma_f32_16x16x32_bf16, 16 at a time.
//   k_moe_route: experts and weights of each token; to eight tokens the first product finds them itself.
//   first product: k_moe_product (a work-group has 16 weight rows, its waves split the sum) where there is little work,
//     else k_moe_rows (a wave has 32 weight rows);
//   second product: k_moe_down, the weighted sum over the experts in it, to 16 tokens and little work; else k_moe_rows or
//     k_moe_product, and k_moe_sum.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "act.hpp"
#include "codec.hpp"
#include "launch.hpp"
#include "mx.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;
// To so many tokens are routed inside the first product (12 tokens, 8 of 128 experts: the layer 76 us so, 68 with the kernel apart).
constexpr int kRouteTokens = 8;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------------------------------- routing

// A logit's place in the order: larger is first, 0 (-inf) never; NaN before all numbers, so that it is chosen and
// shows. -0 is 0.
__device__ __forceinline__ uint32_t order_key(float l) {
    if (l == -__builtin_inff()) return 0u;
    const uint32_t b = __float_as_uint(l + 0.0f);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Reductions over a wave within its rows of 16 lanes and across them (row_shr 1, 2, 4, 8, row_bcast 15, 31; a lane without a
// source keeps `old`); lane 63 has the result.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t old, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, moved<0x111>(v, v));
    v = max(v, moved<0x112>(v, v));
    v = max(v, moved<0x114>(v, v));
    v = max(v, moved<0x118>(v, v));
    v = max(v, moved<0x142>(v, v));
    v = max(v, moved<0x143>(v, v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// The experts of token t, by one wave: lane j < top_k gets choice j (-1: none) and its weight. Lane l holds the logits
// l, l + 64, ... (R of them). `most`: choices to make (the weights are right if all top_k are).
template <int R>
__device__ __forceinline__ void route_of(const MoeArgs &p, int64_t t, int most, int &id, float &w) {
    const int lane = threadIdx.x & 63;
    float l[R];
    uint32_t key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = lane + 64 * r;
        l[r] = -__builtin_inff();
        if (e < p.experts)
            l[r] = p.logits_f32 ? static_cast<const float *>(p.logits)[t * p.ldl + e]
                                : __uint_as_float((uint32_t)static_cast<const uint16_t *>(p.logits)[t * p.ldl + e] << 16);
        key[r] = order_key(l[r]);
    }
    float all = 0.0f, top = 0.0f;
    if (!p.sigmoid) {
        uint32_t k = 0u;
#pragma unroll
        for (int r = 0; r < R; ++r) k = max(k, key[r]);
        k = wave_max(k);
        top = k == 0xFFFFFFFFu ? __builtin_nanf("") : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
        if (!p.normalize) {
#pragma unroll
            for (int r = 0; r < R; ++r) all += key[r] ? __builtin_amdgcn_exp2f((l[r] - top) * kLog2e) : 0.0f;
            all = wave_sum(all);
        }
    }
    id = -1;
    float mine = 0.0f;
    for (int j = 0; j < most; ++j) {
        uint32_t k = 0u;
#pragma unroll
        for (int r = 0; r < R; ++r) k = max(k, key[r]);
        k = wave_max(k);
        if (k == 0u) break;
        bool found = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {  // the lowest index: e = lane + 64 r
            const uint64_t who = __ballot(key[r] == k);
            if (!found && who) {
                found = true;
                const int first = __ffsll((unsigned long long)who) - 1;
                const float v = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(l[r]), first));
                if (lane == j) id = 64 * r + first, mine = v;
                if (lane == first) key[r] = 0u;
            }
        }
    }
    // softmax: e^(l - top); logistic function: e^min(l, 0) / (1 + e^-|l|), against the largest where they are normalised
    // (all of them may be below the smallest number).
    float e = 0.0f;
    if (!p.sigmoid) {
        e = id >= 0 ? __builtin_amdgcn_exp2f((mine - top) * kLog2e) : 0.0f;
    } else {
        float m = 0.0f;
        if (p.normalize) {
            // the largest of numbers up to 0: the least of their patterns without the sign (of no number: 0x7F800000)
            const uint32_t low = wave_max(id >= 0 ? 0x7F800000u - (__float_as_uint(fminf(mine, 0.0f)) & 0x7FFFFFFFu) : 0u);
            m = low == 0u ? 0.0f : -__uint_as_float(0x7F800000u - low);
        }
        const float low = mine < 0.0f ? mine : 0.0f;
        e = id >= 0 ? __builtin_amdgcn_exp2f((low - m) * kLog2e) / (1.0f + __builtin_amdgcn_exp2f(-fabsf(mine) * kLog2e)) : 0.0f;
    }
    if (p.normalize) all = wave_sum(e);
    w = p.normalize || !p.sigmoid ? e / all : e;
}

__device__ __forceinline__ void route(const MoeArgs &p, int64_t t, int most, int &id, float &w) {
    if (p.experts <= 64)
        route_of<1>(p, t, most, id, w);
    else if (p.experts <= 128)
        route_of<2>(p, t, most, id, w);
    else if (p.experts <= 256)
        route_of<4>(p, t, most, id, w);
    else
        route_of<kMoeMaxExperts / 64>(p, t, most, id, w);
}

__global__ __launch_bounds__(256) void k_moe_route(MoeArgs p) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= p.tokens) return;
    int id;
    float w;
    route(p, t, p.top_k, id, w);
    if (lane < p.top_k) p.ids[t * p.top_k + lane] = id, p.weights[t * p.top_k + lane] = w;
}

// ------------------------------------------------------------------------------------------- products

constexpr int kChunk = 128, kChunkLds = 16 * 64 + 16 * 8;  // k per chunk; LDS bytes of 16 rows' codes and scales

// What rounding v to `hi` left; nothing of an infinity.
__device__ __forceinline__ float rest_of(float v, float hi) {
    return fabsf(hi) == __builtin_inff() ? 0.0f : v - hi;
}

// 16-byte piece q (0..3) of row r of a chunk's codes in LDS: the 16 lanes that read one q of 16 rows meet no bank twice.
__device__ __forceinline__ int code_place(int r, int q) { return r * 64 + ((q ^ ((r >> 2) & 3)) << 4); }

// A work-group's pairs, by all of it: the chosen experts in order, each as often as its pairs make groups of SIZE, are a list;
// find() takes its entry `nth` (expert -1: there are not so many), fill() puts the entry's pairs into `list`, in their
// order, so that the entries of an expert share its pairs without a word between them. An expert that many tokens chose is then
// several work-groups' work, not several turns of one (150 tokens, 128 experts of 2048 x 768, four of them chosen by all tokens:
// 126 us, 260 in turns; where all are as likely 111 and 109). A thread's ids are loaded at once and kept: one by one, 1200 of
// them took 8 us of a work-group's time.
template <int THREADS, int SIZE>
struct Pick {
    static constexpr int kMine = 8, kWavesHere = THREADS / 64;
    struct Lds {
        int pairs[kMoeMaxExperts];
        int matches[kMine * kWavesHere];
        uint16_t list[SIZE];
    };
    int id[kMine];
    int expert, first, n;  // the entry's expert, and its pairs first .. first + n - 1
    __device__ __forceinline__ void load(const int *ids, int i0, int pairs) {
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int i = i0 + THREADS * u + threadIdx.x;
            id[u] = i < pairs ? ids[i] : -1;
        }
    }
    __device__ __forceinline__ void find(const MoeArgs &p, const int *ids, int nth, Lds &lds) {
        const int tid = threadIdx.x, lane = tid & 63, pairs = (int)p.tokens * p.top_k;
        if (p.tokens == 1) {  // its choices are all different
            expert = ids[nth], first = 0, n = 1;
            return;
        }
        load(ids, 0, pairs);
        for (int e = tid; e < p.experts; e += THREADS) lds.pairs[e] = 0;
        __syncthreads();
        for (int i0 = 0;;) {
#pragma unroll
            for (int u = 0; u < kMine; ++u)
                if (id[u] >= 0) atomicAdd(&lds.pairs[id[u]], 1);
            i0 += THREADS * kMine;
            if (i0 >= pairs) break;
            load(ids, i0, pairs);
        }
        __syncthreads();
        int before = 0;
        expert = -1;
        for (int e0 = 0; e0 < p.experts; e0 += 64) {
            const int count = e0 + lane < p.experts ? lds.pairs[e0 + lane] : 0, entries = (count + SIZE - 1) / SIZE;
            const int upto = sums_to(entries);
            const uint64_t past = __ballot(before + upto > nth);
            if (past) {
                const int at = __ffsll((unsigned long long)past) - 1;
                expert = e0 + at;
                first = (nth - before - __builtin_amdgcn_readlane(upto - entries, at)) * SIZE;
                n = min(SIZE, __builtin_amdgcn_readlane(count, at) - first);
                return;
            }
            before += __builtin_amdgcn_readlane(upto, 63);
        }
    }
    __device__ __forceinline__ void fill(const MoeArgs &p, const int *ids, int nth, Lds &lds) {
        const int tid = threadIdx.x, lane = tid & 63, pairs = (int)p.tokens * p.top_k;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        if (p.tokens == 1) {
            if (tid == 0) lds.list[0] = (uint16_t)nth;
            lds_barrier();
            return;
        }
        if (pairs > THREADS * kMine) load(ids, 0, pairs);
        int before = 0;  // the expert's pairs in front of i0
        for (int i0 = 0;;) {
            uint64_t who[kMine];
#pragma unroll
            for (int u = 0; u < kMine; ++u) {
                who[u] = __ballot(id[u] == expert);
                if (lane == 0) lds.matches[u * kWavesHere + wave] = __popcll(who[u]);
            }
            lds_barrier();
            const int mine = lane < kMine * kWavesHere ? lds.matches[lane] : 0, upto = sums_to(mine);
#pragma unroll
            for (int u = 0; u < kMine; ++u) {
                const int at = before - first + __builtin_amdgcn_readlane(upto - mine, u * kWavesHere + wave) +
                               __popcll(who[u] & (((uint64_t)1 << lane) - 1));
                if (id[u] == expert && at >= 0 && at < SIZE) lds.list[at] = (uint16_t)(i0 + THREADS * u + tid);
            }
            lds_barrier();
            before += __builtin_amdgcn_readlane(upto, 63);
            i0 += THREADS * kMine;
            if (i0 >= pairs) break;
            load(ids, i0, pairs);
        }
    }
};

// The experts of a few tokens into `ids` (LDS), a wave a token at a time, by every work-group for itself: a launch saved. The
// first one writes them down for the kernels after it.
template <int WAVES>
__device__ __forceinline__ void route_here(const MoeArgs &p, int most, bool write, int *ids) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int t = wave; t < (int)p.tokens; t += WAVES) {
        int id;
        float w;
        route(p, t, most, id, w);
        if (lane < p.top_k) {
            ids[t * p.top_k + lane] = id;
            if (write) p.ids[t * p.top_k + lane] = id, p.weights[t * p.top_k + lane] = w;
        }
    }
    __syncthreads();
}

// NT: 2 if gated. SECOND: the product with W2, else with W1. ROUTE: to eight tokens, whose experts are found here.
template <int NT, bool SECOND, bool ROUTE>
__global__ __launch_bounds__(kThreads) void k_moe_product(MoeArgs p, int tiles) {
    constexpr int kStage = kWaves * NT * kChunkLds, kSums = kWaves * NT * 1024;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kStage > kSums ? kStage : kSums];
    __shared__ typename Pick<kThreads, 16>::Lds pick_lds;
    uint16_t *const list = pick_lds.list;
    __shared__ int route_ids[ROUTE ? kRouteTokens * kMoeMaxTopK : 1];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // (one token: this work-group's expert is choice blockIdx.x / tiles, and those after it are not needed)
    if (ROUTE) route_here<kWaves>(p, p.tokens == 1 && blockIdx.x ? (int)blockIdx.x / tiles + 1 : p.top_k, blockIdx.x == 0, route_ids);
    const int *const ids = ROUTE ? route_ids : p.ids;
    Pick<kThreads, 16> pick;
    pick.find(p, ids, blockIdx.x / tiles, pick_lds);
    const int expert = pick.expert, pairs = pick.n;
    if (expert < 0) return;
    pick.fill(p, ids, blockIdx.x / tiles, pick_lds);
    const int64_t K = SECOND ? p.inner : p.width, F = SECOND ? p.width : p.inner;
    const int64_t f0 = (int64_t)(blockIdx.x % tiles) * 16, nch = (K + kChunk - 1) / kChunk;
    const MoeWeights &W = SECOND ? p.down : p.up;
    const uint8_t *codes = W.codes + expert * (NT * F * (K / 2)), *scales = W.scales + expert * (NT * F * (K / 16));
    const float alpha = W.alpha[expert];
    const uint16_t *x = SECOND ? p.h : static_cast<const uint16_t *>(p.x);
    const int64_t ldx = SECOND ? p.inner : p.ldx;
    uint8_t *const wl = lds + wave * NT * kChunkLds;
    const int64_t crow = min(F - 1, f0 + (lane >> 2)), srow = min(F - 1, f0 + r16);
    {
        const int pair = r16 < pairs ? list[r16] : -1;
        const uint16_t *xr = x + (int64_t)(SECOND ? max(pair, 0) : max(pair, 0) / p.top_k) * ldx;
        f32x4 acc[NT] = {};
        uint4 cv[NT];
        uint2 sv[NT];
        auto load_w = [&](int64_t ch) __attribute__((always_inline)) {
            const int64_t kc = kChunk * ch + 32 * (lane & 3), ks = kChunk * ch;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint8_t *c = codes + ((crow + j * F) * K + kc) / 2, *s = scales + ((srow + j * F) * K + ks) / 16;
                cv[j] = make_uint4(0u, 0u, 0u, 0u);
                sv[j] = make_uint2(0u, 0u);
                if (kc + 32 <= K) {
                    cv[j] = load16(c);
                } else if (kc < K) {  // the row's last 16
                    const uint2 d = load8b(c);
                    cv[j].x = d.x, cv[j].y = d.y;
                }
                if (lane >= 16) continue;
                if (ks + kChunk <= K) {
                    sv[j] = load8b(s);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (ks + 16 * e < K) (e < 4 ? sv[j].x : sv[j].y) |= (uint32_t)s[e] << (8 * (e & 3));
                }
            }
        };
        int64_t ch = wave;
        if (ch < nch) load_w(ch);
#pragma unroll 1
        for (; ch < nch; ch += kWaves) {
            const int64_t k = kChunk * ch + 32 * g;
            uint4 xv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xv[i] = make_uint4(0u, 0u, 0u, 0u);
                if (pair >= 0 && k + 8 * i < K) xv[i] = load16(xr + k + 8 * i);
            }
            wave_handover();
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint8_t *const q = wl + j * kChunkLds;
                *reinterpret_cast<uint4 *>(q + code_place(lane >> 2, lane & 3)) = cv[j];
                if (lane < 16) *reinterpret_cast<uint2 *>(q + 1024 + 8 * lane) = sv[j];
            }
            wave_handover();
            if (ch + kWaves < nch) load_w(ch + kWaves);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint8_t *const q = wl + j * kChunkLds;
                const uint4 cur = *reinterpret_cast<const uint4 *>(q + code_place(r16, g));
                const uint32_t sb = *reinterpret_cast<const u16_lds *>(q + 1024 + 8 * r16 + 2 * g);
                const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)(sb & 0x7F7Fu), false);  // both scales
                const uint4 w[4] = {dequant8(cur.x, d.x), dequant8(cur.y, d.x), dequant8(cur.z, d.y), dequant8(cur.w, d.y)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[i]),
                                                                     __builtin_bit_cast(bf16x8, xv[i]), acc[j], 0, 0, 0);
            }
        }
        __syncthreads();  // the sums take the place of the codes
        float *const red = reinterpret_cast<float *>(lds);
#pragma unroll
        for (int j = 0; j < NT; ++j) *reinterpret_cast<f32x4 *>(&red[(wave * NT + j) * 256 + lane * 4]) = acc[j];
        __syncthreads();
        // Element r of lane l is weight row 4 (l / 16) + r of the tile, pair l % 16 of the list's sixteen.
        if (tid < 256) {
            float z[NT] = {};
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
#pragma unroll
                for (int j = 0; j < NT; ++j) z[j] += red[(w * NT + j) * 256 + tid];
            const int l = tid >> 2;
            const int64_t f = f0 + 4 * (l >> 4) + (tid & 3);
            if (f < F && (l & 15) < pairs) {
                const int q = list[l & 15];
                if (SECOND) {
                    p.z[q * F + f] = p.weights[q] * (alpha * z[0]);
                } else {
                    float a = act_value(alpha * z[0], p.act);
                    if (NT == 2) a *= alpha * z[NT - 1];
                    const uint16_t hi = to_bf16(a);
                    p.h[q * F + f] = hi;
                    if (p.h_low) p.h_low[q * F + f] = to_bf16(rest_of(a, __uint_as_float((uint32_t)hi << 16)));
                }
            }
        }
    }
}

// The second product and the sum over a token's experts together, to 16 tokens: column t of an operand is token t (zeros
// where it did not choose the expert), so that the tokens' sums stay in place from expert to expert. A work-group has 16 rows of y;
// its sixteen waves share the list (chosen expert, chunk of 128 k) in equal runs and are joined in wave order. h comes in
// two bf16 parts, its rounding and what that leaves (2^-17 of h together): the matrix cores are idle anyway.
constexpr int kDownWaves = 16, kDownThreads = 64 * kDownWaves, kDownTokens = 16;

__global__ __launch_bounds__(kDownThreads) void k_moe_down(MoeArgs p) {
    constexpr int kStage = kDownWaves * kChunkLds, kSums = kDownWaves * 1024;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kStage > kSums ? kStage : kSums];
    __shared__ uint8_t seen[kMoeMaxExperts];
    __shared__ uint16_t chosen[kMoeMaxExperts];            // the experts in order
    __shared__ __attribute__((aligned(16))) uint8_t choice[kMoeMaxExperts][kDownTokens];  // of expert e by token t: 1 + j, 0 if not
    __shared__ int number;
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pairs = (int)p.tokens * p.top_k;
    const int64_t K = p.inner, F = p.width;
    if (p.tokens == 1) {  // its choices are all different
        if (wave == 0) {
            const int e = lane < p.top_k ? p.ids[lane] : -1;
            if (e >= 0) {
                chosen[lane] = (uint16_t)e;
                *reinterpret_cast<u32x4 *>(choice[e]) = u32x4{1u + (uint32_t)lane, 0u, 0u, 0u};
            }
            const int n = __popcll(__ballot(e >= 0));
            if (lane == 0) number = n;
        }
        __syncthreads();
    } else {
        for (int e = tid; e < p.experts; e += kDownThreads) {
            seen[e] = 0;
            *reinterpret_cast<u32x4 *>(choice[e]) = u32x4{0u, 0u, 0u, 0u};
        }
        __syncthreads();
        for (int i = tid; i < pairs; i += kDownThreads) {
            const int e = p.ids[i];
            if (e >= 0) seen[e] = 1, choice[e][i / p.top_k] = (uint8_t)(1 + i % p.top_k);
        }
        __syncthreads();
        if (wave == 0) {
            int before = 0;
            for (int e0 = 0; e0 < p.experts; e0 += 64) {
                const bool in = e0 + lane < p.experts && seen[e0 + lane];
                const uint64_t who = __ballot(in);
                if (in) chosen[before + __popcll(who & (((uint64_t)1 << lane) - 1))] = (uint16_t)(e0 + lane);
                before += __popcll(who);
            }
            if (lane == 0) number = before;
        }
        __syncthreads();
    }
    const int nch = (int)((K + kChunk - 1) / kChunk), items = number * nch;
    const int lo = (int)((int64_t)items * wave / kDownWaves), hi = (int)((int64_t)items * (wave + 1) / kDownWaves);
    const int64_t f0 = (int64_t)blockIdx.x * 16;
    uint8_t *const wl = lds + wave * kChunkLds;
    struct Item {
        u32x4 c, h[4], l[4];
        u32x2 s;
        float w;
        int choice;
    };
    auto load = [&](Item &it, int i) __attribute__((always_inline)) {
        const int e = __builtin_amdgcn_readfirstlane((int)chosen[i / nch]), ch = i % nch;
        const int64_t row = (int64_t)e * F + f0;
        const int kc = kChunk * ch + 32 * (lane & 3), ks = kChunk * ch;
        const uint8_t *c = p.down.codes + ((row + (lane >> 2)) * K + kc) / 2, *s = p.down.scales + ((row + r16) * K + ks) / 16;
        it.c = u32x4{0u, 0u, 0u, 0u};
        it.s = u32x2{0u, 0u};
        if (kc + 32 <= K) {
            it.c = *reinterpret_cast<const u32x4_any *>(c);
        } else if (kc < K) {  // the row's last 16
            const u32x2 d = *reinterpret_cast<const u32x2_any *>(c);
            it.c = u32x4{d.x, d.y, 0u, 0u};
        }
        if (lane < 16) {
            if (ks + kChunk <= K) {
                it.s = *reinterpret_cast<const u32x2_any *>(s);
            } else {
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (ks + 16 * b < K) it.s[b >> 2] |= (uint32_t)s[b] << (8 * (b & 3));
            }
        }
        const int j = it.choice = choice[e][r16];
        it.w = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) it.h[k] = it.l[k] = u32x4{0u, 0u, 0u, 0u};
        if (j) {
            const int64_t pair = r16 * p.top_k + j - 1;
            it.w = p.weights[pair] * p.down.alpha[e];
            const int64_t at = pair * K + kChunk * ch + 32 * g;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (kChunk * ch + 32 * g + 8 * k < K) {
                    it.h[k] = *reinterpret_cast<const u32x4 *>(p.h + at + 8 * k);
                    it.l[k] = *reinterpret_cast<const u32x4 *>(p.h_low + at + 8 * k);
                }
        }
    };
    f32x4 total = {0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Item &it) __attribute__((always_inline)) {
        wave_handover();
        *reinterpret_cast<u32x4 *>(wl + code_place(lane >> 2, lane & 3)) = it.c;
        if (lane < 16) *reinterpret_cast<u32x2 *>(wl + 1024 + 8 * lane) = it.s;
        wave_handover();
        const u32x4 cur = *reinterpret_cast<const u32x4 *>(wl + code_place(r16, g));
        const uint32_t sb = *reinterpret_cast<const u16_lds *>(wl + 1024 + 8 * r16 + 2 * g);
        const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)(sb & 0x7F7Fu), false);  // both scales
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bf16x8 w = __builtin_bit_cast(bf16x8, dequant8(cur[k], k < 2 ? d.x : d.y));
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, it.h[k]), acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, it.l[k]), acc, 0, 0, 0);
        }
        // a token that did not choose the expert has zeros, and NaN where the expert's scales are NaN: not taken
#pragma unroll
        for (int k = 0; k < 4; ++k) total[k] = it.choice ? __builtin_fmaf(acc[k], it.w, total[k]) : total[k];
    };
    Item a, b;
    int i = lo;
    if (i < hi) load(a, i);
#pragma unroll 1
    for (; i < hi; i += 2) {
        if (i + 1 < hi) load(b, i + 1);
        multiply(a);
        if (i + 1 >= hi) break;
        if (i + 2 < hi) load(a, i + 2);
        multiply(b);
    }
    __syncthreads();  // the sums take the place of the codes
    float *const red = reinterpret_cast<float *>(lds);
    *reinterpret_cast<f32x4 *>(&red[wave * 256 + lane * 4]) = total;
    __syncthreads();
    if (tid < 256) {
        // Element r of lane l is row 4 (l / 16) + r, token l % 16.
        const int l = tid >> 2, t = l & 15;
        const int64_t f = f0 + 4 * (l >> 4) + (tid & 3);
        if (t < p.tokens) {
            float y = p.res ? __uint_as_float((uint32_t)p.res[t * p.ldr + f] << 16) : 0.0f;
#pragma unroll
            for (int w = 0; w < kDownWaves; ++w) y += red[w * 256 + tid];
            p.y[t * F + f] = to_bf16(y);
        }
    }
}

// Many rows: a wave owns 32 weight rows (gated: 16 gate rows and their 16 up rows) over the whole sum, and a work-group's
// four waves share the tokens' values, which go through LDS in slices of 512 k in the order of the operand. A wave's codes
// and scales of a slice are all in flight while the slice before is multiplied: 9 KB a wave, no barrier waits for them.
// MOST: tiles of 16 pairs at a time. SECOND: the product with W2, its sum cut into p.split parts of slices, else with W1. HOLD: X
// is at most two slices and stays where it is while the work-group goes through several column tiles, without a barrier (40
// tokens, 256 experts of 1024 x 1024: the layer 85 us, 101 without; 200 tokens, 4096 x 512: 232 and 264; four
// slices, two work-groups a CU with more tiles each, gained 6 % where no expert had more than a tile of pairs and lost 8 % where
// some had: one work-group more than fit takes a whole turn). ROUTE: as above.
constexpr int kRowWaves = 4, kRowThreads = 64 * kRowWaves, kSlice = 512, kSliceChunks = kSlice / kChunk;
constexpr int kWaveCodes = 2 * (1024 + 512);  // LDS bytes of a wave: a chunk's codes and a slice's scales of two tiles

template <int NT, int MOST, bool SECOND, bool HOLD, bool ROUTE>
__global__ __launch_bounds__(kRowThreads, 2) void k_moe_rows(MoeArgs p, int tiles, int groups) {
    constexpr int kXBytes = 16 * MOST * kSlice * 2;  // of a slice
    constexpr int kCols = NT == 2 ? 16 * kRowWaves : 32 * kRowWaves;
    __shared__ __attribute__((aligned(16))) uint8_t lds_x[2][kXBytes];
    __shared__ __attribute__((aligned(16))) uint8_t lds_w[kRowWaves][kWaveCodes];
    __shared__ typename Pick<kRowThreads, 16 * MOST>::Lds pick_lds;
    uint16_t *const list = pick_lds.list;
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    __shared__ int route_ids[ROUTE ? kRouteTokens * kMoeMaxTopK : 1];
    if (ROUTE) route_here<kRowWaves>(p, p.top_k, blockIdx.x == 0, route_ids);
    const int *const ids = ROUTE ? route_ids : p.ids;
    Pick<kRowThreads, 16 * MOST> pick;
    pick.find(p, ids, blockIdx.x / groups, pick_lds);
    const int expert = pick.expert, pairs = pick.n;
    if (expert < 0) return;
    const int K = (int)(SECOND ? p.inner : p.width), F = (int)(SECOND ? p.width : p.inner);
    // The work-group's column tiles: first, first + groups, ...
    const int first = (int)(blockIdx.x % groups), turns = HOLD ? (tiles - first + groups - 1) / groups : 1;
    auto column = [&](int turn) __attribute__((always_inline)) { return (first + turn * groups) * kCols + (NT == 2 ? 16 : 32) * wave; };
    const int slices = (K + kSlice - 1) / kSlice;
    const int s_lo = SECOND ? (int)((int64_t)slices * blockIdx.y / gridDim.y) : 0;
    const int s_hi = SECOND ? (int)((int64_t)slices * (blockIdx.y + 1) / gridDim.y) : slices;
    const MoeWeights &W = SECOND ? p.down : p.up;
    const float alpha = W.alpha[expert];
    const uint16_t *x = SECOND ? p.h : static_cast<const uint16_t *>(p.x);
    const int64_t ldx = SECOND ? p.inner : p.ldx;
    uint8_t *const wl = lds_w[wave];
    // Rows of the two tiles that are being loaded; a tile past the last is read as the last.
    const uint8_t *codes[2], *scales[2];
    auto take_rows = [&](int turn) __attribute__((always_inline)) {
        const int f0 = column(turn);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t row = (int64_t)expert * NT * F + (NT == 2 ? min(f0, F - 16) + j * F : min(f0 + 16 * j, F - 16));
            codes[j] = W.codes + row * (K / 2);
            scales[j] = W.scales + row * (K / 16);
        }
    };
    // codes: the lane loads row lane / 4, 16 bytes lane % 4 of a chunk; scales: row lane / 4, the 8 of chunk lane % 4
    const uint32_t crow = (uint32_t)(lane >> 2) * (uint32_t)(K / 2), srow = (uint32_t)(lane >> 2) * (uint32_t)(K / 16);
    auto pass = [&](auto tiles_of_pairs) __attribute__((always_inline)) {
        constexpr int MT = tiles_of_pairs.value, kX = 16 * MT * kSlice * 2 / 16 / kRowThreads;  // tiles; pieces a thread
        u32x4 cv[2][kSliceChunks], xv[kX];
        u32x2 sv[2];
        f32x4 acc[2][MT] = {};
        // Loads past a row's end (K >= 128) are moved back inside it, and what they bring is put in its place when it is stored.
        auto load_codes = [&](int s, int c) __attribute__((always_inline)) {
            const uint32_t at = min((uint32_t)(kSlice * s + kChunk * c) / 2 + 16u * (lane & 3), (uint32_t)K / 2 - 16u) + crow;
#pragma unroll
            for (int j = 0; j < 2; ++j) cv[j][c] = *reinterpret_cast<const u32x4_any *>(codes[j] + at);
        };
        auto load_scales = [&](int s) __attribute__((always_inline)) {
            const uint32_t at = min((uint32_t)(kSlice / 16 * s) + 8u * (lane & 3), (uint32_t)K / 16 - 8u) + srow;
#pragma unroll
            for (int j = 0; j < 2; ++j) sv[j] = *reinterpret_cast<const u32x2_any *>(scales[j] + at);
        };
        auto store_codes = [&](int s, int c) __attribute__((always_inline)) {
            const int k0 = kSlice * s + kChunk * c, k = k0 + 32 * (lane & 3);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                u32x4 v = cv[j][c];
                if (k0 + kChunk > K) {
                    if (k + 32 > K) v = k < K ? u32x4{v.z, v.w, 0u, 0u} : u32x4{0u, 0u, 0u, 0u};
                }
                *reinterpret_cast<u32x4 *>(wl + 1024 * j + code_place(lane >> 2, lane & 3)) = v;
            }
        };
        auto store_scales = [&](int s) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                u32x2 v = sv[j];
                if (kSlice * (s + 1) > K) {
                    const int past = kSlice / 16 * s + 8 * (lane & 3) - (K / 16 - 8);
                    const uint64_t w = past >= 8 ? 0u : __builtin_bit_cast(uint64_t, v) >> (8 * max(past, 0));
                    v = __builtin_bit_cast(u32x2, w);
                }
                *reinterpret_cast<u32x2 *>(wl + 2048 + 512 * j + 8 * lane) = v;
            }
        };
        take_rows(0);
        load_scales(s_lo);
#pragma unroll
        for (int c = 0; c < kSliceChunks; ++c) load_codes(s_lo, c);
        pick.fill(p, ids, blockIdx.x / groups, pick_lds);  // (the codes are on their way)
        // Piece e = tid + 256 i of a slice: token e / 64 of the tiles (a wave has one at a time), k = 8 (e % 64) .. + 7. Tokens
        // past the last are read as the last: their columns are not stored.
        const uint16_t *xr[kX];
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            const int pair = __builtin_amdgcn_readfirstlane((int)list[min(wave + kRowWaves * i, pairs - 1)]);
            xr[i] = x + (int64_t)(SECOND ? pair : pair / p.top_k) * ldx;
        }
        auto load_x = [&](int s) __attribute__((always_inline)) {
            const uint32_t at = min((uint32_t)(kSlice * s) + 8u * lane, (uint32_t)K - 8u);
#pragma unroll
            for (int i = 0; i < kX; ++i) xv[i] = *reinterpret_cast<const u32x4_any *>(xr[i] + at);
        };
        // In LDS: [chunk][token tile][product i][lane] pieces, token r at lane (r ^ f) + 16 g with f of the piece's place in
        // its chunk: the sixteen pieces of a chunk that neighbouring threads write meet no bank twice.
        auto x_place = [&](int c, int m, int i, int gg, int r) __attribute__((always_inline)) {
            return (((c * MT + m) * 4 + i) * 64 + 16 * gg + (r ^ (4 * gg + i))) * 16;
        };
        auto store_x = [&](int s, uint8_t *xb) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kX; ++i) {
                const int r = wave + kRowWaves * i;
                u32x4 v = xv[i];
                if (kSlice * (s + 1) > K && kSlice * s + 8 * lane >= K) v = u32x4{0u, 0u, 0u, 0u};
                *reinterpret_cast<u32x4 *>(xb + x_place(lane >> 4, r >> 4, lane & 3, (lane >> 2) & 3, r & 15)) = v;
            }
        };
        // Slice s of the loaded codes with the X at xb, and the loads of slice `next` (of the rows taken last).
        auto multiply = [&](int s, int next, const uint8_t *xb) __attribute__((always_inline)) {
            wave_handover();  // the slice before's scales have been read (where X is held no barrier lies between)
            store_scales(s);
            load_scales(next);
#pragma unroll
            for (int c = 0; c < kSliceChunks; ++c) {
                __builtin_amdgcn_sched_barrier(0);
                wave_handover();
                store_codes(s, c);
                load_codes(next, c);
                wave_handover();
                bf16x8 b[MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[m][i] = *reinterpret_cast<const bf16x8 *>(xb + x_place(c, m, i, g, r16));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const u32x4 cur = *reinterpret_cast<const u32x4 *>(wl + 1024 * j + code_place(r16, g));
                    const uint32_t sb = *reinterpret_cast<const u16_lds *>(wl + 2048 + 512 * j + 32 * r16 + 8 * c + 2 * g);
                    const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)(sb & 0x7F7Fu), false);  // both scales
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 w = dequant8(cur[i], i < 2 ? d.x : d.y);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            acc[j][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), b[m][i], acc[j][m], 0, 0, 0);
                    }
                }
            }
        };
        auto finish = [&](int turn) __attribute__((always_inline)) {
            const int f0 = column(turn);
            // Element r of the lane is weight row 4 g + r of a tile, pair r16 of a tile of pairs.
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (16 * m + r16 >= pairs) continue;
                const int64_t pair = list[16 * m + r16];
                if (SECOND) {
                    const float w = p.weights[pair];
                    float *z = p.z + ((int64_t)blockIdx.y * p.tokens * p.top_k + pair) * F + f0 + 4 * g;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (f0 + 16 * j < F) *reinterpret_cast<f32x4 *>(z + 16 * j) = (acc[j][m] * alpha) * w;
                } else {
                    uint16_t *h = p.h + pair * F + f0 + 4 * g;
#pragma unroll
                    for (int j = 0; j < (NT == 2 ? 1 : 2); ++j) {
                        if (f0 + 16 * j >= F) continue;
                        float v[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            v[r] = act_value(alpha * acc[j][m][r], p.act);
                            if (NT == 2) v[r] *= alpha * acc[1][m][r];
                        }
                        const uint2 hi = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                        *reinterpret_cast<uint2 *>(h + 16 * j) = hi;
                        if (p.h_low)
                            *reinterpret_cast<uint2 *>(p.h_low + pair * F + f0 + 4 * g + 16 * j) =
                                make_uint2(pack_bf16(rest_of(v[0], bf16_lo(hi.x)), rest_of(v[1], bf16_hi(hi.x))),
                                           pack_bf16(rest_of(v[2], bf16_lo(hi.y)), rest_of(v[3], bf16_hi(hi.y))));
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[j][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        };
        load_x(s_lo);
        if (HOLD) {
            store_x(s_lo, lds_x[0]);
            if (s_hi - s_lo > 1) {
                load_x(s_lo + 1);
                store_x(s_lo + 1, lds_x[1]);
            }
            lds_barrier();
#pragma unroll 1
            for (int turn = 0; turn < turns; ++turn) {
#pragma unroll 1
                for (int s = s_lo; s < s_hi; ++s) {
                    const bool last = s + 1 == s_hi;
                    if (last) take_rows(min(turn + 1, turns - 1));  // (after the last tile itself again: nothing looks at it)
                    multiply(s, last ? s_lo : s + 1, lds_x[s - s_lo]);
                }
                finish(turn);
            }
        } else {
#pragma unroll 1
            for (int s = s_lo; s < s_hi; ++s) {
                store_x(s, lds_x[s & 1]);
                lds_barrier();
                const int next = min(s + 1, s_hi - 1);
                load_x(next);
                multiply(s, next, lds_x[s & 1]);
            }
            finish(0);
        }
    };
    if (MOST == 2 && pairs > 16)
        pass(std::integral_constant<int, MOST>{});
    else
        pass(std::integral_constant<int, 1>{});
}

// y of eight columns of a token per thread: the parts in the order of the choices.
__global__ __launch_bounds__(256) void k_moe_sum(MoeArgs p, int per) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, t = i / per, c = 8 * (i % per);
    if (t >= p.tokens) return;
    float v[8] = {};
    if (p.res) {
        Raw8<uint16_t> r;
        r.load(p.res + t * p.ldr + c, 8);
        r.get(v);
    }
    for (int part = 0; part < p.split; ++part) {
        const float *z = p.z + ((int64_t)part * p.tokens + t) * p.top_k * p.width + c;
#pragma unroll 4
        for (int j = 0; j < p.top_k; ++j) {  // (a choice that is none: what lies there is not taken)
            const f32x4 a = *reinterpret_cast<const f32x4 *>(z + (int64_t)j * p.width);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(z + (int64_t)j * p.width + 4);
            const bool taken = p.ids[t * p.top_k + j] >= 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += taken ? a[k] : 0.0f, v[4 + k] += taken ? b[k] : 0.0f;
        }
    }
    put8(p.y + t * p.width + c, v, 8);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Which kernels a call takes, and how many parts the second product's sum is cut into.
struct Plan {
    int route, up_rows, down_rows, down_sum, mt, split;  // route: a kernel of its own; down_sum: the second product with the sum
    int up_turns, down_turns;  // column tiles of a work-group
};

Plan plan_moe(int64_t tokens, int64_t width, int64_t inner, int experts, int top_k, bool gated) {
    // Experts that some token chooses, if all are as likely.
    double idle = 1.0;
    for (int64_t t = 0; t < tokens && idle > 1e-3; ++t) idle *= 1.0 - (double)top_k / experts;
    const double used = experts * (1.0 - idle);
    Plan plan = {};
    plan.mt = tokens > 16 && tokens * top_k > 12 * used ? 2 : 1;  // pairs of an expert
    // Entries of the list: work-groups by column tiles (counted by experts alone: 256 tokens, 2 of 8 experts of 4096 x 1408 109 us,
    // 77 so; 2 of 16 of 1024 x 512 41 and 27; 200 tokens, 4 of 16 of 2048 x 512 47 and 37).
    const double lists = used * ceil(tokens * top_k / used / (16 * plan.mt));
    const int64_t up = (inner + (gated ? 63 : 127)) / (gated ? 64 : 128), down = (width + 127) / 128;
    // k_moe_rows where there are work-groups for most of the GPU. One token, 8 experts of 2048 x 768 (96 work-groups): the layer
    // 26 us with it, 20 without; 8 tokens, 35 experts of 4096 x 1408 (770): the first product 47 us, 65 without.
    plan.up_rows = width >= kChunk && lists * up >= 192;
    // The same for the second product; where k_moe_down does the sum as well, from more work on: the latter layer (1120
    // work-groups) 90 us, 102 with k_moe_down; the former (128) 21, 18 with it.
    plan.down_rows = inner >= kChunk && lists * down >= (tokens <= kDownTokens ? 512 : 128);
    plan.route = tokens > kRouteTokens;
    plan.down_sum = tokens <= kDownTokens && !plan.down_rows;
    // Parts of the second product's sum, to some 500 work-groups: 33 tokens, 8 experts of 4096 x 14336: 188 us in two, 197 in four.
    plan.split = 1;
    if (plan.down_rows) {
        const int64_t slices = (inner + kSlice - 1) / kSlice;
        while (plan.split < 8 && 4 * plan.split <= slices && lists * down * plan.split < 500) plan.split *= 2;
    }
    // Three work-groups a CU, where X stays.
    plan.up_turns = width <= 2 * kSlice ? (int)std::max(1.0, lists * up / 768.0 + 0.5) : 1;
    plan.down_turns = inner <= 2 * kSlice ? (int)std::max(1.0, lists * down / 768.0 + 0.5) : 1;
    return plan;
}

// Entries that the list of Pick has at most: a pair each, and for each expert the whole groups and one more.
int64_t entries(const MoeArgs &p, int size) {
    const int64_t pairs = p.tokens * p.top_k;
    return std::min(pairs, std::min<int64_t>(p.experts, pairs) + pairs / size);
}

template <int NT, bool SECOND>
void product(const MoeArgs &p, bool by_rows, bool apart, int mt, int turns, hipStream_t st) {
    const int64_t F = SECOND ? p.width : p.inner;
    if (!by_rows) {
        const int tiles = (int)((F + 15) / 16);
        const dim3 grid((unsigned)(entries(p, 16) * tiles));
        if constexpr (!SECOND)
            if (!apart) {
                hipLaunchKernelGGL((k_moe_product<NT, false, true>), grid, dim3(kThreads), 0, st, p, tiles);
                return;
            }
        hipLaunchKernelGGL((k_moe_product<NT, SECOND, false>), grid, dim3(kThreads), 0, st, p, tiles);
        return;
    }
    constexpr int kCols = NT == 2 ? 16 * kRowWaves : 32 * kRowWaves;
    const int tiles = (int)((F + kCols - 1) / kCols), groups = (tiles + turns - 1) / turns;
    const dim3 grid((unsigned)(entries(p, 16 * mt) * groups), SECOND ? p.split : 1), block(kRowThreads);
    auto run = [&](auto mts, auto hold, auto route) {
        hipLaunchKernelGGL((k_moe_rows<NT, mts.value, SECOND, hold.value, route.value>), grid, block, 0, st, p, tiles, groups);
    };
    auto held = [&](auto mts, auto hold) {
        if constexpr (SECOND || mts.value > 1)
            run(mts, hold, std::false_type{});
        else
            apart ? run(mts, hold, std::false_type{}) : run(mts, hold, std::true_type{});
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    if (mt == 2)
        turns > 1 ? held(Two{}, std::true_type{}) : held(Two{}, std::false_type{});
    else
        turns > 1 ? held(One{}, std::true_type{}) : held(One{}, std::false_type{});
}

}  // namespace

// ids, weights, h, then its second part, or z
size_t moe_workspace(int64_t tokens, int64_t width, int64_t inner, int experts, int top_k) {
    const size_t pairs = (size_t)(tokens * top_k);
    const size_t split = std::max(plan_moe(tokens, width, inner, experts, top_k, false).split, plan_moe(tokens, width, inner, experts, top_k, true).split);
    return 2 * round256(4 * pairs) + round256(2 * pairs * inner) + std::max(round256(4 * split * pairs * width), round256(2 * pairs * inner));
}

hipError_t launch_moe(const MoeArgs &a, void *ws, hipStream_t st) {
    MoeArgs p = a;
    const size_t pairs = (size_t)(p.tokens * p.top_k);
    const Plan plan = plan_moe(p.tokens, p.width, p.inner, p.experts, p.top_k, p.gated);
    uint8_t *at = static_cast<uint8_t *>(ws);
    p.ids = reinterpret_cast<int *>(at), at += round256(4 * pairs);
    p.weights = reinterpret_cast<float *>(at), at += round256(4 * pairs);
    p.h = reinterpret_cast<uint16_t *>(at), at += round256(2 * pairs * p.inner);
    p.z = reinterpret_cast<float *>(at);
    p.h_low = plan.down_sum ? reinterpret_cast<uint16_t *>(at) : nullptr;
    p.split = plan.split;
    if (plan.route) {
        hipLaunchKernelGGL(k_moe_route, dim3((unsigned)((p.tokens + 3) / 4)), dim3(256), 0, st, p);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    if (p.gated)
        product<2, false>(p, plan.up_rows, plan.route, plan.mt, plan.up_turns, st);
    else
        product<1, false>(p, plan.up_rows, plan.route, plan.mt, plan.up_turns, st);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (plan.down_sum) {
        hipLaunchKernelGGL(k_moe_down, dim3((unsigned)(p.width / 16)), dim3(kDownThreads), 0, st, p);
        return hipGetLastError();
    }
    product<1, true>(p, plan.down_rows, true, plan.mt, plan.down_turns, st);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int per = (int)(p.width / 8);
    hipLaunchKernelGGL(k_moe_sum, dim3((unsigned)((p.tokens * per + 255) / 256)), dim3(256), 0, st, p, per);
    return hipGetLastError();
}

}  // namespace nvfp4
