// gfx950 W4 products with the rest of a layer's projection in their epilogue, and their gradients.
//
// Forward: z[M][N] = alpha (X Wq^T) + bias with Wq = e2m1(code) e4m3(scale) ([N][K], exact in bf16) and X bf16 or
// MXFP8 (mx.hpp; exact in bf16 down to 2^-133); y = act(z) + residual, or, gated, with F = N / 2,
//     y[:, f] = act(z[:, f]) z[:, F + f] + residual[:, f].
// act: none, silu(z) = z s(z), gelu(z) = z s(2 c (z + 0.044715 z^3)), c = sqrt(2/pi) (the tanh form), s the logistic
// function. z may be kept, bf16 or MXFP8.
// Gradient: dz = dy act'(z) (gated: dy u act'(g) and dy act(g) for z = (g, u)), dX = alpha (dz Wq),
// dbias = the column sums of dz. dz is an output rounded to bf16, and dX is the product of that rounding (the
// matrix cores take bf16; its error, at most 2^-8 of a term and independent between terms, is of the size of dX's
// own rounding: together 0.0023 of dX's norm, where a product of dz in fp32 has 0.0017. dz whole, in two bf16 parts,
// would double the matrix cores' work); dbias adds dz unrounded.
//
// Products are exact and summed in fp32 on the matrix cores; everything after the sum is fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "codec.hpp"
#include "launch.hpp"
#include "mx.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int clamp_count(int64_t left, int most) {
    return left >= most ? most : left > 0 ? (int)left : 0;
}

// A barrier that orders LDS alone: __syncthreads also waits until the work-group's stores to global memory have
// been acknowledged, which nothing here depends on.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Between what a wave's lanes store in LDS and what other lanes of it load there, or store over it: the hardware keeps a
// wave's LDS accesses in order, this keeps the compiler from reordering them. No instruction.
__device__ __forceinline__ void wave_handover() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// ------------------------------------------------------------------------------------- activations

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// 1 / (1 + e^-v): the hardware exp2 and reciprocal, each within about one unit in the last place; v itself
// is rounded once more in v log2(e), a relative error of |v| 2^-24 in e^-v.
__device__ __forceinline__ float logistic(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

__device__ __forceinline__ float act_value(float z, int act) {
    if (act == kActSilu) return z * logistic(z);
    if (act == kActGelu) return z * logistic(kGelu2C * __builtin_fmaf(kGeluA * z * z, z, z));
    return z;
}

// act(z) and act'(z). The gelu's derivative is 0 or 1 to fp32 beyond |z| = 30; the clamp keeps z^2 finite. The clamp
// would take a NaN or an infinity for a number: z - z, 0 for every finite z, makes its slope the NaN that the formulas
// give (an infinity's is inf * 0).
__device__ __forceinline__ float2 act_both(float z, int act) {
    if (act == kActSilu) {
        const float s = logistic(z);
        return make_float2(z * s, s * __builtin_fmaf(z, 1.0f - s, 1.0f));
    }
    const float c = fminf(fmaxf(z, -30.0f), 30.0f);
    const float c2 = c * c;
    const float s = logistic(kGelu2C * __builtin_fmaf(kGeluA * c2, c, c));
    const float slope = __builtin_fmaf(c * s * (1.0f - s), kGelu2C * __builtin_fmaf(3.0f * kGeluA, c2, 1.0f), s);
    return make_float2(z * s, slope + (z - z));
}

// ---------------------------------------------------------------------------------------- epilogue

// Eight values of a row of bias or residual (bf16 or fp32), n of them in the matrix; the rest read as zeros.
// WHOLE, here and below: n is 0 or 8 (the output's columns are a multiple of eight), which leaves one vector
// access behind a mask; else the end of a row is taken element by element.
template <bool WHOLE>
struct RawAny {
    uint4 a, b;
    __device__ __forceinline__ void load(const void *q, int f32, int64_t e, int n) {
        a = b = make_uint4(0u, 0u, 0u, 0u);
        if (WHOLE && n == 0) return;
        if (f32) {
            Raw8<float> r;
            r.load(static_cast<const float *>(q) + e, WHOLE ? 8 : n);
            a = r.a, b = r.b;
        } else {
            Raw8<uint16_t> r;
            r.load(static_cast<const uint16_t *>(q) + e, WHOLE ? 8 : n);
            a = r.a;
        }
    }
    __device__ __forceinline__ void get(int f32, float v[8]) const {
        const uint32_t d[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = f32 ? __uint_as_float(d[i]) : i & 1 ? bf16_hi(d[i >> 1]) : bf16_lo(d[i >> 1]);
    }
};

template <bool WHOLE, typename T>
__device__ __forceinline__ void put(T *q, const float v[8], int n) {
    if (!WHOLE)
        put8(q, v, n);
    else if (n > 0)
        put8(q, v, 8);
}

// What an epilogue does. Plain (y = alpha * sum in bf16, nothing else: the gradient's product, projections without
// extras) is a kernel of its own, since a work-group's epilogue is not overlapped with anything where one fills a
// CU; the others look at the call's arguments as they go. The full one of the 256-row tile, four rows of sums and
// residuals at a time, needs 27 registers more than there are (112 bytes of scratch a thread).
enum { kEpiPlain = 0, kEpiFull = 1, kEpiGated = 2 };

// bias of the output columns f .. f + 7 and of their gate partners (zeros without a bias).
template <int EPI, bool WHOLE>
__device__ __forceinline__ void load_bias(const LinArgs &p, int64_t f, int n, float bg[8], float bu[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) bg[i] = bu[i] = 0.0f;
    if (EPI == kEpiPlain || !p.bias) return;
    RawAny<WHOLE> r;
    r.load(p.bias, p.bias_f32, f, n);
    r.get(p.bias_f32, bg);
    if (EPI == kEpiGated) {
        r.load(p.bias, p.bias_f32, p.F + f, n);
        r.get(p.bias_f32, bu);
    }
}

// Everything after alpha * sum for the output columns f .. f + 7 of R rows m, m + dm, ..., n[r] of which columns are in
// the matrix (0: the lane only takes part in its block's maximum; a quad of lanes holds 32 consecutive columns).
// g: alpha * sum of the columns; u: of their gate partners; res: the residual's values, requested by the caller
// ahead. Row by row inside each step, so that a step's branches are taken once for all rows.
template <int EPI, bool WHOLE, int R>
__device__ __forceinline__ void epilogue(const LinArgs &p, int64_t m, int64_t dm, int64_t f, const int n[R], float g[R][8],
                                         float u[R][8], const float bg[8], const float bu[8],
                                         const RawAny<WHOLE> res[R], int lane) {
    if (EPI == kEpiPlain) {
#pragma unroll
        for (int r = 0; r < R; ++r) put<WHOLE>(static_cast<uint16_t *>(p.y) + (m + r * dm) * p.F + f, g[r], n[r]);
        return;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[r][i] += bg[i];
            if (EPI == kEpiGated) u[r][i] += bu[i];
        }
    if (p.keep == kKeepMx) {
        const int64_t nb = (p.N + kMxBlock - 1) / kMxBlock;
        uint8_t *z = static_cast<uint8_t *>(p.z);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = m + r * dm, e = row * p.N + f, s = row * nb + f / kMxBlock;
            mx_put8<WHOLE>(z + e, p.zs + s, g[r], n[r], lane);
            if (EPI == kEpiGated) mx_put8<WHOLE>(z + e + p.F, p.zs + s + p.F / kMxBlock, u[r], n[r], lane);
        }
    } else if (p.keep == kKeepBf16) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint16_t *z = static_cast<uint16_t *>(p.z) + (m + r * dm) * p.N + f;
            put<WHOLE>(z, g[r], n[r]);
            if (EPI == kEpiGated) put<WHOLE>(z + p.F, u[r], n[r]);
        }
    }
    if (p.act == kActSilu) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) g[r][i] = act_value(g[r][i], kActSilu);
    } else if (p.act == kActGelu) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) g[r][i] = act_value(g[r][i], kActGelu);
    }
    if (EPI == kEpiGated)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) g[r][i] *= u[r][i];
    if (p.res)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float v[8];
            res[r].get(p.res_f32, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[r][i] += v[i];
        }
    if (p.y_f32)
#pragma unroll
        for (int r = 0; r < R; ++r) put<WHOLE>(static_cast<float *>(p.y) + (m + r * dm) * p.F + f, g[r], n[r]);
    else
#pragma unroll
        for (int r = 0; r < R; ++r) put<WHOLE>(static_cast<uint16_t *>(p.y) + (m + r * dm) * p.F + f, g[r], n[r]);
}

// --------------------------------------------------------------------------------------- tile kernel

// The weights go straight from memory into the matrix cores' A operand: a wave owns 64 weight rows (two
// tiles of 32), so no weight is decoded twice in a work-group. X (32 MT rows of bf16, the B operand) goes through
// LDS; the work-group's four waves read it all.
//
// v_mfma_f32_32x32x16_bf16 sums over its 16 k slots in any order, and its 32 A rows may be any rows, so
// both are mapped to suit the memory:
//   k: lane l (half h = l / 32) takes k = 32 h + 8 i .. + 7 of a step of 64 for product i = 0..3: 16 contiguous
//      bytes of codes and two scale bytes per row and step; X is read from LDS with the same map.
//   rows: slot r = 8 b + 4 h' + i' holds weight row 16 h' + 4 b + i', because the result's element e = 4 b + i'
//      of a lane is slot 8 b + 4 h + i': a lane ends with 16 consecutive columns of one row of X.
// Gated: the wave's first tile holds 32 rows f, the second the rows F + f.
constexpr int kTileThreads = 256, kStep = 64;

// Instruction classes of the scheduling groups.
constexpr int kValu = 0x002, kMfma = 0x008, kVmemRead = 0x020, kDsRead = 0x100, kDsWrite = 0x200;

__device__ __forceinline__ int slot_row(int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }

// X of one step in registers, between the loads and the LDS stores.
template <int MT>
struct XStage {
    uint4 v[MT];
};

// Where a thread reads X (eight threads per row, 8 values each): byte offsets from the first row and k of the
// work-group's tile, which are uniform (rows past the last read the last: the API keeps ld below 2^23, so 32 bits
// hold them).
template <int MT>
struct XAddr {
    const uint8_t *x;  // row m0, k = 0
    uint32_t off[MT];
    __device__ __forceinline__ XAddr(const LinArgs &p, int64_t m0, int tid) {
        const int last = (int)min((int64_t)(32 * MT - 1), p.M - 1 - m0);
        x = static_cast<const uint8_t *>(p.x) + m0 * p.ldx * 2;
#pragma unroll
        for (int i = 0; i < MT; ++i)
            off[i] = (uint32_t)min(last, (tid >> 3) + 32 * i) * (uint32_t)p.ldx * 2u + 16u * (uint32_t)(tid & 7);
    }
};

// WHOLE: the step lies inside the slice (else its k are masked).
template <int MT, bool WHOLE>
__device__ __forceinline__ void x_load(XStage<MT> &S, const XAddr<MT> &q, int64_t k0, int64_t kend, int tid) {
    const uint8_t *x = q.x + k0 * 2;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        if (WHOLE || k0 + kStep <= kend) {
            S.v[i] = load16(x + q.off[i]);
        } else {
            Raw8<uint16_t> r;
            r.load(reinterpret_cast<const uint16_t *>(x + q.off[i]), clamp_count(kend - k0 - 8 * (tid & 7), 8));
            S.v[i] = r.a;
        }
    }
}

// LDS rows are 64 bf16 in eight 16-byte chunks, chunk c of row r at position c ^ (r / 2 % 8). Two rows span the 64
// banks; the 16 lanes that read one c of 16 rows at once then meet no bank twice (with r % 8 there were two rows
// to a bank and four more cycles a read; LDS does not bound the kernel: 1 % of its time). That is X's reads; the
// epilogue's and the codes' accesses do conflict: conflict cycles are a tenth of the LDS instructions in the 256-row
// tile, 0.4 of them in the 32-row one.
__device__ __forceinline__ int x_place(int row, int chunk) { return row * kStep + ((chunk ^ ((row >> 1) & 7)) << 3); }

template <int MT>
__device__ __forceinline__ void x_store(const XStage<MT> &S, uint16_t *xs, int tid) {
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<uint4 *>(&xs[x_place((tid >> 3) + 32 * i, tid & 7)]) = S.v[i];
}

// A lane's weights of one step: codes and scales of its row in both tiles, or the decoded fragments.
struct WCodes {
    uint4 c[2];
    uint32_t s[2];
};
struct WFrag {
    uint4 v[2][4];
};
// A wave's codes of two steps (64 rows of 64 bytes) and their scales (8 bytes a row) between memory and LDS. A lane
// needs 16 bytes of each of two rows per step, and a load of just those touches 32 lines for 1 KB: four times the
// address cycles of whole rows, which four lanes read together here.
struct WStage {
    uint4 c[4];
    uint2 s;
};
constexpr int kWaveCodes = 64 * 64, kWaveScales = 64 * 8;  // LDS bytes of a wave

// 16-byte chunk q (0..3) of row r of a wave's codes.
__device__ __forceinline__ int w_place(int r, int q) { return r * 64 + ((q ^ ((r >> 2) & 3)) << 4); }

// Where the weights come from.
//   kSrcCodes: as stored, the sum running along their rows (the forward).
//   kSrcFrag: decoded beforehand, in the order of the fragments (k_lin_decode, k_lin_transpose): coalesced and
//     without the decoding, a step of a 256 x 256 tile takes 1.47 us instead of 1.66.
//   kSrcTurn: as stored, the sum running along their columns (the gradient): a wave decodes its 64 columns of 64
//     weight rows, pairs the values along the sum, and turns them into fragments in LDS. What a decoding pass
//     before would write and read again (four bytes a weight) is saved; the work is repeated for every tile of
//     rows of X.
enum { kSrcCodes = 0, kSrcFrag = 1, kSrcTurn = 2 };

// kSrcTurn: the codes of 8 weight rows by 8 columns per lane (lane = 8 (rows / 8) + columns / 8), and the scale bytes
// of the wave's 64 columns for row `lane`.
struct TStage {
    uint32_t c[8];
    uint32_t s;
};
constexpr int kTurnFrags = 8192, kTurnLds = kTurnFrags + 4 * 64;  // LDS bytes of a wave: fragments, scales
// 16-byte piece u (32 half + slot) of product i and column tile j. The pieces that eight lanes write at once are 4 or 8
// apart: the swizzle puts them in different banks, and keeps eight consecutive ones in different banks.
__device__ __forceinline__ int turn_place(int j, int i, int u) { return (((j * 4 + i) * 64) + ((u ^ ((u >> 3) & 7)) ^ j)) * 16; }

// MT: tiles of 32 rows of X.
template <int MT, int SRC, int EPI>
__global__ __launch_bounds__(kTileThreads, MT >= 4 ? 1 : 2) void k_lin_tile(LinArgs p) {
    constexpr int kTpr = MT >= 8 ? 2 : 1, kXHalf = 32 * MT * kStep;  // tiles per epilogue round; one X buffer
    constexpr bool kCodes = SRC == kSrcCodes, kFrag = SRC == kSrcFrag, kTurn = SRC == kSrcTurn;
    constexpr int kWaveLds = kCodes ? kWaveCodes + kWaveScales : kTurn ? kTurnLds : 0;
    constexpr int kLdsX = 2 * kXHalf * 2, kLdsLoop = kLdsX + 4 * kWaveLds;
    constexpr int kLds = kLdsLoop > kTpr * 32768 ? kLdsLoop : kTpr * 32768;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
    uint16_t *const xs = reinterpret_cast<uint16_t *>(lds);
    constexpr bool kGated = EPI == kEpiGated;
    const int tid = threadIdx.x, lane = tid & 63, r32 = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // Work-groups go to the 8 XCDs round robin: give each XCD a contiguous run of tiles, and order the tiles
    // in bands of four along M, so that the work-groups on an XCD share rows of X and of W in its L2.
    const unsigned total = gridDim.x, q8 = total / 8, r8 = total % 8, xcd = blockIdx.x % 8;
    const unsigned b = xcd * q8 + min(xcd, r8) + blockIdx.x / 8;
    const unsigned slice = b / p.tiles, t0 = b % p.tiles;
    const unsigned band = t0 / (4 * p.tiles_n), in = t0 % (4 * p.tiles_n);
    const unsigned bm = min(4u, p.tiles_m - 4 * band);
    const int64_t m0 = (int64_t)(4 * band + in % bm) * (32 * MT);
    const int64_t tn = p.tn0 + in / bm;
    const int64_t kbeg = (int64_t)slice * p.kslice, kend = min(p.L, kbeg + p.kslice);
    const int64_t kfull = kbeg + (kend - kbeg) / (2 * kStep) * (2 * kStep);  // the end of its whole pairs of steps
    const int64_t f0 = kGated ? tn * 128 + 32 * wave : tn * 256 + 64 * wave;
    const int64_t steps_all = (p.L + kStep - 1) / kStep, ktiles = (p.F + 31) / 32;  // kFrag; F = N unless gated
    // The wave's weight rows: tile j starts at row w0[j] (uniform) and has `rows[j]` of them; rows past the last
    // read the last.
    int64_t w0[2];
    int rows[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t first = kGated ? min(p.F - 1, f0) : min(p.N - 1, f0 + 32 * j);
        rows[j] = (int)min((int64_t)32, (kGated ? p.F : p.N) - first);
        w0[j] = first + (kGated && j ? p.F : 0);
    }

    using Weights = typename std::conditional<kCodes, WCodes, WFrag>::type;
    f32x16 acc[2][MT] = {};
    // X is loaded one step ahead of its store, two where a step is short.
    constexpr int kSets = MT >= 8 ? 1 : 2;
    XStage<MT> X[kSets];
    const XAddr<MT> xa(p, m0, tid);
    Weights W[2];
    WStage S;
    bf16x8 A[2][2], B[2][MT];  // the fragments of one phase and of the next (A: decoded weights alone)

    // The stage's codes: load i takes rows 16 i + lane / 4 of the wave's 64, chunk lane % 4; its scales: row lane.
    uint32_t soff[4], sscale = 0u;
    uint8_t *const wl = lds + kLdsX + wave * kWaveLds;
    if constexpr (kCodes) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = min(slot_row((16 * i + (lane >> 2)) & 31), rows[i >> 1] - 1);
            soff[i] = (uint32_t)row * (uint32_t)(p.L / 2) + 16u * (lane & 3);
        }
        // relative to w0[0]: at most N L / 16 <= 2^31 bytes
        sscale = (uint32_t)(((half ? w0[1] - w0[0] : 0) + min(slot_row(r32), (half ? rows[1] : rows[0]) - 1)) * (p.L / 16));
    }
    auto stage_load = [&](int64_t k0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) S.c[i] = load16(p.codes + (w0[i >> 1] * p.L + k0) / 2 + soff[i]);
        S.s = load8b(p.scales + (w0[0] * p.L + k0) / 16 + sscale);
    };
    auto stage_store = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(wl + w_place(16 * i + (lane >> 2), lane & 3)) = S.c[i];
        *reinterpret_cast<uint2 *>(wl + kWaveCodes + 8 * lane) = S.s;
    };
    // The lane's codes and scales of step `odd` of the stored pair. Only the wave itself writes and reads them: a
    // wave_handover, or a barrier that stands there anyway, lies between.
    auto stage_read = [&](Weights &D, int odd) __attribute__((always_inline)) {
        if constexpr (kCodes)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                D.c[j] = *reinterpret_cast<const uint4 *>(wl + w_place(32 * j + r32, 2 * odd + half));
                D.s[j] = *reinterpret_cast<const u16_lds *>(wl + kWaveCodes + 8 * (32 * j + r32) + 4 * odd + 2 * half);
            }
    };
    auto frag_load = [&](Weights &D, int64_t k0) __attribute__((always_inline)) {
        if constexpr (kFrag)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t kt = kGated ? min(ktiles - 1, f0 / 32) + j * ktiles : min(ktiles - 1, f0 / 32 + j);
                const uint8_t *q = reinterpret_cast<const uint8_t *>(p.wt) + ((kt * steps_all + k0 / kStep) * 4096);
#pragma unroll
                for (int i = 0; i < 4; ++i) D.v[j][i] = load16(q + (uint32_t)(lane * 16) + i * 1024);
            }
    };
    // kSrcTurn: the wave's 64 columns start at cb; lanes past the last column read it again, and the scale bytes start at
    // block sb / 16 (F >= 64), so that every read lies inside a row.
    TStage T[2];
    const int kg = lane & 7, ng = lane >> 3;
    const int64_t cb = kTurn ? min(f0, p.F - 16) : 0, sb = kTurn ? min(cb, p.F - 64) : 0;
    const int kgc = kTurn ? (int)min((int64_t)kg, (p.F - cb) / 8 - 1) : 0;
    const uint32_t toff = kTurn ? (uint32_t)ng * 8u * (uint32_t)(p.F / 2) + 4u * kgc : 0u;
    const int tblock = kTurn ? (int)((cb - sb) / 16) + (kgc >> 1) : 0;
    auto turn_load = [&](auto whole, TStage &D, int64_t n0) __attribute__((always_inline)) {
        if constexpr (kTurn) {
            const uint8_t *c = p.codes + (n0 * p.F + cb) / 2;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                D.c[r] = 0u;
                if (whole.value || n0 + 8 * ng + r < kend)
                    D.c[r] = load4(c + (int64_t)r * (p.F / 2) + toff);
            }
            D.s = 0u;
            if (whole.value || n0 + lane < kend) D.s = load4(p.scales + (n0 * p.F + sb) / 16 + (uint32_t)lane * (uint32_t)(p.F / 16));
        }
    };
    float td[8];
    auto turn_scales = [&](const TStage &D) __attribute__((always_inline)) {
        if constexpr (kTurn) {
            uint8_t *const q = wl + kTurnFrags;
#pragma unroll
            for (int b = 0; b < 4; ++b) q[64 * b + lane] = (uint8_t)(D.s >> (8 * b));
            wave_handover();
            const uint2 s = *reinterpret_cast<const uint2 *>(q + 64 * tblock + 8 * ng);
            const uint32_t w[2] = {s.x & 0x7F7F7F7Fu, s.y & 0x7F7F7F7Fu};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
                td[4 * i] = a.x, td[4 * i + 1] = a.y, td[4 * i + 2] = b.x, td[4 * i + 3] = b.y;
            }
        }
    };
    // Columns 2 CP and 2 CP + 1 of the lane's eight, as fragment pieces of eight rows each.
    auto turn_columns = [&](const TStage &D, auto pair) __attribute__((always_inline)) {
        if constexpr (kTurn) {
            constexpr int CP = decltype(pair)::value;
            float v[2][8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const f32x2 q = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(D.c[r], 1.0f, CP);
                v[0][r] = q.x * td[r], v[1][r] = q.y * td[r];
            }
            auto two = [](float x, float y) { return __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u); };
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int o = 8 * (kg & 3) + 2 * CP + e, slot = 8 * ((o >> 2) & 3) + 4 * (o >> 4) + (o & 3);
                *reinterpret_cast<uint4 *>(wl + turn_place(kg >> 2, ng & 3, 32 * (ng >> 2) + slot)) =
                    make_uint4(two(v[e][0], v[e][1]), two(v[e][2], v[e][3]), two(v[e][4], v[e][5]), two(v[e][6], v[e][7]));
            }
        }
    };
    auto turn_read = [&](Weights &D) __attribute__((always_inline)) {
        if constexpr (kTurn)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) D.v[j][i] = *reinterpret_cast<const uint4 *>(wl + turn_place(j, i, lane));
    };
    auto turn_all = [&](const TStage &D) __attribute__((always_inline)) {
        turn_scales(D);
        turn_columns(D, std::integral_constant<int, 0>{});
        turn_columns(D, std::integral_constant<int, 1>{});
        turn_columns(D, std::integral_constant<int, 2>{});
        turn_columns(D, std::integral_constant<int, 3>{});
    };
    auto a_frag = [&](bf16x8 (&D)[2], const Weights &w, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (kCodes) {
                const uint32_t c = i == 0 ? w.c[j].x : i == 1 ? w.c[j].y : i == 2 ? w.c[j].z : w.c[j].w;
                const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)(w.s[j] & 0x7F7Fu), false);  // both scales
                D[j] = __builtin_bit_cast(bf16x8, dequant8(c, i < 2 ? d.x : d.y));
            }
        }
    };
    auto b_frag = [&](bf16x8 (&D)[MT], int buf, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
            D[t] = *reinterpret_cast<const bf16x8 *>(&xs[buf * kXHalf + x_place(32 * t + r32, 4 * half + i)]);
    };
    auto products = [&](const Weights &w, int i, int at) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                bf16x8 a;
                if constexpr (!kCodes)
                    a = __builtin_bit_cast(bf16x8, w.v[j][i]);
                else
                    a = A[at][j];
                acc[j][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, B[at][t], acc[j][t], 0, 0, 0);
            }
    };
    // Step `odd` of a pair, from X buffer `odd`, in four phases. At its start the fragments of phase 0 are formed and
    // X of the next kSets steps is in registers or on its way. Phase i forms the fragments of phase i + 1 while the
    // matrix cores work on its own. X: stored in phase 0 for the next step, loaded in phase 1 for the one kSets later.
    // Codes: a pair is stored in phase 0 of the odd step (every read of the pair before has been issued) and
    // loaded in phase 1 for the pair after; the lane's own are read in phase 2 for the next step. Decoded weights
    // are loaded in phase 0 for the next step; turned ones are formed in phases 0 to 2 from codes loaded two steps
    // before, and read back in phase 3. The one barrier stands before the last phase: by then every
    // wave has stored X of the next step and has read all of this one's, so that phase 3 can read ahead from the other
    // buffer and the next step can store into this one. What is loaded past the last whole pair is that pair again.
    // One wave per SIMD (MT = 8) hides nothing behind another wave, so the order inside a phase is asked for:
    // LDS reads (and weights decoded) between the first products, stores and loads between the rest.
    auto step = [&](auto parity, int64_t k0) __attribute__((always_inline)) {
        constexpr int odd = decltype(parity)::value;
        constexpr int kPairWork = kCodes && odd ? 2 : 1;  // the odd step moves the codes too
        Weights &w = W[odd], &next = W[odd ^ 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i == 3) lds_barrier();
            if ((kTurn && i == 0) || (kCodes && odd && i == 2)) wave_handover();
            b_frag(B[(i + 1) & 1], i < 3 ? odd : odd ^ 1, (i + 1) & 3);
            a_frag(A[(i + 1) & 1], i < 3 ? w : next, (i + 1) & 3);
            if (i == 0) {
                x_store<MT>(X[(odd ^ 1) & (kSets - 1)], xs + (odd ^ 1) * kXHalf, tid);
                if (kCodes && odd) stage_store();
                frag_load(next, min(k0 + kStep, kfull - kStep));
                turn_scales(T[odd ^ 1]);
                turn_columns(T[odd ^ 1], std::integral_constant<int, 0>{});
            }
            if (i == 1) {
                x_load<MT, true>(X[(odd ^ 1) & (kSets - 1)], xa, min(k0 + (1 + kSets) * kStep, kfull - kStep), kend, tid);
                if (kCodes && odd) stage_load(min(k0 + 3 * kStep, kfull - 2 * kStep));
                turn_columns(T[odd ^ 1], std::integral_constant<int, 1>{});
                turn_columns(T[odd ^ 1], std::integral_constant<int, 2>{});
            }
            if (i == 2) {
                stage_read(next, odd ^ 1);
                turn_columns(T[odd ^ 1], std::integral_constant<int, 3>{});
                turn_load(std::true_type{}, T[odd ^ 1], min(k0 + 3 * kStep, kfull - kStep));
            }
            if (i == 3) turn_read(next);
            products(w, i, i & 1);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
                __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
                if (!kFrag) __builtin_amdgcn_sched_group_barrier(kValu, 40 / MT, 0);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
                if (i == 0) __builtin_amdgcn_sched_group_barrier(kDsWrite, kPairWork, 0);
                if (kTurn && i > 0 && i < 3) __builtin_amdgcn_sched_group_barrier(kDsWrite, 1, 0);
                if ((i == 2 && kCodes) || (i == 3 && kTurn)) __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
                if (i == 1 || (i == 0 && kFrag) || (i == 2 && kTurn)) __builtin_amdgcn_sched_group_barrier(kVmemRead, kPairWork, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (kfull > kbeg) {
        x_load<MT, true>(X[0], xa, kbeg, kend, tid);
        if (kCodes) stage_load(kbeg);
        turn_load(std::true_type{}, T[0], kbeg);
        turn_load(std::true_type{}, T[1], kbeg + kStep);
        frag_load(W[0], kbeg);
        x_store<MT>(X[0], xs, tid);
        if (kTurn) {
            turn_all(T[0]);
            turn_load(std::true_type{}, T[0], min(kbeg + 2 * kStep, kfull - kStep));
            wave_handover();
            turn_read(W[0]);
        }
        if (kCodes) {
            stage_store();
            stage_load(min(kbeg + 2 * kStep, kfull - 2 * kStep));
        }
        x_load<MT, true>(X[kSets - 1], xa, kbeg + kStep, kend, tid);
        if (kSets == 2) x_load<MT, true>(X[0], xa, min(kbeg + 2 * kStep, kfull - kStep), kend, tid);
        lds_barrier();
        b_frag(B[0], 0, 0);
        stage_read(W[0], 0);
        a_frag(A[0], W[0], 0);
        // Nothing in flight at the loop's entry: its waits then count the loads of its own turns alone.
        __builtin_amdgcn_s_waitcnt(0);
#pragma unroll 1
        for (int64_t k0 = kbeg; k0 < kfull; k0 += 2 * kStep) {
            step(std::integral_constant<int, 0>{}, k0);
            step(std::integral_constant<int, 1>{}, k0 + kStep);
        }
        lds_barrier();
    }
    // The slice's last, fewer than 128 k, with masks and one step at a time.
#pragma unroll 1
    for (int64_t k0 = kfull; k0 < kend; k0 += kStep) {
        x_load<MT, false>(X[0], xa, k0, kend, tid);
        frag_load(W[0], k0);
        if (kTurn) {
            turn_load(std::false_type{}, T[0], k0);
            turn_all(T[0]);
            wave_handover();
            turn_read(W[0]);
        }
        if constexpr (kCodes)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t k = k0 + 32 * half, e = (w0[j] + min(slot_row(r32), rows[j] - 1)) * p.L + k;
                W[0].c[j] = make_uint4(0u, 0u, 0u, 0u);
                W[0].s[j] = 0u;
                if (k + 32 <= kend) {
                    W[0].c[j] = load16(p.codes + e / 2);
                    W[0].s[j] = load2b(p.scales + e / 16);
                } else if (k < kend) {  // the row's last 16
                    const uint2 c2 = load8b(p.codes + e / 2);
                    W[0].c[j].x = c2.x, W[0].c[j].y = c2.y;
                    W[0].s[j] = p.scales[e / 16];
                }
            }
        x_store<MT>(X[0], xs, tid);
        lds_barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b_frag(B[0], 0, i);
            a_frag(A[0], W[0], i);
            products(W[0], i, 0);
        }
        lds_barrier();
    }

    // The sums go through LDS, kTpr tiles of 32 rows by 256 weight rows at a time, so that the epilogue works on
    // whole rows: a thread takes eight consecutive output columns, a row's threads are consecutive. 16-byte
    // chunk c of row r sits at c ^ (r % 16).
    float *const es = reinterpret_cast<float *>(lds);
    auto place = [](int row, int chunk) { return row * 256 + ((chunk ^ (row & 15)) << 2); };
    const float alpha = p.part ? 1.0f : *p.alpha;
    constexpr int cols = kGated ? 128 : 256, threads = cols / 8;  // output columns of the work-group; threads per row
    constexpr int stride = kTileThreads / threads;  // a thread's rows are so far apart
    const int fl = 8 * (tid % threads);
    const int ch = kGated ? 16 * (fl / 32) + (fl % 32) / 4 : fl / 4;    // the chunk of column fl
    const int64_t f = tn * cols + fl;
    const int nf = clamp_count(p.F - f, 8);
    // A thread's rows of a round, up to four at a time: with one work-group per CU nothing else hides the latency
    // of their LDS reads and residuals.
    constexpr int kMine = 32 * kTpr / stride;
    auto rows_out = [&](auto whole, int round) __attribute__((always_inline)) {
        constexpr bool kWholeRow = decltype(whole)::value;
        constexpr int kRows = !kWholeRow ? 1 : kMine < 4 ? kMine : 4;
        float bg[8], bu[8];
        load_bias<EPI, kWholeRow>(p, f, p.part ? 0 : nf, bg, bu);
#pragma unroll 1
        for (int row = tid / threads; row < 32 * kTpr; row += kRows * stride) {
            const int64_t m = m0 + 32 * kTpr * round + row;
            int n[kRows];
            RawAny<kWholeRow> res[kRows];
            float g[kRows][8], u[kRows][8];
#pragma unroll
            for (int r = 0; r < kRows; ++r) n[r] = m + r * stride < p.M ? nf : 0;
            if (EPI != kEpiPlain && p.res && !p.part)
#pragma unroll
                for (int r = 0; r < kRows; ++r) res[r].load(p.res, p.res_f32, (m + r * stride) * p.ldr + f, n[r]);
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(&es[place(row + r * stride, ch + c)]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) g[r][4 * c + i] = alpha * v[i];
                    if (kGated) {
                        const f32x4 w = *reinterpret_cast<const f32x4 *>(&es[place(row + r * stride, ch + 8 + c)]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) u[r][4 * c + i] = alpha * w[i];
                    }
                }
            if (p.part) {  // fp32 sums of this slice, without alpha
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    float *q = p.part + ((int64_t)slice * p.M + m + r * stride) * p.part_n + f;
                    put<kWholeRow>(q, g[r], n[r]);
                    if (kGated) put<kWholeRow>(q + p.part_n / 2, u[r], n[r]);
                }
            } else {
                epilogue<EPI, kWholeRow, kRows>(p, m, stride, f, n, g, u, bg, bu, res, lane);
            }
        }
    };
#pragma unroll 1
    for (int round = 0; round < MT / kTpr; ++round) {
        auto dump = [&](int t, const f32x16 &a0, const f32x16 &a1) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const f32x16 &a = j ? a1 : a0;
                    *reinterpret_cast<f32x4 *>(&es[place(32 * t + r32, 16 * wave + 8 * j + 4 * half + e / 4)]) =
                        f32x4{a[e], a[e + 1], a[e + 2], a[e + 3]};
                }
        };
#pragma unroll
        for (int r = 0; r < MT / kTpr; ++r)  // a branch per round: the accumulators are not indexed at run time
            if (r == round)
#pragma unroll
                for (int t = 0; t < kTpr; ++t) dump(t, acc[0][r * kTpr + t], acc[1][r * kTpr + t]);
        lds_barrier();
        if (p.F % 8 == 0 || (tn + 1) * cols <= p.F)  // no column group of the tile ends inside the eight
            rows_out(std::true_type{}, round);
        else
            rows_out(std::false_type{}, round);
        lds_barrier();
    }
}

constexpr int kReduceThreads = 256;

// The slices' sums added in slice order, then the epilogue: eight columns per thread, rows padded to whole
// 32-column blocks so that a quad holds a block.
template <int EPI, bool WHOLE>
__global__ __launch_bounds__(kReduceThreads) void k_lin_reduce(LinArgs p, int slices, int64_t f0, int64_t per_row, int64_t groups) {
    const float alpha = *p.alpha;
    for (int64_t i = (int64_t)blockIdx.x * kReduceThreads + threadIdx.x; i < groups;
         i += (int64_t)gridDim.x * kReduceThreads) {
        const int64_t m = i / per_row, f = f0 + 8 * (i - m * per_row);
        const int n[1] = {clamp_count(p.F - f, 8)};
        RawAny<WHOLE> res[1];
        float g[1][8] = {}, u[1][8] = {}, bg[8], bu[8];
        if (EPI != kEpiPlain && p.res) res[0].load(p.res, p.res_f32, m * p.ldr + f, n[0]);
        load_bias<EPI, WHOLE>(p, f, n[0], bg, bu);
#pragma unroll 4
        for (int s = 0; s < slices; ++s) {
            const float *q = p.part + ((int64_t)s * p.M + m) * p.part_n + f;
            RawAny<WHOLE> r;
            float v[8];
            r.load(q, 1, 0, n[0]);
            r.get(1, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[0][e] += v[e];
            if (EPI == kEpiGated) {
                r.load(q + p.part_n / 2, 1, 0, n[0]);
                r.get(1, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[0][e] += v[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) g[0][e] *= alpha, u[0][e] *= alpha;
        epilogue<EPI, WHOLE, 1>(p, m, 0, f, n, g, u, bg, bu, res, (int)(threadIdx.x & 63));
    }
}

// -------------------------------------------------------------------------------------- skinny kernel

// Few rows of X (M <= 64), bound by reading the weights once: a work-group owns 16 output columns (gated: their
// 16 gate rows and 16 up rows), its waves split K in chunks of 128 (wave w takes chunks w, w + WAVES, ...) and its
// sums are joined through LDS in wave order. Products on v_mfma_f32_16x16x32_bf16, weights as A: lane l has row
// l % 16 and, for product i = 0..3 of a chunk, k = 32 (l / 16) + 8 i .. + 7; X^T as B with the same map.
// Neighbouring lanes of an operand are rows apart in memory, and a load of 64 scattered 16-byte pieces takes four
// times the address cycles of a contiguous one (they, not the bytes, bound the kernel when both operands were
// loaded so: 24 x 22016 x 4096 gated in 35 us). So a wave reads its chunk of codes in whole 64-byte pieces and
// turns it in LDS, and X comes in fragment order, written by k_lin_xfrag, or, up to kDirectRows rows, straight
// from memory: so few lanes cost little, and a launch is saved.
constexpr int kSkinnyMaxM = 64, kDirectRows = 8;
constexpr int kChunk = 128, kChunkLds = 16 * 64 + 16 * 8;  // k per chunk; LDS bytes of a tile's codes and scales

// X in the order in which k_lin_skinny's lanes read it: per chunk and tile of 16 rows 4 KB, [i][lane][8]. Rows past M
// and k past K are zeros. A work-group writes one chunk of one tile.
template <bool XMX>
__global__ __launch_bounds__(256) void k_lin_xfrag(LinArgs p, uint16_t *__restrict__ out) {
    const int lane = threadIdx.x & 63, i = threadIdx.x >> 6;
    const int64_t m = 16 * (int64_t)blockIdx.y + (lane & 15), k = kChunk * (int64_t)blockIdx.x + 32 * (lane >> 4) + 8 * i;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (m < p.M && k < p.L) {  // K % 16 == 0: the eight are in or out
        if (XMX) {
            RawMx8 r;
            r.load(static_cast<const uint8_t *>(p.x) + m * p.ldx + k, p.xs + m * ((p.L + kMxBlock - 1) / kMxBlock) + k / kMxBlock, 8);
            float f[8];
            r.get(f);
            v = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        } else {
            v = load16(static_cast<const uint16_t *>(p.x) + m * p.ldx + k);
        }
    }
    reinterpret_cast<uint4 *>(out)[((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * 256 + threadIdx.x] = v;
}

// MT: tiles of 16 rows of X; NT: 2 if gated. XF: X in fragment order (p.wt's place in LinArgs holds it), else direct,
// MT = 1.
template <int MT, int NT, bool XF, bool XMX, int WAVES>
__global__ __launch_bounds__(64 * WAVES)
// Four waves a SIMD, 128 registers, to four tiles of sums. The forms of four tiles need 2 (gated) and 4 registers more
// and spill them, which costs less than a wave: 24 x 22016 x 4096 gated 22.0 us, 24.6 without the bound (64 x 4096 x 4096,
// 16 waves: 13.0 both).
__attribute__((amdgpu_waves_per_eu(NT * MT <= 4 ? 4 : 1)))
void k_lin_skinny(LinArgs p) {
    // each wave's chunk of codes and scales; afterwards each wave's sums
    constexpr int kStage = WAVES * NT * kChunkLds, kSums = WAVES * MT * 1024;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kStage > kSums ? kStage : kSums];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t f0 = (int64_t)blockIdx.x * 16;
    const int64_t K = p.L, nch = (K + kChunk - 1) / kChunk, nb = (K + kMxBlock - 1) / kMxBlock;
    uint8_t *const wl = lds + wave * NT * kChunkLds;
    // codes: the lane loads row lane / 4, 16 bytes lane % 4; scales: row lane % 16, its 8 bytes
    const int64_t crow = min(p.F - 1, f0 + (lane >> 2)), srow = min(p.F - 1, f0 + r16);
    f32x4 acc[NT][MT] = {};
    uint4 cv[2][NT];
    uint2 sv[2][NT];
    const uint8_t *pc[NT], *ps[NT];  // of the wave's first chunk
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        pc[j] = p.codes + ((crow + j * p.F) * K + kChunk * wave + 32 * (lane & 3)) / 2;
        ps[j] = p.scales + ((srow + j * p.F) * K + kChunk * wave) / 16;
    }
    auto load_w = [&](uint4 (&c)[NT], uint2 (&s)[NT], int64_t ch) __attribute__((always_inline)) {
        const int64_t by = (ch - wave) * (kChunk / 16);  // uniform
        if ((ch + 1) * kChunk <= K) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                c[j] = load16(pc[j] + 8 * by);
                if (lane < 16) s[j] = load8b(ps[j] + by);
            }
            return;
        }
        const int64_t kc = kChunk * ch + 32 * (lane & 3), ks = kChunk * ch;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            c[j] = make_uint4(0u, 0u, 0u, 0u);
            s[j] = make_uint2(0u, 0u);
            if (kc + 32 <= K) {
                c[j] = load16(pc[j] + 8 * by);
            } else if (kc < K) {  // the row's last 16
                const uint2 d = load8b(pc[j] + 8 * by);
                c[j].x = d.x, c[j].y = d.y;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (ks + 16 * e < K) (e < 4 ? s[j].x : s[j].y) |= (uint32_t)ps[j][by + e] << (8 * (e & 3));
        }
    };
    auto chunk = [&](const uint4 (&c)[NT], const uint2 (&s)[NT], int64_t ch) __attribute__((always_inline)) {
        const int64_t k = kChunk * ch + 32 * g;
        uint4 xv[MT][4];
        if constexpr (XF) {
            const uint4 *q = reinterpret_cast<const uint4 *>(p.wt) + ch * MT * 256 + lane;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[t][i] = q[t * 256 + i * 64];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) xv[0][i] = make_uint4(0u, 0u, 0u, 0u);
            if (r16 < p.M) {
                if constexpr (XMX) {
                    const uint8_t *q = static_cast<const uint8_t *>(p.x) + r16 * p.ldx + k;
                    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
                    float sc = 0.0f;
                    if ((ch + 1) * kChunk <= K) {
                        a = load16(q);
                        b = load16(q + 16);
                        sc = mx_scale_value(p.xs[r16 * nb + k / kMxBlock]);
                    } else if (k < K) {
                        a = load16(q);
                        sc = mx_scale_value(p.xs[r16 * nb + k / kMxBlock]);
                        if (k + 32 <= K) b = load16(q + 16);
                    }
                    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float f[8];
                        mx_decode4(w[2 * i], sc, f);
                        mx_decode4(w[2 * i + 1], sc, f + 4);
                        xv[0][i] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
                    }
                } else {
                    const uint16_t *q = static_cast<const uint16_t *>(p.x) + r16 * p.ldx + k;
                    if ((ch + 1) * kChunk <= K) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) xv[0][i] = load16(q + 8 * i);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (k + 8 * i < K) xv[0][i] = load16(q + 8 * i);
                    }
                }
            }
        }
        // Only the wave itself writes and reads its part of LDS. A row's 64 bytes are four pieces, piece q at
        // q ^ (row / 4 % 4).
        wave_handover();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            uint8_t *const q = wl + j * kChunkLds;
            *reinterpret_cast<uint4 *>(q + w_place(lane >> 2, lane & 3)) = c[j];
            if (lane < 16) *reinterpret_cast<uint2 *>(q + 1024 + 8 * lane) = s[j];
        }
        wave_handover();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint8_t *const q = wl + j * kChunkLds;
            const uint4 cur = *reinterpret_cast<const uint4 *>(q + w_place(r16, g));
            const uint32_t sb = *reinterpret_cast<const u16_lds *>(q + 1024 + 8 * r16 + 2 * g);
            const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)(sb & 0x7F7Fu), false);  // both scales
            const uint4 w[4] = {dequant8(cur.x, d.x), dequant8(cur.y, d.x), dequant8(cur.z, d.y), dequant8(cur.w, d.y)};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[i]),
                                                                        __builtin_bit_cast(bf16x8, xv[t][i]), acc[j][t], 0, 0, 0);
        }
    };
    // two chunks' weights in flight
    int64_t c = wave;
    if (c < nch) load_w(cv[0], sv[0], c);
    if (c + WAVES < nch) load_w(cv[1], sv[1], c + WAVES);
#pragma unroll 1
    for (; c < nch; c += 2 * WAVES) {
        chunk(cv[0], sv[0], c);
        if (c + 2 * WAVES < nch) load_w(cv[0], sv[0], c + 2 * WAVES);
        if (c + WAVES >= nch) break;
        chunk(cv[1], sv[1], c + WAVES);
        if (c + 3 * WAVES < nch) load_w(cv[1], sv[1], c + 3 * WAVES);
    }
    __syncthreads();  // the sums take the place of the codes
    float (*const red)[MT][256] = reinterpret_cast<float (*)[MT][256]>(lds);
    // Element r of lane l is weight row 4 (l / 16) + r of the tile, row 16 t + l % 16 of X. A thread sums the outputs
    // o = tid, tid + 64 WAVES, ... of MT * 256.
    constexpr int kMine = (MT * 256 + 64 * WAVES - 1) / (64 * WAVES);
    float z[NT][kMine] = {};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (j) __syncthreads();
#pragma unroll
        for (int t = 0; t < MT; ++t)
            *reinterpret_cast<f32x4 *>(&red[wave][t][lane * 4]) = acc[j][t];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
            const int o = tid + 64 * WAVES * q;
            if (o < MT * 256)
#pragma unroll
                for (int w = 0; w < WAVES; ++w) z[j][q] += red[w][o >> 8][o & 255];
        }
    }
    const float alpha = *p.alpha;
    auto scalar = [](const void *b, int f32, int64_t e) {
        return f32 ? static_cast<const float *>(b)[e] : __uint_as_float((uint32_t)static_cast<const uint16_t *>(b)[e] << 16);
    };
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        const int o = tid + 64 * WAVES * q, l = (o >> 2) & 63;
        const int64_t f = f0 + 4 * (l >> 4) + (o & 3), m = 16 * (o >> 8) + (l & 15);
        if (o >= MT * 256 || f >= p.F || m >= p.M) continue;
        float a = alpha * z[0][q], u = NT == 2 ? alpha * z[NT - 1][q] : 0.0f;
        if (p.bias) {
            a += scalar(p.bias, p.bias_f32, f);
            if (NT == 2) u += scalar(p.bias, p.bias_f32, p.F + f);
        }
        if (p.keep == kKeepBf16) {
            uint16_t *e = static_cast<uint16_t *>(p.z) + m * p.N + f;
            e[0] = to_bf16(a);
            if (NT == 2) e[p.F] = to_bf16(u);
        }
        a = act_value(a, p.act);
        if (NT == 2) a *= u;
        if (p.res) a += scalar(p.res, p.res_f32, m * p.ldr + f);
        if (p.y_f32)
            static_cast<float *>(p.y)[m * p.F + f] = a;
        else
            static_cast<uint16_t *>(p.y)[m * p.F + f] = to_bf16(a);
    }
}

// ------------------------------------------------------------------------------------------ gradient

// Weights decoded to bf16 in the order in which k_lin_tile's lanes read them: 32 weight rows by a step of 64 k
// make 4 KB, [i][lane][8]: lane's row is slot_row(lane % 32), its k are 32 (lane / 32) + 8 i + 0..7. The tiles of F
// rows are padded to whole ones (gated: the up rows' tiles follow the gate rows'); what lies past the last row or
// past K is zeros. A wave takes one tile of rows by four steps: it reads whole lines and writes 1 KB at a time.
__global__ __launch_bounds__(256) void k_lin_decode(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                  int64_t F, int64_t K, uint16_t *__restrict__ wt) {
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int64_t ktiles = (F + 31) / 32, steps = (K + kStep - 1) / kStep;
    const int64_t kt = blockIdx.x, s0 = (int64_t)blockIdx.y * 16 + 4 * (threadIdx.x >> 6);
    const int64_t row = 32 * kt + slot_row(lane & 31), up = blockIdx.z;
    const int64_t e0 = (row + up * F) * K;
    uint4 c[4];
    uint32_t sb[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int64_t k = (s0 + s) * kStep + 32 * half;
        c[s] = make_uint4(0u, 0u, 0u, 0u);
        sb[s] = 0u;
        if (row < F && k + 32 <= K) {
            c[s] = load16(codes + (e0 + k) / 2);
            sb[s] = load2b(scales + (e0 + k) / 16);
        } else if (row < F && k < K) {  // the row's last 16
            const uint2 d = load8b(codes + (e0 + k) / 2);
            c[s].x = d.x, c[s].y = d.y;
            sb[s] = scales[(e0 + k) / 16];
        }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s0 + s >= steps) break;
        const float d0 = e4m3_value(sb[s] & 0x7Fu), d1 = e4m3_value((sb[s] >> 8) & 0x7Fu);
        uint4 *q = reinterpret_cast<uint4 *>(wt + (((up * ktiles + kt) * steps + s0 + s) * 4) * 512) + lane;
        q[0] = dequant8(c[s].x, d0);
        q[64] = dequant8(c[s].y, d0);
        q[128] = dequant8(c[s].z, d1);
        q[192] = dequant8(c[s].w, d1);
    }
}

// The transposed weights in the same order, for the gradient: 32 columns k (the product's rows) by a step of 64 rows n
// (its sum). A work-group takes 64 rows by 256 columns, a thread 8 x 8 of them: eight dwords of codes, whose decoded
// values are paired along n as they are packed; the eight tiles of 4 KB are put together in LDS and written
// whole. Rows past N are zeros.
__global__ __launch_bounds__(256) void k_lin_transpose(const uint8_t *__restrict__ codes,
                                                     const uint8_t *__restrict__ scales, int64_t N, int64_t K,
                                                     uint16_t *__restrict__ wt) {
    __shared__ uint4 lds[8 * 256];
    const int64_t step = blockIdx.y, steps = gridDim.y;
    const int kg = threadIdx.x & 31, ng = threadIdx.x >> 5;
    const int64_t k0 = (int64_t)blockIdx.x * 256 + 8 * kg, n0 = step * kStep + 8 * ng;
    uint32_t c[8], sb[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        c[r] = sb[r] = 0u;
        if (k0 < K && n0 + r < N) {  // K % 16 == 0: the eight columns are in or out
            const int64_t e = (n0 + r) * K + k0;
            c[r] = *reinterpret_cast<const uint32_t *>(codes + e / 2);
            sb[r] = scales[e / 16];
        }
    }
    float v[8][8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const float d = e4m3_value(sb[r] & 0x7Fu);
        const f32x2 q0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[r], 1.0f, 0);
        const f32x2 q1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[r], 1.0f, 1);
        const f32x2 q2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[r], 1.0f, 2);
        const f32x2 q3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[r], 1.0f, 3);
        v[r][0] = q0.x * d, v[r][1] = q0.y * d, v[r][2] = q1.x * d, v[r][3] = q1.y * d;
        v[r][4] = q2.x * d, v[r][5] = q2.y * d, v[r][6] = q3.x * d, v[r][7] = q3.y * d;
    }
    auto pair = [](float a, float b) { return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u); };
    // Column o of a tile sits in slot 8 b + 4 h' + i', o = 16 h' + 4 b + i'. A tile's 16-byte pieces are rotated by the
    // tile in LDS, so that the lanes of different tiles do not meet in the same banks.
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
        const int o = 8 * (kg & 3) + kk;
        const int slot = 8 * ((o >> 2) & 3) + 4 * (o >> 4) + (o & 3), tile = kg >> 2;
        const int at = (ng & 3) * 64 + 32 * (ng >> 2) + slot;
        lds[tile * 256 + ((at + tile) & 255)] =
            make_uint4(pair(v[0][kk], v[1][kk]), pair(v[2][kk], v[3][kk]), pair(v[4][kk], v[5][kk]), pair(v[6][kk], v[7][kk]));
    }
    __syncthreads();
    const int64_t tile0 = (int64_t)blockIdx.x * 8, tiles = (K + 31) / 32;
#pragma unroll
    for (int tile = 0; tile < 8; ++tile)
        if (tile0 + tile < tiles)
            reinterpret_cast<uint4 *>(wt + ((tile0 + tile) * steps + step) * 2048)[threadIdx.x] =
                lds[tile * 256 + ((threadIdx.x + tile) & 255)];
}

// dz of eight columns per thread, and its column sums over the work-group's chunk of rows (waves take every
// fourth row; their sums are joined in wave order). act = none: the sums of dy alone.
template <bool ZMX>
__global__ __launch_bounds__(256) void k_lin_dz(LinGradArgs p, int64_t chunk, float *__restrict__ part) {
    __shared__ float red[2][4][64 * 8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t f = 8 * ((int64_t)blockIdx.x * 64 + lane);
    const int n = clamp_count(p.F - f, 8);
    const int64_t r0 = (int64_t)blockIdx.y * chunk, r1 = min(p.M, r0 + chunk);
    const int64_t nb = (p.N + kMxBlock - 1) / kMxBlock;
    auto z8 = [&](int64_t m, int64_t col, float v[8]) {
        if (ZMX) {
            RawMx8 r;
            r.load(static_cast<const uint8_t *>(p.z) + m * p.ldz + col, p.zs + m * nb + col / kMxBlock, n);
            r.get(v);
        } else {
            Raw8<uint16_t> r;
            r.load(static_cast<const uint16_t *>(p.z) + m * p.ldz + col, n);
            r.get(v);
        }
    };
    float sg[8] = {}, su[8] = {};
    if (n > 0)
        for (int64_t m = r0 + wave; m < r1; m += 4) {
            float dy[8], g[8], u[8];
            Raw8<uint16_t> r;
            r.load(p.dy + m * p.lddy + f, n);
            r.get(dy);
            if (p.act == kActNone) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sg[i] += dy[i];
                continue;
            }
            z8(m, f, g);
            if (p.gated) z8(m, p.F + f, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 a = act_both(g[i], p.act);
                if (p.gated) {
                    g[i] = dy[i] * u[i] * a.y;
                    u[i] = dy[i] * a.x;
                    su[i] += u[i];
                } else {
                    g[i] = dy[i] * a.y;
                }
                sg[i] += g[i];
            }
            put8(p.dz + m * p.N + f, g, n);
            if (p.gated) put8(p.dz + m * p.N + p.F + f, u, n);
        }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) red[0][wave][8 * lane + i] = sg[i], red[1][wave][8 * lane + i] = su[i];
    __syncthreads();
    for (int o = threadIdx.x; o < 512; o += 256) {
        const int64_t col = (int64_t)blockIdx.x * 512 + o;
        if (col >= p.F) continue;
        float *q = part + (int64_t)blockIdx.y * p.N + col;
        q[0] = ((red[0][0][o] + red[0][1][o]) + red[0][2][o]) + red[0][3][o];
        if (p.gated) q[p.F] = ((red[1][0][o] + red[1][1][o]) + red[1][2][o]) + red[1][3][o];
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// What a launch of the tile kernel takes, in us, as measured on an MI355X. A step of 64 k costs, with one work-group
// per CU and with two (heights 1 and 2; the taller take a CU each), by where the weights come from:
//   height (of 32 rows)   1            2            4      8
//   as stored             0.62 / 0.96  0.75 / 1.27  1.00   1.66
//   decoded before        0.38 / 0.74  0.51 / 0.97  0.80   1.47
//   turned                0.83 / 1.09  0.85 / 1.35  1.09   1.78
// on top of 6, 8, 13 and 15 per work-group (launch, first loads, epilogue), and slices of K cost 4 and 8 bytes per
// sum at 4 TB/s.
constexpr int kHeights[4] = {1, 2, 4, 8};
constexpr double kFixed[4] = {6.0, 8.0, 13.0, 15.0};
constexpr double kLaunch = 3.0;  // a launch more

double tile_us(int src, int h, int64_t groups, double steps) {
    static constexpr double kAlone[3][4] = {{0.62, 0.75, 1.00, 1.66}, {0.38, 0.51, 0.80, 1.47}, {0.83, 0.85, 1.09, 1.78}};
    static constexpr double kPaired[3][2] = {{0.96, 1.27}, {0.74, 0.97}, {1.09, 1.35}};
    const double alone = kFixed[h] + steps * kAlone[src][h];
    if (h >= 2) return (double)ceil_div(groups, 256) * alone;
    const double paired = kFixed[h] + steps * kPaired[src][h];
    const int64_t rest = groups % 512;
    return (double)(groups / 512) * paired + (rest > 256 ? paired : rest > 0 ? alone : 0.0);
}

// The height (kHeights[h0] at least) and the K split of the least estimated time for `tn` columns of tiles, whose
// sums have n values a row.
TileCut cut_tiles(int64_t M, int64_t L, int64_t tn, int64_t n, int src, int h0) {
    const int64_t pairs = ceil_div(L, 2 * kStep);
    TileCut best = {};
    for (int h = h0; h < 4; ++h) {
        const int64_t tm = ceil_div(M, 32 * kHeights[h]);
        for (int64_t want = 1; want <= 16 && want <= pairs; ++want) {
            const int64_t per = ceil_div(pairs, want);
            if (ceil_div(pairs, per) != want) continue;
            const double sums = (double)want * (double)M * (double)n;
            if (want > 1 && sums * sizeof(float) > (double)((int64_t)1 << 30)) break;
            double t = tile_us(src, h, tm * tn * want, 2.0 * (double)per);
            if (want > 1) t += 4.0 + sums * 8.0 / 4.0e6;
            if (best.mt == 0 || t < best.us) best = {kHeights[h], tn, want, per * 2 * kStep, t};
        }
    }
    return best;
}

// The tiles of an [M] x [F] output over a sum of length L: all columns of tiles alike, or, where the last round of
// work-groups would be short, the columns of the whole rounds and the rest of them as launches of their own, the
// rest lower or with K split (3000 x 11008 x 4096 is 516 of the tallest tiles: 325 us with the third round's in half the
// height, 249 us with 504 of them in two rounds and the last column's K split; 1500 x 11008 x 4096: 203 and 132 us).
LinPlan plan_tile(int64_t M, int64_t L, int64_t F, int64_t N, bool gated, int src, int h0 = 0) {
    const int64_t cols = gated ? 128 : 256, tn = ceil_div(F, cols), per_col = gated ? 2 : 1;
    const double steps = 2.0 * (double)ceil_div(L, 2 * kStep);
    LinPlan best = {};
    best.main = cut_tiles(M, L, tn, N, src, h0);
    best.us = best.main.us;
    for (int h = h0; h < 4; ++h) {
        const int64_t tm = ceil_div(M, 32 * kHeights[h]);
        for (int64_t slots = 256; slots <= (h < 2 ? 512 : 256); slots *= 2) {
            const int64_t whole = tm * tn / slots * slots / tm;  // columns of the whole rounds
            if (whole == 0 || whole == tn) continue;
            const double us = kLaunch + tile_us(src, h, tm * whole, steps);
            if (us >= best.us) continue;
            const TileCut rest = cut_tiles(M, L, tn - whole, (F - whole * cols) * per_col, src, h0);
            if (us + rest.us >= best.us) continue;
            best.us = us + rest.us;
            best.main = {kHeights[h], whole, 1, ceil_div(L, 2 * kStep) * 2 * kStep, us};
            best.rest = rest;
        }
    }
    const int64_t rest_n = (F - (best.rest.mt ? best.main.tiles_n * cols : 0)) * per_col;
    const TileCut &split = best.rest.mt ? best.rest : best.main;  // where there is a rest, K is whole before it
    best.part_bytes = split.slices > 1 ? align256((size_t)(split.slices * M * rest_n) * sizeof(float)) : 0;
    return best;
}

// What decoding the weights before costs, in us: 2.56 bytes a weight at 4.4 TB/s, and a launch.
double decode_us(int64_t N, int64_t K) { return 3.0 + (double)N * (double)K * (2.5625 / 4.4e6); }

template <int SRC, int EPI>
hipError_t tile_launch_height(const LinArgs &p, int mt, int64_t slices, hipStream_t st) {
    const dim3 grid((unsigned)(p.tiles * slices)), block(kTileThreads);
    if constexpr (SRC == kSrcFrag && EPI != kEpiPlain) {  // the forward of many rows: tall tiles alone
        if (mt == 4)
            hipLaunchKernelGGL((k_lin_tile<4, SRC, EPI>), grid, block, 0, st, p);
        else if (mt == 8)
            hipLaunchKernelGGL((k_lin_tile<8, SRC, EPI>), grid, block, 0, st, p);
        else
            return hipErrorInvalidValue;
    } else {
        switch (mt) {
            case 1: hipLaunchKernelGGL((k_lin_tile<1, SRC, EPI>), grid, block, 0, st, p); break;
            case 2: hipLaunchKernelGGL((k_lin_tile<2, SRC, EPI>), grid, block, 0, st, p); break;
            case 4: hipLaunchKernelGGL((k_lin_tile<4, SRC, EPI>), grid, block, 0, st, p); break;
            default: hipLaunchKernelGGL((k_lin_tile<8, SRC, EPI>), grid, block, 0, st, p); break;
        }
    }
    return hipGetLastError();
}

// The columns of tiles [first, first + cut.tiles_n), and the sum of their slices where K is split.
template <int SRC, int EPI>
hipError_t tile_launch_cut(LinArgs p, const TileCut &cut, int64_t first, hipStream_t st) {
    constexpr int64_t cols = EPI == kEpiGated ? 128 : 256;
    const int64_t tm = ceil_div(p.M, 32 * cut.mt);
    p.tn0 = first, p.tiles_n = (unsigned)cut.tiles_n, p.tiles_m = (unsigned)tm, p.tiles = (unsigned)(tm * cut.tiles_n);
    p.kslice = cut.kslice;
    const int64_t f0 = first * cols, f = std::min(p.F, (first + cut.tiles_n) * cols) - f0;
    p.part_n = EPI == kEpiGated ? 2 * f : f;
    p.part = cut.slices > 1 ? p.part - f0 : nullptr;
    hipError_t err = tile_launch_height<SRC, EPI>(p, cut.mt, cut.slices, st);
    if (err == hipSuccess && cut.slices > 1) {
        const int64_t per_row = ceil_div(f, kMxBlock) * 4, groups = p.M * per_row;
        const dim3 rg((unsigned)std::min<int64_t>(ceil_div(groups, kReduceThreads), 4096));
        if (p.F % 8 == 0)
            hipLaunchKernelGGL((k_lin_reduce<EPI, true>), rg, dim3(kReduceThreads), 0, st, p, (int)cut.slices, f0, per_row, groups);
        else
            hipLaunchKernelGGL((k_lin_reduce<EPI, false>), rg, dim3(kReduceThreads), 0, st, p, (int)cut.slices, f0, per_row, groups);
        err = hipGetLastError();
    }
    return err;
}

template <int SRC, int EPI>
hipError_t tile_launch_as(const LinArgs &p, const LinPlan &plan, hipStream_t st) {
    const hipError_t err = tile_launch_cut<SRC, EPI>(p, plan.main, 0, st);
    return err != hipSuccess || plan.rest.mt == 0 ? err : tile_launch_cut<SRC, EPI>(p, plan.rest, plan.main.tiles_n, st);
}

template <int SRC>
hipError_t tile_launch(const LinArgs &p, const LinPlan &plan, hipStream_t st) {
    if constexpr (SRC != kSrcTurn) {
        if (p.gated) return tile_launch_as<SRC, kEpiGated>(p, plan, st);
        if (p.bias || p.res || p.act != kActNone || p.keep != kKeepNone || p.y_f32)
            return tile_launch_as<SRC, kEpiFull>(p, plan, st);
    }
    return tile_launch_as<SRC, kEpiPlain>(p, plan, st);
}

template <int NT, int WAVES>
hipError_t skinny_launch_as(LinArgs p, void *ws, hipStream_t st) {
    const dim3 grid((unsigned)ceil_div(p.F, 16)), block(64 * WAVES);
    if (p.M <= kDirectRows) {
        if (p.x_mx)
            hipLaunchKernelGGL((k_lin_skinny<1, NT, false, true, WAVES>), grid, block, 0, st, p);
        else
            hipLaunchKernelGGL((k_lin_skinny<1, NT, false, false, WAVES>), grid, block, 0, st, p);
        return hipGetLastError();
    }
    const int64_t mt = ceil_div(p.M, 16);
    const dim3 xgrid((unsigned)ceil_div(p.L, kChunk), (unsigned)mt);
    if (p.x_mx)
        hipLaunchKernelGGL(k_lin_xfrag<true>, xgrid, dim3(256), 0, st, p, static_cast<uint16_t *>(ws));
    else
        hipLaunchKernelGGL(k_lin_xfrag<false>, xgrid, dim3(256), 0, st, p, static_cast<uint16_t *>(ws));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    p.wt = static_cast<const uint16_t *>(ws);
    if (mt == 1)
        hipLaunchKernelGGL((k_lin_skinny<1, NT, true, false, WAVES>), grid, block, 0, st, p);
    else if (mt == 2)
        hipLaunchKernelGGL((k_lin_skinny<2, NT, true, false, WAVES>), grid, block, 0, st, p);
    else if constexpr (NT == 1 || WAVES == 8) {  // skinny_launch gives six tiles and more to 8 waves
        if (mt == 3)
            hipLaunchKernelGGL((k_lin_skinny<3, NT, true, false, WAVES>), grid, block, 0, st, p);
        else
            hipLaunchKernelGGL((k_lin_skinny<4, NT, true, false, WAVES>), grid, block, 0, st, p);
    }
    return hipGetLastError();
}

// Waves per work-group: 16 while the work-groups are few (one or two a CU), so that enough loads are in flight; 8
// where there are more, which spend less on joining their sums (M = 1: 4096 x 4096 5.0 us with 16, 5.3 with 8;
// 22016 x 4096 gated 19.5 and 14.9), and where the accumulators of six or more tiles would not fit the
// registers of 16 (M = 64, 22016 x 4096 gated: 71 and 31 us).
template <int NT>
hipError_t skinny_launch(const LinArgs &p, void *ws, hipStream_t st) {
    return ceil_div(p.F, 16) > 512 || NT * ceil_div(p.M, 16) >= 6 ? skinny_launch_as<NT, 8>(p, ws, st)
                                                                 : skinny_launch_as<NT, 16>(p, ws, st);
}

struct GradPlan {
    LinPlan tile;
    bool turn;  // the weights turned in the product, not decoded before
    int64_t chunk, chunks;
    size_t wt_bytes, sum_bytes;
};

GradPlan plan_grad(int64_t M, int64_t K, int64_t N, int64_t F, bool bias) {
    GradPlan g = {};
    g.tile = plan_tile(M, N, K, K, false, kSrcFrag);
    if (K >= 64) {  // kSrcTurn's reads of 64 columns' scales
        const LinPlan turned = plan_tile(M, N, K, K, false, kSrcTurn);
        g.turn = turned.us < g.tile.us + decode_us(N, K);
        if (g.turn) g.tile = turned;
    }
    g.wt_bytes = g.turn ? 0 : align256((size_t)(ceil_div(K, 32) * ceil_div(N, kStep)) * 4096);
    g.chunk = std::max<int64_t>(bias ? 16 : 4, ceil_div(M * ceil_div(F, 512), 2048));
    g.chunk = std::max(g.chunk, ceil_div(M, 65535));
    g.chunks = ceil_div(M, g.chunk);
    g.sum_bytes = bias ? align256((size_t)(g.chunks * N) * sizeof(float)) : 0;
    return g;
}

}  // namespace

LinPlan plan_linear(int64_t M, int64_t K, int64_t N, bool x_mx, bool gated, int keep) {
    // The skinny kernel (main.mt = 0) to the most rows that it has tiles for: there it is still ahead of the tile kernel
    // (4096 x 4096: 64 rows 13.0 us, 65 rows in tiles 20.3; gated 22016 x 4096, 64 rows: 33.6 and 40.4). Its epilogue has no 32
    // columns of a row together, so a z kept in MXFP8 takes the tile kernel (gated 22016 x 4096, 1 row: 27.1 us, with z
    // in bf16 15.7; 24 rows: 29.9 and 22.5).
    if (M <= kSkinnyMaxM && keep != kKeepMx) {
        LinPlan p = {};
        if (M > kDirectRows) p.frag_bytes = (size_t)(ceil_div(K, kChunk) * ceil_div(M, 16)) * 4096;
        return p;
    }
    const int64_t F = gated ? N / 2 : N;
    LinPlan p = plan_tile(M, K, F, N, gated, kSrcCodes);
    if (M > 1024) {  // the decoding is paid back by many tiles of rows (4096 x 4096 weights: from about 2300 rows) or not at all
        const LinPlan q = plan_tile(M, K, F, N, gated, kSrcFrag, 2);
        if (q.us + decode_us(N, K) < p.us) {
            p = q;
            p.frag_bytes = (size_t)(ceil_div(F, 32) * (gated ? 2 : 1) * ceil_div(K, kStep)) * 4096;
        }
    }
    if (x_mx) p.x_bytes = align256((size_t)(M * K) * 2);
    return p;
}

hipError_t launch_linear(const LinArgs &args, void *ws, hipStream_t stream) {
    const LinPlan plan = plan_linear(args.M, args.L, args.N, args.x_mx, args.gated, args.keep);
    LinArgs p = args;
    if (plan.main.mt == 0) {
        return p.gated ? skinny_launch<2>(p, ws, stream) : skinny_launch<1>(p, ws, stream);
    }
    uint8_t *base = static_cast<uint8_t *>(ws);
    if (plan.x_bytes) {  // an MXFP8 X is decoded once, not by every work-group that reads it
        const hipError_t err = launch_mx_dequantize(static_cast<const uint8_t *>(p.x), p.ldx, p.xs, p.M, p.L, base, false, stream);
        if (err != hipSuccess) return err;
        p.x = base, p.ldx = p.L, p.x_mx = 0;
        base += plan.x_bytes;
    }
    if (plan.frag_bytes) {
        p.wt = reinterpret_cast<uint16_t *>(base);
        const dim3 grid((unsigned)ceil_div(p.F, 32), (unsigned)ceil_div(p.L, 16 * kStep), p.gated ? 2 : 1);
        hipLaunchKernelGGL(k_lin_decode, grid, dim3(256), 0, stream, p.codes, p.scales, p.F, p.L, reinterpret_cast<uint16_t *>(base));
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        p.part = reinterpret_cast<float *>(base + plan.frag_bytes);
        return tile_launch<kSrcFrag>(p, plan, stream);
    }
    p.part = reinterpret_cast<float *>(base);
    return tile_launch<kSrcCodes>(p, plan, stream);
}

size_t linear_grad_workspace(int64_t M, int64_t K, int64_t N, int64_t F, bool bias) {
    if (M == 0) return 0;
    const GradPlan g = plan_grad(M, K, N, F, bias);
    return g.wt_bytes + g.sum_bytes + g.tile.part_bytes;
}

hipError_t launch_linear_grad(const LinGradArgs &g, const uint8_t *codes, const uint8_t *scales, const float *alpha,
                              int64_t K, void *dx, float *dbias, void *ws, hipStream_t stream) {
    if (g.M == 0) return dbias ? launch_column_sum(nullptr, 0, g.N, dbias, stream) : hipSuccess;
    const GradPlan plan = plan_grad(g.M, K, g.N, g.F, dbias != nullptr);
    uint8_t *base = static_cast<uint8_t *>(ws);
    uint16_t *wt = reinterpret_cast<uint16_t *>(base);
    float *sums = reinterpret_cast<float *>(base + plan.wt_bytes);
    float *part = reinterpret_cast<float *>(base + plan.wt_bytes + plan.sum_bytes);
    hipError_t err = hipSuccess;
    if (g.act != kActNone || dbias) {
        const dim3 grid((unsigned)ceil_div(g.F, 512), (unsigned)plan.chunks);
        if (g.z_mx)
            hipLaunchKernelGGL(k_lin_dz<true>, grid, dim3(256), 0, stream, g, plan.chunk, dbias ? sums : nullptr);
        else
            hipLaunchKernelGGL(k_lin_dz<false>, grid, dim3(256), 0, stream, g, plan.chunk, dbias ? sums : nullptr);
        err = hipGetLastError();
        if (err == hipSuccess && dbias) err = launch_column_sum(sums, plan.chunks, g.N, dbias, stream);
    }
    if (err != hipSuccess) return err;
    if (!plan.turn) {
        const dim3 grid((unsigned)ceil_div(K, 256), (unsigned)ceil_div(g.N, kStep));
        hipLaunchKernelGGL(k_lin_transpose, grid, dim3(256), 0, stream, codes, scales, g.N, K, wt);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    LinArgs p = {};
    p.x = g.act == kActNone ? g.dy : g.dz;
    p.ldx = g.act == kActNone ? g.lddy : g.N;
    p.M = g.M, p.L = g.N, p.N = K, p.F = K;
    p.alpha = alpha;
    p.y = dx;
    p.wt = wt, p.codes = codes, p.scales = scales;
    p.part = part;
    return plan.turn ? tile_launch<kSrcTurn>(p, plan.tile, stream) : tile_launch<kSrcFrag>(p, plan.tile, stream);
}

}  // namespace nvfp4
