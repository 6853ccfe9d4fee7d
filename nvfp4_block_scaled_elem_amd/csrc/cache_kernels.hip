// gfx950 rotary positions, and the writing of keys and values into a paged cache in 8 bits.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "cache.hpp"
#include "codec.hpp"
#include "launch.hpp"
#include "mx.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------------------------------- rotary

// Raw8's bytes in plain vectors, which stay in registers when they are assigned (uint4 went through scratch).
__device__ __forceinline__ u32x4 plain(uint4 v) { return u32x4{v.x, v.y, v.z, v.w}; }
__device__ __forceinline__ uint4 back(u32x4 v) { return make_uint4(v.x, v.y, v.z, v.w); }
struct Held16 {
    u32x4 a;
    __device__ __forceinline__ void load(const uint16_t *p, int n) {
        Raw8<uint16_t> r;
        r.load(p, n);
        a = plain(r.a);
    }
    __device__ __forceinline__ void get(float v[8]) const {
        Raw8<uint16_t> r;
        r.a = back(a);
        r.get(v);
    }
};
struct Held32 {
    u32x4 a, b;
    __device__ __forceinline__ void load(const float *p, int n) {
        Raw8<float> r;
        r.load(p, n);
        a = plain(r.a), b = plain(r.b);
    }
    __device__ __forceinline__ void get(float v[8]) const {
        Raw8<float> r;
        r.a = back(a), r.b = back(b);
        r.get(v);
    }
};
template <typename T>
using Held = typename std::conditional<sizeof(T) == 2, Held16, Held32>::type;

// y[j] = a cos t - b sin t, y[j + R/2] = b cos t + a sin t for (a, b) = (x[j], x[j + R/2]), j < R/2, with the angle
// t = pos[axis of j] base^(-2j/R); columns from R on pass. Bound by x and y (16 bytes a thread each way).
//
// The angle is formed in binary64, in turns: base^(-2j/R) = 2^(j c) with c = c_hi + c_lo, j c_hi exact, so that
// it is within a few 2^-53 of its value, which for angles to 2^27 is below binary32's step of a turn's fraction; a whole
// number of turns is dropped exactly, and what is left, at most half a turn, goes to the sine and cosine in binary32.
//
// A work-group takes p.per tokens and a share of the heads: its threads compute the tokens' sines and cosines once,
// into LDS, while the first rows are on their way, and turn the heads with them.
// WHOLE: pairs and passing columns come in whole eights.
template <typename T, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_rotary(RotaryArgs p) {
    __shared__ float2 cs[kRotaryPairs];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * p.per;
    const int tokens = (int)min((int64_t)p.per, p.tokens - t0);
    const int h0 = blockIdx.y * p.heads_per, heads = min(p.heads_per, p.heads - h0);
    const int turned = (p.half + 7) >> 3, groups = turned + p.pass;  // pieces of 8 columns (turned: 8 pairs)
    const int items = tokens * heads * groups;
    struct Item {
        Held<T> a, b;
        int t, g;
        int64_t y;
    };
    auto place = [&](Item &it, int i) __attribute__((always_inline)) {
        const int g = i % groups, th = i / groups, h = th % heads, t = th / heads;
        it.t = t, it.g = g;
        it.y = (t0 + t) * p.ys + (h0 + h) * p.yh;
        const T *x = static_cast<const T *>(p.x) + (t0 + t) * p.xs + (h0 + h) * p.xh;
        if (g < turned) {
            const int n = WHOLE ? 8 : min(8, p.half - 8 * g);
            it.a.load(x + 8 * g, n);
            it.b.load(x + p.half + 8 * g, n);
        } else {
            const int c = 2 * p.half + 8 * (g - turned);
            it.a.load(x + c, WHOLE ? 8 : min(8, p.dim - c));
            it.b = it.a;
        }
    };
    Item it;
    place(it, min(tid, items - 1));
    for (int e = tid; e < tokens * p.half; e += kThreads) {
        const int t = e / p.half, j = e % p.half;
        int axis = 0;
#pragma unroll
        for (int a = 0; a < kRotaryAxes - 1; ++a) axis += j >= p.end[a];
        const int64_t at = axis * p.pos_ld + t0 + t;
        const double pos = p.pos64 ? (double)static_cast<const int64_t *>(p.pos)[at] : (double)static_cast<const int *>(p.pos)[at];
        const double f = exp2(j * p.c_hi) * (1.0 + j * p.c_lo * 0.6931471805599453);
        const double turns = pos * (f * 0.15915494309189535);
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[e] = make_float2(c, p.inverse ? -s : s);
    }
    __syncthreads();
    for (int i = tid; i < items; i += kThreads) {
        Item next;
        place(next, min(i + kThreads, items - 1));
        T *y = static_cast<T *>(p.y) + it.y;
        float a[8], b[8];
        it.a.get(a);
        if (it.g < turned) {
            const int n = WHOLE ? 8 : min(8, p.half - 8 * it.g);
            it.b.get(b);
            float u[8], v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 w = k < n ? cs[it.t * p.half + 8 * it.g + k] : make_float2(0.0f, 0.0f);
                u[k] = __builtin_fmaf(a[k], w.x, -(b[k] * w.y));
                v[k] = __builtin_fmaf(b[k], w.x, a[k] * w.y);
            }
            put8(y + 8 * it.g, u, n);
            put8(y + p.half + 8 * it.g, v, n);
        } else {
            const int c = 2 * p.half + 8 * (it.g - turned);
            put8(y + c, a, WHOLE ? 8 : min(8, p.dim - c));
        }
        it = next;
    }
}

// ------------------------------------------------------------------------------------ cache, written

// The new tokens of one block (64 slots) of one sequence, for one head, keys (blockIdx.z = 0) or values (1):
//   e = the least power of two with max|x| <= 448 * 2^e over them, and at least the block's scale where it holds
//       earlier tokens, whose codes are then rounded to the new scale (exact but below 2^-6 of it);
//   codes = E4M3(x / 2^e), nearest, ties to even. Slots behind the sequence's end stay as they are.
// A NaN or an infinity gives the block scale byte 255 and codes 0x7F (all its tokens read as NaN), which it keeps until
// a new sequence begins in it. So does a magnitude from kBeyond = 248 * 2^120 on: the nearest code is 256 * 2^120 = 2^128, an infinity
// in binary32 and bf16, whose products with the zero probabilities of rows that do not see its token would be NaN.
//
// Bound by x, read once (a thread keeps its values between the maximum and the codes), and, for single tokens, by the chain
// of loads length -> page -> scale.
constexpr uint32_t kBeyond = 0x7F780000u;

template <typename T>
__global__ __launch_bounds__(kThreads) void k_kv_append(AppendArgs p) {
    constexpr int kMost = kPage / 4 * kMaxHeadDim / 8 / kThreads;  // pieces, four slots of 8 columns, of a thread
    constexpr int kPitch = kPage + 4;                          // of a column's 64 codes in LDS
    __shared__ uint32_t red[kThreads / 64];
    __shared__ __attribute__((aligned(16))) uint8_t tile[kMaxHeadDim * kPitch];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t head = blockIdx.y;
    const bool values = blockIdx.z != 0;
    int s = blockIdx.x, nth = 0;
    if (p.seq.starts) {
        s = piece_sequence(p.seq, blockIdx.x, 1, log2_of(kPage), 2);
        nth = (int)blockIdx.x - piece_base(p.seq, s, 1, log2_of(kPage), 2);
    }
    const Seq q = sequence(p.seq, s);
    const int begin = max(q.len - q.n, 0);  // the first new token's place; more new tokens than tokens: the first are left out
    const int block = begin / kPage + nth;
    const int lo = max(begin, block * kPage), hi = min(q.len, (block + 1) * kPage);
    if (nth < 0 || lo >= hi) return;
    const int page = page_of(p.seq, s, block);
    if (page < 0) return;
    const int n = hi - lo, slot0 = lo - block * kPage, dim = p.dim, per = dim / 8;
    const int64_t row0 = q.first + (q.n - (q.len - lo));
    const T *x = static_cast<const T *>(values ? p.v : p.k) + row0 * (values ? p.vs : p.ks) + head * (values ? p.vh : p.kh);
    const int64_t xs = values ? p.vs : p.ks;
    const int64_t at = (int64_t)page * p.heads + head;
    uint8_t *const codes = (values ? p.v_codes : p.k_codes) + at * kPage * dim;
    uint8_t *const scale = (values ? p.v_scales : p.k_scales) + at;
    const uint32_t old = slot0 ? *scale : 0u;

    // Piece e: slots 4 (slot0 / 4 + e / per) .. + 3 as far as they are the call's, columns 8 (e % per) .. + 7.
    const int quad0 = slot0 / 4, items = ((slot0 + n - 1) / 4 - quad0 + 1) * per;
    Raw8<T> raw[kMost][4];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int e = tid + i * kThreads;
        if (i * kThreads < items && e < items) {
            const int t = 4 * (quad0 + e / per) - slot0;
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[i][j].load(x + (int64_t)(t + j) * xs + 8 * (e % per), t + j >= 0 && t + j < n ? 8 : 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[8];
                raw[i][j].get(v);
                top = max(top, amax8(v));
            }
        }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    if (lane == 0) red[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) top = max(top, red[w]);
    const uint32_t sb = top >= kBeyond ? 255u : max(old, mx_scale_byte(top));
    if (tid == 0) *scale = (uint8_t)sb;  // every thread has read `old` before the barrier

    if (slot0 && sb > old) {  // the earlier tokens' codes to the larger scale
        const uint32_t down = sb - old;
        const float r = __uint_as_float(down < 127u ? (127u - down) << 23 : 0u);
        auto move4 = [&](uint32_t c) __attribute__((always_inline)) {
            if (sb == 255u) return 0x7F7F7F7Fu;
            float v[4];
            mx_decode4(c, r, v);
            int d = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
            return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], d, true);
        };
        if (!values) {
            uint32_t *c = reinterpret_cast<uint32_t *>(codes);
            for (int e = tid; e < slot0 * dim / 4; e += kThreads) c[e] = move4(c[e]);
        } else {
            const int quads = (slot0 + 3) / 4;
            for (int e = tid; e < quads * dim; e += kThreads) {
                uint8_t *c = codes + (e / quads) * kPage + 4 * (e % quads);
                const int left = slot0 - 4 * (e % quads);
                const uint32_t d = move4(*reinterpret_cast<const uint32_t *>(c));
                if (left >= 4) {
                    *reinterpret_cast<uint32_t *>(c) = d;
                } else {  // the new tokens' codes in the same dword are other threads' to write
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (i < left) c[i] = (uint8_t)(d >> (8 * i));
                }
            }
        }
    }
    const bool few = n < 4;  // values: straight to memory, byte by byte
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int e = tid + i * kThreads;
        if (i * kThreads < items && e < items) {
            const int slot = 4 * (quad0 + e / per), d = 8 * (e % per);
            uint2 c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[8];
                raw[i][j].get(v);
                c[j] = mx_encode8(v, sb);
            }
            if (!values || few) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (slot + j < slot0 || slot + j >= slot0 + n) continue;
                    if (!values) {
                        *reinterpret_cast<uint2 *>(codes + (slot + j) * dim + d) = c[j];
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            codes[(d + k) * kPage + slot + j] = (uint8_t)((k < 4 ? c[j].x : c[j].y) >> (8 * (k & 3)));
                    }
                }
            } else {  // four slots of a column in a dword
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    auto byte_of = [&](int j) { return (k < 4 ? c[j].x : c[j].y) >> (8 * (k & 3)) & 255u; };
                    *reinterpret_cast<uint32_t *>(tile + (d + k) * kPitch + slot) =
                        byte_of(0) | byte_of(1) << 8 | byte_of(2) << 16 | byte_of(3) << 24;
                }
            }
        }
    }
    if (!values || few) return;
    __syncthreads();
    for (int e = tid; e < dim * 4; e += kThreads) {  // 16 slots of a column
        const int d = e >> 2, c0 = 16 * (e & 3);
        const uint8_t *from = tile + d * kPitch + c0;
        uint8_t *to = codes + d * kPage + c0;
        const int a = max(slot0 - c0, 0), b = min(slot0 + n - c0, 16);
        if (a >= b) continue;
        const uint32_t *w = reinterpret_cast<const uint32_t *>(from);
        if (a == 0 && b == 16) {
            *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int k = a; k < b; ++k) to[k] = from[k];
        }
    }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, bool f32, hipStream_t st) {
    RotaryArgs p = a;
    p.per = (int)std::min<int64_t>({kRotaryPairs / p.half, 16, std::max<int64_t>(1, p.tokens)});
    const int64_t gx = (p.tokens + p.per - 1) / p.per;
    // Few tokens: their heads go to several work-groups, each with work for all its threads.
    const int64_t items = (int64_t)p.per * p.heads * ((p.half + 7) / 8 + p.pass);
    const int64_t want = std::min<int64_t>((512 + gx - 1) / gx, (items + kThreads - 1) / kThreads);
    const int64_t gy = std::max<int64_t>(1, std::min<int64_t>(want, p.heads));
    p.heads_per = (int)((p.heads + gy - 1) / gy);
    const dim3 grid((unsigned)gx, (unsigned)((p.heads + p.heads_per - 1) / p.heads_per));
    const bool whole = p.half % 8 == 0 && (p.dim - 2 * p.half) % 8 == 0;
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, p); };
    if (f32)
        run(whole ? k_rotary<float, true> : k_rotary<float, false>);
    else
        run(whole ? k_rotary<uint16_t, true> : k_rotary<uint16_t, false>);
    return hipGetLastError();
}

hipError_t launch_kv_append(const AppendArgs &p, bool f32, hipStream_t st) {
    const int pieces = p.seq.starts ? p.seq.tokens / kPage + 2 * p.seq.seqs : p.seq.seqs;
    const dim3 grid((unsigned)pieces, (unsigned)p.heads, 2);
    if (f32)
        hipLaunchKernelGGL(k_kv_append<float>, grid, dim3(kThreads), 0, st, p);
    else
        hipLaunchKernelGGL(k_kv_append<uint16_t>, grid, dim3(kThreads), 0, st, p);
    return hipGetLastError();
}

}  // namespace nvfp4
