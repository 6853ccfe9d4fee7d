// gfx950 kernels of the root-mean-square norm with the residual's addition, its gradient, and the MXFP8
// form (mx.hpp) as an operation of its own.
//
// Norm of a row x (with residual r, or r = 0), weights w, n columns:
//     h = x + r,   q = (sum h^2 / n + eps)^(-1/2),   y = h q w.
// Gradient at h of a loss with gradients dy at y and dh at h (0 where there is none):
//     dx = q (w dy) - h q^3 (sum w dy h) / n + dh,   dw = sum over rows of dy h q.
// All of it is binary32 on the values as read; each output is rounded once, to its own type. h is used
// unrounded for y and stored rounded.
//
// Both are streams: a row is read once into registers (eight consecutive columns per thread and step, 16
// bytes of bf16), its sums go through one reduction, and the outputs are formed from the registers. The
// row's group of threads is chosen by the row's length, see norm_config and norm_grad_config.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "codec.hpp"
#include "launch.hpp"
#include "mx.hpp"

namespace nvfp4 {

namespace {

constexpr int kWave = 64;

// Sum over a group of ROWT threads (a wave, or a whole work-group of ROWT), the same in every thread. The
// waves' sums are added in wave order; `slot` is LDS of ROWT / 64 floats that no other reduction in flight
// uses.
template <int ROWT>
__device__ __forceinline__ float group_sum(float x, float *slot, int tid) {
    x = wave_sum_f32(x);
    x = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), kWave - 1));
    if (ROWT == kWave) return x;
    if ((tid & (kWave - 1)) == 0) slot[tid / kWave] = x;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < ROWT / kWave; ++w) s += slot[w];
    return s;
}

template <int ROWT>
__device__ __forceinline__ float2 group_sum2(float x, float y, float2 *slot, int tid) {
    x = wave_sum_f32(x);
    y = wave_sum_f32(y);
    x = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), kWave - 1));
    y = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(y), kWave - 1));
    if (ROWT == kWave) return make_float2(x, y);
    if ((tid & (kWave - 1)) == 0) slot[tid / kWave] = make_float2(x, y);
    __syncthreads();
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < ROWT / kWave; ++w) s.x += slot[w].x, s.y += slot[w].y;
    return s;
}

// (sum h^2 / n + eps)^(-1/2), by the IEEE square root and divisions.
__device__ __forceinline__ float rms_rcp(float ss, int64_t cols, float eps) {
    return 1.0f / __builtin_sqrtf(ss / (float)cols + eps);
}

__device__ __forceinline__ void load_w8(const NormArgs &p, int64_t e, int n, float w[8]) {
    if (p.w_f32) {
        Raw8<float> r;
        r.load(static_cast<const float *>(p.w) + e, n);
        r.get(w);
    } else {
        Raw8<uint16_t> r;
        r.load(static_cast<const uint16_t *>(p.w) + e, n);
        r.get(w);
    }
}

__device__ __forceinline__ int valid8(int64_t cols, int64_t e) {
    const int64_t n = cols - e;
    return n >= 8 ? 8 : n > 0 ? (int)n : 0;
}

// y of eight columns to the output's type. All four lanes of a quad call it (MXFP8 takes their maximum).
__device__ __forceinline__ void put_y(const NormArgs &p, int64_t row, int64_t e, int n, const float y[8], int lane) {
    if (p.out == kOutMx) {
        const int64_t nb = (p.cols + kMxBlock - 1) / kMxBlock;
        mx_put8(static_cast<uint8_t *>(p.y) + row * p.cols + e, p.ys + row * nb + e / kMxBlock, y, n, lane);
    } else if (p.out == kOutF32) {
        put8(static_cast<float *>(p.y) + row * p.cols + e, y, n);
    } else {
        put8(static_cast<uint16_t *>(p.y) + row * p.cols + e, y, n);
    }
}

// ---------------------------------------------------------------------------------------------- norm

// ROWT threads hold a row of at most ROWT * VPT * 8 columns in registers; work-groups of max(ROWT, 256)
// threads, so with ROWT = 64 a work-group takes four rows, a wave each.
template <typename T, int ROWT, int VPT>
__global__ __launch_bounds__(ROWT < 256 ? 256 : ROWT) void k_rms_norm(NormArgs p) {
    __shared__ float slot[ROWT / kWave];
    constexpr int kRows = ROWT < 256 ? 256 / ROWT : 1;
    const int tid = threadIdx.x % ROWT;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / ROWT;
    if (row >= p.rows) return;  // whole waves, and only where rows have a wave each
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *r = static_cast<const T *>(p.r) + row * p.ldr;
    Raw8<T> xv[VPT], rv[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t e = 8 * (int64_t)(v * ROWT + tid);
        xv[v].load(x + e, valid8(p.cols, e));
    }
    if (p.r)
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t e = 8 * (int64_t)(v * ROWT + tid);
            rv[v].load(r + e, valid8(p.cols, e));
        }
    float w[VPT][8], h[VPT][8], ss = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t e = 8 * (int64_t)(v * ROWT + tid);
        load_w8(p, e, valid8(p.cols, e), w[v]);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        xv[v].get(h[v]);
        if (p.r) {
            float t[8];
            rv[v].get(t);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] += t[i];
            const int64_t e = 8 * (int64_t)(v * ROWT + tid);
            put8(static_cast<T *>(p.h) + row * p.cols + e, h[v], valid8(p.cols, e));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(h[v][i], h[v][i], ss);
    }
    const float q = rms_rcp(group_sum<ROWT>(ss, slot, tid), p.cols, p.eps);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t e = 8 * (int64_t)(v * ROWT + tid);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = h[v][i] * q * w[v][i];
        put_y(p, row, e, valid8(p.cols, e), y, tid);
    }
}

constexpr int kLongThreads = 1024;

// Rows longer than the registers hold: read twice (the second time from the caches). The sum h is stored
// in the second pass, so h may be written over r.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void k_rms_norm_long(NormArgs p) {
    __shared__ float slot[kLongThreads / kWave];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *r = static_cast<const T *>(p.r) + row * p.ldr;
    const int64_t padded = (p.cols + kMxBlock - 1) / kMxBlock * kMxBlock;  // whole quads
    auto row8 = [&](int64_t e, int n, float h[8]) {
        Raw8<T> a, b;
        a.load(x + e, n);
        if (p.r) b.load(r + e, n);
        a.get(h);
        if (p.r) {
            float t[8];
            b.get(t);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] += t[i];
        }
    };
    float ss = 0.0f;
    for (int64_t e = 8 * (int64_t)tid; e < p.cols; e += 8 * kLongThreads) {
        float h[8];
        row8(e, valid8(p.cols, e), h);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(h[i], h[i], ss);
    }
    const float q = rms_rcp(group_sum<kLongThreads>(ss, slot, tid), p.cols, p.eps);
    for (int64_t e = 8 * (int64_t)tid; e < padded; e += 8 * kLongThreads) {
        const int n = valid8(p.cols, e);
        float h[8], w[8], y[8];
        row8(e, n, h);
        load_w8(p, e, n, w);
        if (p.r) put8(static_cast<T *>(p.h) + row * p.cols + e, h, n);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = h[i] * q * w[i];
        put_y(p, row, e, n, y, tid);
    }
}

// ------------------------------------------------------------------------------------------ gradient

// The gradient's row h: plain, or MXFP8.
template <typename T, bool MX>
struct RawH8;
template <typename T>
struct RawH8<T, false> : Raw8<T> {
    __device__ __forceinline__ void fetch(const NormArgs &p, int64_t row, int64_t e, int n) {
        this->load(static_cast<const T *>(p.x) + row * p.ldx + e, n);
    }
};
template <typename T>
struct RawH8<T, true> : RawMx8 {
    __device__ __forceinline__ void fetch(const NormArgs &p, int64_t row, int64_t e, int n) {
        const int64_t nb = (p.cols + kMxBlock - 1) / kMxBlock;
        load(static_cast<const uint8_t *>(p.x) + row * p.ldx + e, p.xs + row * nb + e / kMxBlock, n);
    }
};

// A group of ROWT threads takes the rows g, g + groups, ...; each thread keeps its columns' weights and
// their gradient's sums in registers over all of them and writes the sums as one row of `part` (added in
// order by k_column_sum, so the result does not depend on timing). The next row's loads are in flight
// while this row's sums are reduced; the LDS slots alternate, so a row costs one barrier.
template <typename T, bool MX, int ROWT, int VPT>
__global__ __launch_bounds__(ROWT < 256 ? 256 : ROWT) void k_rms_norm_grad(NormArgs p, float *__restrict__ part,
                                                                          int64_t groups) {
    __shared__ float2 slot[2][ROWT / kWave];
    constexpr int kRows = ROWT < 256 ? 256 / ROWT : 1;
    const int tid = threadIdx.x % ROWT;
    const int64_t group = (int64_t)blockIdx.x * kRows + threadIdx.x / ROWT;
    if (group >= groups) return;  // whole waves, and only where groups are waves
    RawH8<T, MX> hv[VPT];
    Raw8<T> gv[VPT], dv[VPT];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t e = 8 * (int64_t)(v * ROWT + tid);
            const int n = valid8(p.cols, e);
            hv[v].fetch(p, row, e, n);
            gv[v].load(static_cast<const T *>(p.dy) + row * p.lddy + e, n);
            if (p.r) dv[v].load(static_cast<const T *>(p.r) + row * p.ldr + e, n);
        }
    };
    // the next row in flight, unless its registers are needed (fp32 rows of 16 KB and more)
    constexpr bool kAhead = !(ROWT == 1024 && sizeof(T) == 4);
    if (kAhead) fetch(group);
    float w[VPT][8], dw[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t e = 8 * (int64_t)(v * ROWT + tid);
        load_w8(p, e, valid8(p.cols, e), w[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = group; row < p.rows; row += groups, turn ^= 1) {
        if (!kAhead) fetch(row);
        RawH8<T, MX> h0[VPT];
        Raw8<T> g0[VPT], d0[VPT];
        float ss = 0.0f, gh = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            h0[v] = hv[v], g0[v] = gv[v], d0[v] = dv[v];
            float h[8], g[8];
            h0[v].get(h);
            g0[v].get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = __builtin_fmaf(h[i], h[i], ss);
                gh = __builtin_fmaf(g[i] * w[v][i], h[i], gh);
            }
        }
        if (kAhead && row + groups < p.rows) fetch(row + groups);
        const float2 s = group_sum2<ROWT>(ss, gh, slot[turn], tid);
        const float q = rms_rcp(s.x, p.cols, p.eps);
        const float c = q * q * (s.y / (float)p.cols);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int64_t e = 8 * (int64_t)(v * ROWT + tid);
            float h[8], g[8], d[8], o[8];
            if (ROWT == 1024) {  // 128 registers a thread: the row stays in its memory form over the reduction
                h0[v].again();
                g0[v].again();
            }
            h0[v].get(h);
            g0[v].get(g);
            if (p.r) d0[v].get(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = q * __builtin_fmaf(-h[i], c, g[i] * w[v][i]);
                if (p.r) o[i] += d[i];
                dw[v][i] = __builtin_fmaf(g[i], h[i] * q, dw[v][i]);
            }
            put8(static_cast<T *>(p.y) + row * p.cols + e, o, valid8(p.cols, e));
        }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int64_t e = 8 * (int64_t)(v * ROWT + tid);
        put8(part + group * p.cols + e, dw[v], valid8(p.cols, e));
    }
}

// Rows longer than the registers hold: dx by three reads of a row, its q to `qrow`; then dw by columns.
template <typename T, bool MX>
__global__ __launch_bounds__(kLongThreads) void k_rms_norm_grad_long(NormArgs p, float *__restrict__ qrow) {
    __shared__ float2 slot[kLongThreads / kWave];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    auto row8 = [&](int64_t e, int n, float h[8], float g[8], float w[8]) {
        RawH8<T, MX> hv;
        Raw8<T> gv;
        hv.fetch(p, row, e, n);
        gv.load(static_cast<const T *>(p.dy) + row * p.lddy + e, n);
        load_w8(p, e, n, w);
        hv.get(h);
        gv.get(g);
    };
    float ss = 0.0f, gh = 0.0f;
    for (int64_t e = 8 * (int64_t)tid; e < p.cols; e += 8 * kLongThreads) {
        float h[8], g[8], w[8];
        row8(e, valid8(p.cols, e), h, g, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ss = __builtin_fmaf(h[i], h[i], ss);
            gh = __builtin_fmaf(g[i] * w[i], h[i], gh);
        }
    }
    const float2 s = group_sum2<kLongThreads>(ss, gh, slot, tid);
    const float q = rms_rcp(s.x, p.cols, p.eps);
    const float c = q * q * (s.y / (float)p.cols);
    if (tid == 0) qrow[row] = q;
    for (int64_t e = 8 * (int64_t)tid; e < p.cols; e += 8 * kLongThreads) {
        const int n = valid8(p.cols, e);
        float h[8], g[8], w[8], d[8], o[8];
        row8(e, n, h, g, w);
        if (p.r) {
            Raw8<T> dv;
            dv.load(static_cast<const T *>(p.r) + row * p.ldr + e, n);
            dv.get(d);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i] = q * __builtin_fmaf(-h[i], c, g[i] * w[i]);
            if (p.r) o[i] += d[i];
        }
        put8(static_cast<T *>(p.y) + row * p.cols + e, o, n);
    }
}

// The sums of dy h q over a chunk of rows, for 2048 columns per work-group: one row of `part` per chunk.
template <typename T, bool MX>
__global__ __launch_bounds__(256) void k_rms_norm_dw_long(NormArgs p, const float *__restrict__ qrow, int64_t chunk,
                                                        float *__restrict__ part) {
    const int64_t e = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    const int n = valid8(p.cols, e);
    if (n == 0) return;
    const int64_t r0 = (int64_t)blockIdx.y * chunk, r1 = min(p.rows, r0 + chunk);
    float dw[8] = {};
    for (int64_t row = r0; row < r1; ++row) {
        RawH8<T, MX> hv;
        Raw8<T> gv;
        hv.fetch(p, row, e, n);
        gv.load(static_cast<const T *>(p.dy) + row * p.lddy + e, n);
        const float q = qrow[row];
        float h[8], g[8];
        hv.get(h);
        gv.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] = __builtin_fmaf(g[i], h[i] * q, dw[i]);
    }
    put8(part + (int64_t)blockIdx.y * p.cols + e, dw, n);
}

// out[c] = sum over `rows` rows of part[.][c], in a fixed order: a work-group takes 32 columns, its 32 half-waves
// every 32nd row each, and their sums are added in that order (1024 x 4096: 3.5 us; with 64 columns and four
// waves, 64 work-groups, 11 us). No rows: zeros. The grid's x and y count the groups of 32 columns together: a dimension
// holds fewer than 2^32 threads, 2^27 columns.
__global__ __launch_bounds__(1024) void k_column_sum(const float *__restrict__ part, int64_t rows, int64_t cols,
                                                    float *__restrict__ out) {
    __shared__ float s[32][32];
    const int lane = threadIdx.x & 31, h = threadIdx.x >> 5;
    const int64_t c = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 32 + lane;
    float a = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t r = h; r < rows; r += 32) a += part[r * cols + c];
    }
    s[h][lane] = a;
    __syncthreads();
    if (h == 0 && c < cols) {
        float t = s[0][lane];
#pragma unroll
        for (int i = 1; i < 32; ++i) t += s[i][lane];
        out[c] = t;
    }
}

// --------------------------------------------------------------------------------------------- codec

// Eight values per thread, four threads per 32-value block; rows are padded to whole blocks. U: the type
// that indexes the groups of eight.
template <typename T, typename U>
__global__ __launch_bounds__(256) void k_mx_quantize(const T *__restrict__ x, int64_t ldx, U groups, U per_row,
                                                    int64_t cols, uint8_t *__restrict__ codes,
                                                    uint8_t *__restrict__ scales) {
    const U g = (U)blockIdx.x * 256u + threadIdx.x;
    if (g >= groups) return;  // whole quads: `groups` is a multiple of four
    const U row = g / per_row, v = g - row * per_row;
    const int64_t e = 8 * (int64_t)v;
    const int n = valid8(cols, e);
    Raw8<T> r;
    r.load(x + (int64_t)row * ldx + e, n);
    float f[8];
    r.get(f);
    mx_put8(codes + (int64_t)row * cols + e, scales + (int64_t)(g >> 2), f, n, (int)threadIdx.x);
}

template <typename T, typename U>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t *__restrict__ codes, int64_t ldc,
                                                      const uint8_t *__restrict__ scales, U groups, U per_row,
                                                      int64_t cols, T *__restrict__ y) {
    const U g = (U)blockIdx.x * 256u + threadIdx.x;
    if (g >= groups) return;
    const U row = g / per_row, v = g - row * per_row;
    const int64_t e = 8 * (int64_t)v;
    const int n = valid8(cols, e);
    if (n == 0) return;
    RawMx8 r;
    r.load(codes + (int64_t)row * ldc + e, scales + (int64_t)(g >> 2), n);
    float f[8];
    r.get(f);
    put8(y + (int64_t)row * cols + e, f, n);
}

// Threads per row and groups of eight columns per thread. A wave per row to 1024 columns (no barrier);
// beyond, 256 threads, or 1024 where the rows are too few to fill the card and a row's latency counts.
struct NormConfig {
    int rowt, vpt;  // vpt 0: the row does not fit
};
NormConfig norm_config(int64_t rows, int64_t cols) {
    const int64_t v = (cols + 7) / 8;
    if (v <= 64) return {64, 1};
    if (v <= 128) return {64, 2};
    if (rows <= 512) return v <= 256 ? NormConfig{256, 1} : v <= 1024 ? NormConfig{1024, 1} : v <= 2048 ? NormConfig{1024, 2} : NormConfig{0, 0};
    return v <= 256 ? NormConfig{256, 1} : v <= 512 ? NormConfig{256, 2} : v <= 1024 ? NormConfig{256, 4} : v <= 2048 ? NormConfig{256, 8} : NormConfig{0, 0};
}
// The gradient holds five rows of eight per thread and step, so at most two steps per thread. 1024 threads have 128
// registers each, which two steps exceed: 40 to 52 bytes of scratch a thread for bf16, 76 to 84 for fp32 (777 x 14336
// from MXFP8: 12 MB written and 13 MB read beyond the operands' 93).
NormConfig norm_grad_config(int64_t cols) {
    const int64_t v = (cols + 7) / 8;
    if (v <= 64) return {64, 1};
    if (v <= 128) return {64, 2};
    if (v <= 256) return {256, 1};
    if (v <= 512) return {256, 2};
    if (v <= 1024) return {512, 2};
    return v <= 2048 ? NormConfig{1024, 2} : NormConfig{0, 0};
}

constexpr int64_t kLongChunk = 64;            // rows per partial sum of k_rms_norm_dw_long
constexpr int64_t kSumGridX = (int64_t)1 << 16;  // most work-groups of k_column_sum along x

int64_t norm_grad_groups(int64_t rows, int64_t cols) {
    const NormConfig c = norm_grad_config(cols);
    if (c.vpt == 0) return (rows + kLongChunk - 1) / kLongChunk;
    // As many groups as keep the card's loads in flight; each writes a row of partial sums, so no more (8192 x 4096: 512
    // groups 39 us, 1024 43; 20000 x 1000, a wave each: 2048 groups 31 us, 1024 38, 4096 39).
    return std::min<int64_t>(rows, c.rowt == 64 ? 4096 / c.vpt : c.rowt == 256 ? 1024 / c.vpt : 256);
}

template <typename T>
hipError_t norm_dispatch(const NormArgs &p, hipStream_t st) {
    const NormConfig c = norm_config(p.rows, p.cols);
    const dim3 grid((unsigned)(c.rowt == 64 ? (p.rows + 3) / 4 : p.rows));
#define NVFP4_NORM(R, V)                                                                                     \
    if (c.rowt == R && c.vpt == V) {                                                                           \
        hipLaunchKernelGGL((k_rms_norm<T, R, V>), grid, dim3(R < 256 ? 256 : R), 0, st, p);                      \
        return hipGetLastError();                                                                              \
    }
    NVFP4_NORM(64, 1)
    NVFP4_NORM(64, 2)
    NVFP4_NORM(256, 1)
    NVFP4_NORM(256, 2)
    NVFP4_NORM(256, 4)
    NVFP4_NORM(256, 8)
    NVFP4_NORM(1024, 1)
    NVFP4_NORM(1024, 2)
#undef NVFP4_NORM
    hipLaunchKernelGGL((k_rms_norm_long<T>), grid, dim3(kLongThreads), 0, st, p);
    return hipGetLastError();
}

template <typename T, bool MX>
hipError_t norm_grad_dispatch(const NormArgs &p, float *dw, float *ws, hipStream_t st) {
    const NormConfig c = norm_grad_config(p.cols);
    const int64_t groups = norm_grad_groups(p.rows, p.cols);
    bool done = p.rows == 0;
    const dim3 grid((unsigned)(c.rowt == 64 ? (groups + 3) / 4 : groups));
#define NVFP4_NORM_GRAD(R, V)                                                                                \
    if (!done && c.rowt == R && c.vpt == V) {                                                                  \
        hipLaunchKernelGGL((k_rms_norm_grad<T, MX, R, V>), grid, dim3(R < 256 ? 256 : R), 0, st, p, ws, groups);   \
        done = true;                                                                                           \
    }
    NVFP4_NORM_GRAD(64, 1)
    NVFP4_NORM_GRAD(64, 2)
    NVFP4_NORM_GRAD(256, 1)
    NVFP4_NORM_GRAD(256, 2)
    NVFP4_NORM_GRAD(512, 2)
    NVFP4_NORM_GRAD(1024, 2)
#undef NVFP4_NORM_GRAD
    if (!done) {
        float *qrow = ws + groups * p.cols;
        hipLaunchKernelGGL((k_rms_norm_grad_long<T, MX>), dim3((unsigned)p.rows), dim3(kLongThreads), 0, st, p, qrow);
        const dim3 g2((unsigned)((p.cols + 2047) / 2048), (unsigned)groups);
        hipLaunchKernelGGL((k_rms_norm_dw_long<T, MX>), g2, dim3(256), 0, st, p, qrow, kLongChunk, ws);
    }
    const hipError_t err = hipGetLastError();
    return err != hipSuccess ? err : launch_column_sum(ws, p.rows == 0 ? 0 : groups, p.cols, dw, st);
}

}  // namespace

hipError_t launch_column_sum(const float *part, int64_t rows, int64_t cols, float *out, hipStream_t stream) {
    const int64_t blocks = (cols + 31) / 32, y = (blocks + kSumGridX - 1) / kSumGridX;
    const dim3 grid((unsigned)((blocks + y - 1) / y), (unsigned)y);
    hipLaunchKernelGGL(k_column_sum, grid, dim3(1024), 0, stream, part, rows, cols, out);
    return hipGetLastError();
}

hipError_t launch_rms_norm(const NormArgs &p, bool f32, hipStream_t stream) {
    return f32 ? norm_dispatch<float>(p, stream) : norm_dispatch<uint16_t>(p, stream);
}

size_t rms_norm_grad_workspace(int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    const int64_t long_rows = norm_grad_config(cols).vpt == 0 ? rows : 0;
    return (size_t)(norm_grad_groups(rows, cols) * cols + long_rows) * sizeof(float);
}

hipError_t launch_rms_norm_grad(const NormArgs &p, bool f32, bool mx, float *dw, float *ws, hipStream_t stream) {
    if (mx) return f32 ? norm_grad_dispatch<float, true>(p, dw, ws, stream) : norm_grad_dispatch<uint16_t, true>(p, dw, ws, stream);
    return f32 ? norm_grad_dispatch<float, false>(p, dw, ws, stream) : norm_grad_dispatch<uint16_t, false>(p, dw, ws, stream);
}

hipError_t launch_mx_quantize(const void *x, bool f32, int64_t rows, int64_t cols, int64_t ldx, uint8_t *codes,
                              uint8_t *scales, hipStream_t stream) {
    const int64_t per_row = (cols + kMxBlock - 1) / kMxBlock * 4, groups = rows * per_row;
    const dim3 grid((unsigned)((groups + 255) / 256)), block(256);
    const bool small = groups < ((int64_t)1 << 31);
#define NVFP4_MXQ(T, U) \
    hipLaunchKernelGGL((k_mx_quantize<T, U>), grid, block, 0, stream, static_cast<const T *>(x), ldx, (U)groups, (U)per_row, cols, codes, scales)
    if (f32) {
        if (small) NVFP4_MXQ(float, uint32_t);
        else NVFP4_MXQ(float, uint64_t);
    } else {
        if (small) NVFP4_MXQ(uint16_t, uint32_t);
        else NVFP4_MXQ(uint16_t, uint64_t);
    }
#undef NVFP4_MXQ
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t rows, int64_t cols,
                                void *y, bool f32, hipStream_t stream) {
    const int64_t per_row = (cols + kMxBlock - 1) / kMxBlock * 4, groups = rows * per_row;
    const dim3 grid((unsigned)((groups + 255) / 256)), block(256);
    const bool small = groups < ((int64_t)1 << 31);
#define NVFP4_MXD(T, U) \
    hipLaunchKernelGGL((k_mx_dequantize<T, U>), grid, block, 0, stream, codes, ldc, scales, (U)groups, (U)per_row, cols, static_cast<T *>(y))
    if (f32) {
        if (small) NVFP4_MXD(float, uint32_t);
        else NVFP4_MXD(float, uint64_t);
    } else {
        if (small) NVFP4_MXD(uint16_t, uint32_t);
        else NVFP4_MXD(uint16_t, uint64_t);
    }
#undef NVFP4_MXD
    return hipGetLastError();
}

}  // namespace nvfp4
