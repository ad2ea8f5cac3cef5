// RMS norm of bf16 rows with the residual's addition, rounded for the next
// projection (bf16, int8 or OCP E4M3 by the token or by 128 inputs).
//
// One pass over the row: it stays in registers as the bf16 it is rounded to
// (r = bf16(x + residual)), and one reduction gives both statistics.  With
// t = r * gamma (exact in f32) and d = 1 / sqrt(mean r^2 + eps) the normalised
// value is t * d; its code for the absmax a * d is the code of t for the absmax
// a, since d cancels out of t * d * (Q / (a * d)).  So the codes wait for
// max |t| alone and only the scale, a * d / Q, takes the sum of squares.
//
// Bound by memory for many rows: 8192 x 4096 with the residual, E4M3 out,
// moves 235 MB in 42 us (5.6 TB/s; a large copy reaches 5.1), and fetches and
// writes exactly those bytes.  One row of 4096 takes 2.4 us: the call's host time
// (6.3 to 6.9 us) bounds it.  A row has the threads that hold it
// in one to four 16-byte chunks each: a wavefront up to 512 inputs (four rows
// to a workgroup), 256 threads up to 8192, 1024 up to 32768, and two passes
// over longer ones (256 rows of 131072 inputs into E4M3: 27 us, with the residual
// 61; held in registers, which spill, 68 and 105.  Of 65536 inputs, which
// registers would hold, 13.2 and 29.8 us, held 9.9 and 25.0).
#include <type_traits>

#include "layer_device.h"

namespace qlin {

namespace {

__device__ __forceinline__ v4u add8(const v4u& a, const v4u& b) {
    v4u r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = bf16_pair(bf16_lo(a[i]) + bf16_lo(b[i]), bf16_hi(a[i]) + bf16_hi(b[i]));
    return r;
}

// THREADS lanes per row, ROWS rows per workgroup (more than one only for rows
// of one wavefront); CPT 16-byte chunks of the row per thread.
constexpr int kLongThreads = 1024;

template <int THREADS, int ROWS, int CPT, int OUT>
__global__ __launch_bounds__(THREADS * ROWS) void norm_kernel(NormCall a) {
    static_assert(ROWS == 1 || THREADS == kWave, "a row of several wavefronts takes the workgroup's barrier");
    constexpr int kWaves = THREADS / kWave;
    __shared__ float red[2 * kWaves];
    const int tid = ROWS > 1 ? threadIdx.x % THREADS : threadIdx.x;
    const int64_t m = ROWS > 1 ? (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS : blockIdx.x;
    if (ROWS > 1 && m >= a.M) return;
    const int nchunks = (int)(a.K >> 3);
    const v4u* x = reinterpret_cast<const v4u*>(a.x + m * a.K);
    const v4u* res = a.residual ? reinterpret_cast<const v4u*>(a.residual + m * a.K) : nullptr;
    const v4u* gamma = reinterpret_cast<const v4u*>(a.gamma);
    const v4u zero = v4u{0, 0, 0, 0};

    v4u r[CPT], g[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
        const int c = tid + j * THREADS;
        r[j] = c < nchunks ? x[c] : zero;
        g[j] = c < nchunks ? gamma[c] : zero;
    }
    if (res) {
        v4u* sum = reinterpret_cast<v4u*>(a.sum + m * a.K);
        v4u b[CPT];
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = tid + j * THREADS;
            b[j] = c < nchunks ? res[c] : zero;
        }
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
            const int c = tid + j * THREADS;
            r[j] = add8(r[j], b[j]);
            if (c < nchunks) sum[c] = r[j];
        }
    }

    float squares = 0.0f, amax = 0.0f, group[OUT == kNormFp8Block ? CPT : 1];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
        float f[8], w[8], top = 0.0f;
        widen8(r[j], f);
        widen8(g[j], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) squares = __builtin_fmaf(f[i], f[i], squares);
        if constexpr (OUT != kNormBf16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) top = larger(top, fabsf(f[i] * w[i]));
        }
        if constexpr (OUT == kNormFp8Block) group[j] = lanes_absmax<16>(top);   // 16 chunks: 128 inputs
        else amax = larger(amax, top);
    }
    squares = wave_sum_f32(squares);
    if constexpr (OUT == kNormInt8 || OUT == kNormFp8) amax = __uint_as_float(wave_max_u32(__float_as_uint(amax)));
    if constexpr (kWaves > 1) {
        const int wave = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0) red[wave] = squares, red[kWaves + wave] = amax;
        __syncthreads();
        squares = red[0], amax = red[kWaves];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) squares += red[w], amax = larger(amax, red[kWaves + w]);
    }
    const float d = 1.0f / sqrtf(squares / (float)a.K + a.eps);

    constexpr bool kFp8 = OUT == kNormFp8 || OUT == kNormFp8Block;
    Rounding rr = {};
    if constexpr (OUT == kNormInt8 || OUT == kNormFp8) {
        rr = rounding<kFp8>(amax);
        if (tid == 0) a.s[m] = scale_of<kFp8>(amax * d);
    }
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
        const int c = tid + j * THREADS;
        if (c >= nchunks) break;
        float f[8], w[8];
        widen8(r[j], f);
        widen8(g[j], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= w[i];
        if constexpr (OUT == kNormBf16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= d;
            reinterpret_cast<v4u*>(static_cast<uint16_t*>(a.y) + m * a.K)[c] = narrow8(f);
        } else {
            if constexpr (OUT == kNormFp8Block) {
                rr = rounding<true>(group[j]);
                if (c % 16 == 0) a.s[m * (a.K / 128) + c / 16] = scale_of<true>(group[j] * d);
            }
            reinterpret_cast<v2u*>(static_cast<uint8_t*>(a.y) + m * a.K)[c] = codes8<kFp8>(f, rr);
        }
    }
}

// Rows longer than a workgroup's registers hold: read twice, the second time
// from the caches (the row, or the sum that the first pass wrote).
template <int OUT>
__global__ __launch_bounds__(kLongThreads) void norm_long_kernel(NormCall a) {
    constexpr int kWaves = kLongThreads / kWave;
    constexpr bool kFp8 = OUT == kNormFp8 || OUT == kNormFp8Block;
    __shared__ float red[2 * kWaves];
    const int tid = threadIdx.x, nchunks = (int)(a.K >> 3);
    const int64_t m = blockIdx.x;
    const v4u* x = reinterpret_cast<const v4u*>(a.x + m * a.K);
    const v4u* res = a.residual ? reinterpret_cast<const v4u*>(a.residual + m * a.K) : nullptr;
    const v4u* gamma = reinterpret_cast<const v4u*>(a.gamma);
    v4u* sum = reinterpret_cast<v4u*>(a.sum + m * a.K);
    float squares = 0.0f, amax = 0.0f;
    for (int c = tid; c < nchunks; c += kLongThreads) {
        v4u r = x[c];
        if (res) r = add8(r, res[c]), sum[c] = r;
        float f[8], w[8];
        widen8(r, f);
        widen8(gamma[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) squares = __builtin_fmaf(f[i], f[i], squares), amax = larger(amax, fabsf(f[i] * w[i]));
    }
    squares = wave_sum_f32(squares);
    amax = __uint_as_float(wave_max_u32(__float_as_uint(amax)));
    if (tid % kWave == 0) red[tid / kWave] = squares, red[kWaves + tid / kWave] = amax;
    __syncthreads();
    squares = red[0], amax = red[kWaves];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) squares += red[w], amax = larger(amax, red[kWaves + w]);
    const float d = 1.0f / sqrtf(squares / (float)a.K + a.eps);
    Rounding rr = rounding<kFp8>(amax);
    if (OUT != kNormBf16 && OUT != kNormFp8Block && tid == 0) a.s[m] = scale_of<kFp8>(amax * d);
    const v4u* row = res ? sum : x;
    const int turns = (nchunks + kLongThreads - 1) / kLongThreads;
    for (int k = 0; k < turns; ++k) {          // (whole groups of 16 lanes stay together: their maximum is taken)
        const int c = tid + k * kLongThreads;
        float f[8] = {}, w[8];
        if (c < nchunks) {
            widen8(row[c], f);
            widen8(gamma[c], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= w[i];
        }
        if constexpr (OUT == kNormFp8Block) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = larger(top, fabsf(f[i]));
            top = lanes_absmax<16>(top);
            rr = rounding<true>(top);
            if (c < nchunks && c % 16 == 0) a.s[m * (a.K / 128) + c / 16] = scale_of<true>(top * d);
        }
        if (c >= nchunks) continue;
        if constexpr (OUT == kNormBf16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= d;
            reinterpret_cast<v4u*>(static_cast<uint16_t*>(a.y) + m * a.K)[c] = narrow8(f);
        } else {
            reinterpret_cast<v2u*>(static_cast<uint8_t*>(a.y) + m * a.K)[c] = codes8<kFp8>(f, rr);
        }
    }
}

template <int OUT>
hipError_t launch_out(const NormCall& c, hipStream_t st) {
    const int64_t chunks = c.K / 8;
    auto go = [&](auto threads, auto rows, auto cpt) {
        constexpr int T = decltype(threads)::value, R = decltype(rows)::value, C = decltype(cpt)::value;
        hipLaunchKernelGGL((norm_kernel<T, R, C, OUT>), dim3((unsigned)((c.M + R - 1) / R)), dim3(T * R), 0, st, c);
    };
    using std::integral_constant;
    integral_constant<int, 1> one;
    integral_constant<int, 2> two;
    integral_constant<int, 4> four;
    integral_constant<int, 64> t64;
    integral_constant<int, 256> t256;
    integral_constant<int, 1024> t1024;
    if (chunks <= 64) go(t64, four, one);
    else if (chunks <= 256) go(t256, one, one);
    else if (chunks <= 512) go(t256, one, two);
    else if (chunks <= 1024) go(t256, one, four);
    else if (chunks <= 4096) go(t1024, one, four);
    else hipLaunchKernelGGL(norm_long_kernel<OUT>, dim3((unsigned)c.M), dim3(kLongThreads), 0, st, c);
    return hipGetLastError();
}

}  // namespace

// A launch holds 2^32 threads: many rows take several.
hipError_t launch_norm(NormOut out, const NormCall& c, hipStream_t st) {
    constexpr int64_t kRows = int64_t(1) << 21;
    const int64_t codes = out == kNormBf16 ? 2 : 1, scales = out == kNormFp8Block ? c.K / 128 : 1;
    for (int64_t m = 0; m < c.M; m += kRows) {
        NormCall part = c;
        part.M = c.M - m < kRows ? c.M - m : kRows;
        part.x += m * c.K;
        if (c.residual) part.residual += m * c.K, part.sum += m * c.K;
        part.y = static_cast<uint8_t*>(c.y) + m * c.K * codes;
        if (c.s) part.s += m * scales;
        hipError_t e;
        switch (out) {
            case kNormBf16: e = launch_out<kNormBf16>(part, st); break;
            case kNormInt8: e = launch_out<kNormInt8>(part, st); break;
            case kNormFp8: e = launch_out<kNormFp8>(part, st); break;
            default: e = launch_out<kNormFp8Block>(part, st);
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qlin
