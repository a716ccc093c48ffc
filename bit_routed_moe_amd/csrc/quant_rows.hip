// Rows to 8-bit integers with one scale each:
//   top = max |x|, scale = top / 127, code = the whole number nearest to
//   x * 127 / top (ties to even)
// The nearest whole number is decided exactly: a first guess q from an fp32
// product is within 1 of it, and the sign of |2 (127 x - q top)| - top, which
// takes no rounding (in fp32 for bf16 rows, whose products with 127 and q have
// 15 bits each; in fp64 for fp32 rows), settles it.  So codes do not depend on
// how a division is rounded.
//
// Bound by memory; a row is read once, its values stay in registers between
// the maximum and the codes (up to 4 pieces of 16 bytes per thread; what a
// longer row has beyond that is read twice).
#include "common.hpp"
#include "launch.hpp"

namespace ds4 {

namespace {

template <typename T>
struct QrVec;
template <>
struct QrVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float get(u32x4 r, int i) { return __uint_as_float(r[i]); }
};
template <>
struct QrVec<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float get(u32x4 r, int i) {
        return __uint_as_float(i & 1 ? r[i >> 1] & 0xFFFF0000u : r[i >> 1] << 16);
    }
};

// Piece c of a row; what lies behind column K reads as zero.
template <typename T>
__device__ __forceinline__ u32x4 qr_load(const T* row, int c, int K) {
    constexpr int N = QrVec<T>::N, W = sizeof(T) / 2;
    u32x4 r = *reinterpret_cast<const u32x4*>(row + (size_t)c * N);
    const int n = (K - c * N) * W;   // halves of 16 bits that exist
    if (n < 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = 2 * i + 1 < n ? r[i] : (2 * i < n ? r[i] & 0xFFFFu : 0u);
    }
    return r;
}

// The largest |value| of a piece, as fp32 bits (which order like the values;
// NaN is above infinity).
template <typename T>
__device__ __forceinline__ uint32_t qr_top(u32x4 r) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < QrVec<T>::N; ++i) m = max(m, __float_as_uint(QrVec<T>::get(r, i)) & 0x7FFFFFFFu);
    return m;
}

// The code of x; up: a power of 2 that brings top into the middle of fp32's
// range, t = up * top, inv about 127 / t.
template <typename T>
__device__ __forceinline__ int qr_code(float x, float up, float t, float inv) {
    x *= up;
    float q = rintf(x * inv);
    bool over, tie, pos;
    if constexpr (sizeof(T) == 2) {
        const float d = 2.0f * __builtin_fmaf(x, 127.0f, -(q * t));
        over = fabsf(d) > t;
        tie = fabsf(d) == t;
        pos = d > 0.0f;
    } else {
        const double d = 2.0 * __builtin_fma((double)x, 127.0, -((double)q * (double)t));
        over = fabs(d) > (double)t;
        tie = fabs(d) == (double)t;
        pos = d > 0.0;
    }
    int code = (int)q;
    if (over || (tie && (code & 1))) code += pos ? 1 : -1;
    return code;
}

template <typename T>
__device__ __forceinline__ void qr_put(int8_t* out, int c, int K, u32x4 r, float up, float t, float inv, bool fine) {
    constexpr int N = QrVec<T>::N;
    uint32_t w[N / 4];
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
        w[h] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int q = qr_code<T>(QrVec<T>::get(r, 4 * h + i), up, t, inv);
            w[h] |= ((uint32_t)q & 0xFFu) << (8 * i);
        }
        if (!fine) w[h] = 0;
    }
    int8_t* p = out + (size_t)c * N;
    if (K - c * N >= N) {
        if constexpr (N == 8)
            *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
        else
            *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < K - c * N) p[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// W waves per row, 256 / (64 W) rows per workgroup (W = 16: 1024 threads, one row).
template <typename T, int W>
__global__ __launch_bounds__(W > 4 ? 64 * W : 256) void qr_kernel(int rows, int K, const T* __restrict__ x, int64_t ldx,
                                                                 int8_t* __restrict__ codes, int64_t ldq,
                                                                 float* __restrict__ scale) {
    constexpr int HELD = 4, NT = 64 * W, RPB = W > 4 ? 1 : 4 / W;
    const int tid = threadIdx.x % NT, sub = threadIdx.x / NT;
    const int64_t row = (int64_t)blockIdx.x * RPB + sub;
    const bool has = row < rows;
    const T* const xr = x + (size_t)(has ? row : 0) * ldx;
    const int chunks = (K + QrVec<T>::N - 1) / QrVec<T>::N;
    u32x4 held[HELD];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        held[i] = u32x4{0, 0, 0, 0};
        if (i * NT + tid < chunks) held[i] = qr_load(xr, i * NT + tid, K);
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) m = max(m, qr_top<T>(held[i]));
    for (int c = HELD * NT + tid; c < chunks; c += NT) m = max(m, qr_top<T>(qr_load(xr, c, K)));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, WAVE));
    if constexpr (W > 1) {
        __shared__ uint32_t tops[RPB][W];
        if ((tid & 63) == 0) tops[sub][tid >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) m = max(m, tops[sub][i]);
    }
    if (!has) return;
    const float top = __uint_as_float(m);
    const bool fine = m < 0x7F800000u;
    if (tid == 0) scale[row] = fine ? top / 127.0f : __uint_as_float(0x7FC00000u);
    // (zero rows: any t above 0 gives codes 0)
    const float up = top > 0x1p64f ? 0x1p-64f : (top < 0x1p-64f ? 0x1p64f : 1.0f);
    const float t = m == 0 || !fine ? 1.0f : top * up, inv = 127.0f / t;
    int8_t* const out = codes + (size_t)row * ldq;
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (i * NT + tid < chunks) qr_put<T>(out, i * NT + tid, K, held[i], up, t, inv, fine);
    for (int c = HELD * NT + tid; c < chunks; c += NT) qr_put<T>(out, c, K, qr_load(xr, c, K), up, t, inv, fine);
}

template <typename T>
hipError_t qr_run(int rows, int K, const T* x, int64_t ldx, int8_t* codes, int64_t ldq, float* scale, hipStream_t s) {
    const int chunks = (K + QrVec<T>::N - 1) / QrVec<T>::N;
    if (chunks <= 4 * 64)   // a wave holds the row
        qr_kernel<T, 1><<<(uint32_t)((rows + 3) / 4), 256, 0, s>>>(rows, K, x, ldx, codes, ldq, scale);
    else if (rows <= 256)   // fewer rows than CUs: 16 waves each
        qr_kernel<T, 16><<<(uint32_t)rows, 1024, 0, s>>>(rows, K, x, ldx, codes, ldq, scale);
    else
        qr_kernel<T, 4><<<(uint32_t)rows, 256, 0, s>>>(rows, K, x, ldx, codes, ldq, scale);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(int rows, int K, bool f32, const void* x, int64_t ldx, int8_t* codes, int64_t ldq,
                                float* scale, hipStream_t s) {
    if (f32) return qr_run(rows, K, static_cast<const float*>(x), ldx, codes, ldq, scale, s);
    return qr_run(rows, K, static_cast<const uint16_t*>(x), ldx, codes, ldq, scale, s);
}

}  // namespace ds4
