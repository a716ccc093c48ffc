// Rows to 8-bit integers with one scale each:
//   top = max |x|, scale = top / 127, code = the whole number nearest to
//   x * 127 / top (ties to even)
// The nearest whole number is decided exactly.  With x = X 2^a and top = T 2^b,
// X and T whole numbers of m bits and a <= b, the quotient v = 127 X 2^(a-b) / T
// is a half between whole numbers or at least 2^(a-b) / (2T) > 2^(a-b-m-1) away
// from one.  v is computed as x hi + x lo, hi + lo = 127 / top to twice the
// arithmetic's p bits, and rounded once: it is off by at most 2^(a-b+8-p) (its
// size is below 2^(a-b+8)), far less than that distance, and a half, which p
// bits hold, comes out as itself, so rounding to the even whole number decides
// it.  bf16 rows (m = 8) take fp32 (p = 24), fp32 rows (m = 24) fp64 (p = 53).
// (Comparing the remainder of a first guess, exactly, cost twice the
// instructions: 20.7 against 16.4 us at 4096 rows of 7168 bf16.)
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
    typedef double F;
    static __device__ __forceinline__ float get(u32x4 r, int i) { return __uint_as_float(r[i]); }
};
template <>
struct QrVec<uint16_t> {
    static constexpr int N = 8;
    typedef float F;
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

// 127 / t in two parts, in the arithmetic that decides codes.
template <typename F>
struct QrInv {
    float up;    // a power of 2 that brings top into the middle of fp32's range; t = up * top
    F hi, lo;
};
template <typename F>
__device__ __forceinline__ QrInv<F> qr_inv(float top, bool fine) {
    QrInv<F> v;
    v.up = top > 0x1p64f ? 0x1p-64f : (top < 0x1p-64f ? 0x1p64f : 1.0f);
    // (zero rows: any t above 0 gives codes 0)
    const F t = top > 0.0f && fine ? (F)(top * v.up) : (F)1;
    v.hi = (F)127 / t;
    v.lo = __builtin_fma((F)-v.hi, t, (F)127) / t;
    return v;
}
template <>
__device__ __forceinline__ QrInv<float> qr_inv<float>(float top, bool fine) {
    QrInv<float> v;
    v.up = top > 0x1p64f ? 0x1p-64f : (top < 0x1p-64f ? 0x1p64f : 1.0f);
    const float t = top > 0.0f && fine ? top * v.up : 1.0f;
    v.hi = 127.0f / t;
    v.lo = __builtin_fmaf(-v.hi, t, 127.0f) / t;
    return v;
}

__device__ __forceinline__ int qr_code(float x, const QrInv<float>& v) {
    x *= v.up;
    return (int)rintf(__builtin_fmaf(x, v.hi, x * v.lo));
}
__device__ __forceinline__ int qr_code(float x, const QrInv<double>& v) {
    const double d = (double)(x * v.up);
    return (int)__builtin_rint(__builtin_fma(d, v.hi, d * v.lo));
}

template <typename T>
__device__ __forceinline__ void qr_put(int8_t* out, int c, int K, u32x4 r, const QrInv<typename QrVec<T>::F>& inv, bool fine) {
    constexpr int N = QrVec<T>::N;
    uint32_t w[N / 4];
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
        w[h] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int q = qr_code(QrVec<T>::get(r, 4 * h + i), inv);
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
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RPB + sub;
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
    const QrInv<typename QrVec<T>::F> inv = qr_inv<typename QrVec<T>::F>(top, fine);
    int8_t* const out = codes + (size_t)row * ldq;
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (i * NT + tid < chunks) qr_put<T>(out, i * NT + tid, K, held[i], inv, fine);
    for (int c = HELD * NT + tid; c < chunks; c += NT) qr_put<T>(out, c, K, qr_load(xr, c, K), inv, fine);
}

template <typename T>
hipError_t qr_run(int rows, int K, const T* x, int64_t ldx, int8_t* codes, int64_t ldq, float* scale, hipStream_t s) {
    const QuantGrid q = quantize_rows_grid(rows, K, sizeof(T) == 4);
    const dim3 g((uint32_t)q.x, (uint32_t)q.y);
    if (q.waves == 1)
        qr_kernel<T, 1><<<g, q.threads, 0, s>>>(rows, K, x, ldx, codes, ldq, scale);
    else if (q.waves == 16)
        qr_kernel<T, 16><<<g, q.threads, 0, s>>>(rows, K, x, ldx, codes, ldq, scale);
    else
        qr_kernel<T, 4><<<g, q.threads, 0, s>>>(rows, K, x, ldx, codes, ldq, scale);
    return hipGetLastError();
}

}  // namespace

QuantGrid quantize_rows_grid(int rows, int K, bool f32) {
    const int per = f32 ? QrVec<float>::N : QrVec<uint16_t>::N, pieces = (K + per - 1) / per;
    // a wave where it holds the row, 16 where there are fewer rows than CUs, else 4
    const int waves = pieces <= 4 * 64 ? 1 : (rows <= 256 ? 16 : 4);
    const int threads = waves == 16 ? 1024 : 256, at_once = threads / (64 * waves);
    // (a launch's threads along one dimension have to be below 2^32)
    const int blocks = (rows + at_once - 1) / at_once, y = blocks > (1 << 23) ? 2 : 1;
    return QuantGrid{waves, threads, (blocks + y - 1) / y, y};
}

hipError_t launch_quantize_rows(int rows, int K, bool f32, const void* x, int64_t ldx, int8_t* codes, int64_t ldq,
                                float* scale, hipStream_t s) {
    if (f32) return qr_run(rows, K, static_cast<const float*>(x), ldx, codes, ldq, scale, s);
    return qr_run(rows, K, static_cast<const uint16_t*>(x), ldx, codes, ldq, scale, s);
}

}  // namespace ds4
