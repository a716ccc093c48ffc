// Products in 8-bit integers with a scale for each row of x and of w:
//   z[r][n] = (sum_k xq[src(r)][k] wq_e[n][k]) * xs[src(r)] * ws_e[n] + bias_e[n]
//   y[r]    = act(z[r]) + residual[r]
// The sums are exact (int32).  Scales, bias, activation and residual are fp32,
// y is rounded once.
#pragma once
#include "matmul.hpp"

namespace ds4 {

struct M8Args : MmArgs {
    const float* xs;   // [x_rows]
    const float* ws;   // [E][N]
    int32_t* ipart;    // splits of the contraction: [ksplits][P][ldp]
};

template <typename T>
__device__ __forceinline__ void m8_ld8(const T* p, int n, bool vec, float (&v)[8]) {
    if (vec) {
        if constexpr (sizeof(T) == 2) {
            const u32x4 o = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(o[i] << 16);
                v[2 * i + 1] = __uint_as_float(o[i] & 0xFFFF0000u);
            }
        } else {
            const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? mm_ld(p + i) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void m8_st8(T* p, const float (&v)[8], int n, bool vec) {
    if (vec) {
        if constexpr (sizeof(T) == 2) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<u32x4*>(p) = o;
        } else {
            reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
            reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) mm_st(p + i, v[i]);
    }
}

// A row's scale as sum * xs * ws takes it.  A sum is at most 2^31, so sum * xs
// stays in fp32 for |xs| < 2^96; from there on 2^-64 of the scale comes first and
// 2^64 last, both exact, so that nothing on the way to a z that fp32 holds is
// infinite.  (Small scales lose nothing: sum is a whole number.)
struct M8RowScale {
    float s;
    bool far;
};
__device__ __forceinline__ M8RowScale m8_row_scale(float xs) {
    const bool far = fabsf(xs) >= 0x1p96f;
    return {far ? xs * 0x1p-64f : xs, far};
}

// z of 8 columns from n on (cnt of them exist) of a row with scale xs.
template <typename T>
__device__ __forceinline__ void m8_z8(const M8Args& a, int e, float xs, int n, int cnt, const int32_t (&sum)[8],
                                      float (&z)[8]) {
    const size_t o = (size_t)e * a.N + n;      // (rows of an odd N start anywhere)
    float ws[8];
    m8_ld8(a.ws + o, cnt, cnt >= 8 && (o & 3) == 0, ws);
    const M8RowScale rs = m8_row_scale(xs);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = (float)sum[i] * rs.s * ws[i];
    if (__builtin_expect(rs.far, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] *= 0x1p64f;
    }
    if (a.bias) {
        float b[8];
        m8_ld8(static_cast<const T*>(a.bias) + o, cnt, cnt >= 8 && (o & (16 / sizeof(T) - 1)) == 0, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += b[i];
    }
}

// act(z) + residual of 8 columns of row r, out; with SwiGLU z holds the gates
// and u the up columns.
template <typename T, bool GLU>
__device__ __forceinline__ void m8_out8(const M8Args& a, int r, int n, int cnt, float (&z)[8], const float* u) {
    if constexpr (GLU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = z[i] / (1.0f + expf(-z[i])) * u[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = mm_act(z[i], a.act);
    }
    const size_t o = (size_t)r * a.ldy + n;
    if (a.residual) {
        float v[8];
        m8_ld8(static_cast<const T*>(a.residual) + o, cnt, cnt >= 8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += v[i];
    }
    m8_st8(static_cast<T*>(a.y) + o, z, cnt, cnt >= 8);
}

// What a product runs on: a tile shape and its splits of the contraction, or
// the few-row kernel (shape < 0).
struct M8Pick {
    int shape, splits;
    double us;   // estimated
};
M8Pick m8_pick(int P, int K, int N, int E);
// Rows per chunk of a grouped call (0 on the few-row kernel), and whether its
// chunks are listed by a plan launch (else each workgroup scans).
int m8_chunk_rows(const M8Pick& pick);
bool m8_wants_plan(const M8Pick& pick, int P, int N, int E);
// Scratch of a launch (M8Args::ipart), and a bound for all up to P rows.
size_t m8_split_bytes(const M8Pick& pick, int P, int N);
size_t m8_split_bound(int P, int K, int N);
hipError_t launch_m8(const M8Args& a, const M8Pick& pick, bool f32, hipStream_t s);

// Products of few rows (matmul_int8_rows.hip): whether they run there, given
// the best tile shape's estimate.
bool m8_rows_takes(int P, int K, int N, int E, double tile_us);
hipError_t launch_m8_rows(const M8Args& a, bool f32, hipStream_t s);

}  // namespace ds4
