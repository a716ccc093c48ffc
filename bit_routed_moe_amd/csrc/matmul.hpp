// Products at original precision (bf16 or fp32 weights), grouped by expert or
// dense: arguments, activations and the epilogue that every kernel shares.
//
//   forward  z[r][n] = sum_k x[src(r)][k] w_e[n][k] + bias_e[n]
//            y[r]    = act(z[r]) + residual[r]
//   dgrad    dx[r][k] = sum_n dz[r][n] w_e[n][k]
//   wgrad    dw_e[n][k] = sum_{r in e} dz[r][n] x[src(r)][k]
// with e the group of row r (rows offsets[e] .. offsets[e+1]-1; one group of
// all rows when there are no offsets) and src(r) = sorted_pair[r] / top_k
// (r itself without sorted_pair).
#pragma once
#include "common.hpp"
#include "launch.hpp"

namespace ds4 {

enum MmAct { MM_NONE = 0, MM_RELU = 1, MM_SILU = 2, MM_GELU = 3, MM_GELU_TANH = 4, MM_SWIGLU = 5 };
enum MmMode { MM_FWD = 0, MM_DGRAD = 1, MM_WGRAD = 2 };

// Smallest rows per chunk that mm_chunk_rows returns (sizes the plan).
constexpr int MM_MIN_CHUNK = 64;

// One piece of a group's rows: forward and dgrad run a row tile of it.
struct MmChunk {
    int32_t group, row0, n, pad;
};

__device__ __forceinline__ float mm_sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// tanh form of GELU: 0.5 z (1 + tanh u) = z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
constexpr float MM_GT_A = 1.5957691216057308f;              // 2 sqrt(2/pi)
constexpr float MM_GT_B = 1.5957691216057308f * 0.044715f;

// act(z) for the element-wise activations (SwiGLU pairs two columns).
__device__ __forceinline__ float mm_act(float z, int act) {
    switch (act) {
        case MM_RELU: return z > 0.0f ? z : (z == z ? 0.0f : z);
        case MM_SILU: return z / (1.0f + expf(-z));
        case MM_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
        case MM_GELU_TANH: return z / (1.0f + expf(-z * (MM_GT_A + MM_GT_B * z * z)));
        default: return z;
    }
}

// act'(z).
__device__ __forceinline__ float mm_act_grad(float z, int act) {
    switch (act) {
        case MM_RELU: return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
        case MM_SILU: {
            const float p = mm_sigmoid(z);
            return p * (1.0f + z * (1.0f - p));
        }
        case MM_GELU:
            return 0.5f * erfcf(-0.70710678118654752f * z) + z * (0.3989422804014327f * expf(-0.5f * z * z));
        case MM_GELU_TANH: {
            // past |z| = 100 the sigmoid is exactly 0 or 1 and z^2 may overflow
            const float c = fminf(fmaxf(z, -100.0f), 100.0f);
            const float p = mm_sigmoid(c * (MM_GT_A + MM_GT_B * c * c));
            const float g = p + c * (p * (1.0f - p)) * (MM_GT_A + 3.0f * MM_GT_B * c * c);
            return z == z ? g : z;
        }
        default: return 1.0f;
    }
}

template <typename T>
__device__ __forceinline__ float mm_ld(const T* p);
template <>
__device__ __forceinline__ float mm_ld<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float mm_ld<uint16_t>(const uint16_t* p) { return bf16_to_f32(*p); }

template <typename T>
__device__ __forceinline__ void mm_st(T* p, float v);
template <>
__device__ __forceinline__ void mm_st<float>(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void mm_st<uint16_t>(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16(v); }

// Group e's rows, all rows without offsets; an invalid range counts as empty,
// so corrupt offsets reach no row outside [0, P).
__device__ __forceinline__ void mm_group_rows(const int32_t* offsets, int e, int P, int& row0, int& n) {
    row0 = 0;
    n = P;
    if (!offsets) return;
    row0 = offsets[e];
    const int end = offsets[e + 1];
    n = (row0 >= 0 && end <= P && end >= row0) ? end - row0 : 0;
}

// Source row of sorted row r in x (clamped into x, so corrupt pair ids read
// no memory outside it).
__device__ __forceinline__ int mm_src(const MmArgs& a, int r) {
    if (!a.sorted_pair) return r;
    const int s = (int)((uint32_t)a.sorted_pair[r] / (uint32_t)a.top_k);
    return min(max(s, 0), a.x_rows - 1);
}

// Chunk c of the plan (or of the one group); false past the end.
__device__ __forceinline__ bool mm_chunk(const MmArgs& a, int c, int bm, MmChunk& ch) {
    if (a.chunks) {
        if (c >= a.n_chunks[0]) return false;
        ch = a.chunks[c];
        return true;
    }
    int row0, n;
    mm_group_rows(a.offsets, 0, a.P, row0, n);
    ch.group = 0;
    ch.row0 = row0 + c * bm;
    ch.n = min(bm, n - c * bm);
    return ch.n > 0;
}

// Logical output column of column c (0 ..) of a tile.  SwiGLU interleaves 16
// gate columns with the 16 up columns they pair with, so both reach the same
// lane; -1 past the last column.
__device__ __forceinline__ int mm_col(const MmArgs& a, bool glu, int tile0, int c) {
    if (!glu) {
        const int n = tile0 + c;
        return n < a.N ? n : -1;
    }
    const int half = a.N >> 1;
    const int f = (tile0 >> 1) + ((c >> 5) << 4) + (c & 15);
    return f < half ? f + ((c & 16) ? half : 0) : -1;
}

// Epilogue of one element-wise output: z (fp32) at (r, n) of group e.
template <typename T>
__device__ __forceinline__ void mm_out(const MmArgs& a, int e, int r, int n, float z) {
    if (a.bias) z += mm_ld(static_cast<const T*>(a.bias) + (size_t)e * a.N + n);
    if (a.z) mm_st(static_cast<T*>(a.z) + (size_t)r * a.ldz + n, z);
    float v = mm_act(z, a.act);
    const size_t o = (size_t)r * a.ldy + n;
    if (a.residual) v += mm_ld(static_cast<const T*>(a.residual) + o);
    mm_st(static_cast<T*>(a.y) + o, v);
}

// The same for one SwiGLU pair: g at column f, u at column N/2 + f.
template <typename T>
__device__ __forceinline__ void mm_out_glu(const MmArgs& a, int e, int r, int f, float g, float u) {
    const int half = a.N >> 1;
    if (a.bias) {
        const T* b = static_cast<const T*>(a.bias) + (size_t)e * a.N;
        g += mm_ld(b + f);
        u += mm_ld(b + half + f);
    }
    if (a.z) {
        T* zr = static_cast<T*>(a.z) + (size_t)r * a.ldz;
        mm_st(zr + f, g);
        mm_st(zr + half + f, u);
    }
    float v = g / (1.0f + expf(-g)) * u;
    const size_t o = (size_t)r * a.ldy + f;
    if (a.residual) v += mm_ld(static_cast<const T*>(a.residual) + o);
    mm_st(static_cast<T*>(a.y) + o, v);
}

// bf16 tile kernels (matmul_tile.hip).
struct MtPick {
    int shape, splits;
};
MtPick mt_pick(int mode, int P, int K, int N, int E);
int mt_chunk_rows(int mode, int P, int K, int N, int E);
// Scratch for the partial sums of a split contraction.
size_t mt_split_bytes(int mode, int P, int K, int N, int E, bool exact);
hipError_t launch_mt(const MmArgs& a, int mode, hipStream_t s);

// bf16 forward products of few rows (matmul_rows.hip).
bool mr_takes(int P, int N, int E);
hipError_t launch_mr_forward(const MmArgs& a, hipStream_t s);

}  // namespace ds4
