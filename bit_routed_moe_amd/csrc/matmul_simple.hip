// Products at original precision, one tile kernel for every mode and type:
// 64 x 64 outputs per workgroup of 4 waves, fp32 matrix instructions
// (v_mfma_f32_16x16x4_f32) on operands staged through LDS in fp32.
#include "matmul.hpp"

namespace ds4 {

namespace {

constexpr int MS_T = 64;       // tile rows and columns
constexpr int MS_K = 16;       // contraction columns per stage
constexpr int MS_LD = MS_K + 4;

// Four consecutive elements of a row from element c on; zeros past n.
template <typename T>
__device__ __forceinline__ f32x4 ms_ld4(const T* row, int c, int n) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c + 4 <= n) {
        if constexpr (sizeof(T) == 4) {
            v = *reinterpret_cast<const f32x4*>(row + c);
        } else {
            const u32x2 p = *reinterpret_cast<const u32x2*>(row + c);
            v[0] = __uint_as_float(p[0] << 16);
            v[1] = __uint_as_float(p[0] & 0xFFFF0000u);
            v[2] = __uint_as_float(p[1] << 16);
            v[3] = __uint_as_float(p[1] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < n) v[i] = mm_ld(row + c + i);
    }
    return v;
}

template <typename T, int MODE, typename G>
__global__ __launch_bounds__(256) void ms_kernel(MmArgs a, int tiles_m, int tiles_n) {
    __shared__ float As[MS_T][MS_LD], Bs[MS_T][MS_LD];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int m16 = lane & 15, q = lane >> 4;
    const bool glu = MODE == MM_FWD && a.act == MM_SWIGLU;
    MmChunk ch;
    int tn, m0 = 0, kdim;
    if constexpr (MODE == MM_WGRAD) {
        ch.group = blockIdx.y;
        mm_group_rows(a.offsets, ch.group, a.P, ch.row0, ch.n);
        m0 = (blockIdx.x % tiles_m) * MS_T;
        tn = (blockIdx.x / tiles_m) * MS_T;
        kdim = ch.n;
    } else {
        if (!mm_chunk(a, blockIdx.x % tiles_m, MS_T, ch)) return;
        tn = (blockIdx.x / tiles_m) * MS_T;
        kdim = MODE == MM_FWD ? a.K : a.N;
    }
    const T* wg = static_cast<const T*>(a.w) + (size_t)ch.group * a.N * a.ldw;
    const T* x = static_cast<const T*>(a.x);
    const T* dz = static_cast<const T*>(a.dz);

    // staging: K-contiguous operands: thread -> row tid/4, columns 4*(tid%4);
    // the others: thread -> contraction row tid/16, tile columns 4*(tid%16)
    const int sr = tid >> 2, sc = (tid & 3) * 4;
    const int tk = tid >> 4, tc = (tid & 15) * 4;
    const T* arow = nullptr;
    const T* brow = nullptr;
    if constexpr (MODE == MM_FWD) {
        if (sr < ch.n) arow = x + (size_t)mm_src(a, ch.row0 + sr) * a.ldx;
        const int n = mm_col(a, glu, tn, sr);
        if (n >= 0) brow = wg + (size_t)n * a.ldw;
    } else if constexpr (MODE == MM_DGRAD) {
        if (sr < ch.n) arow = dz + (size_t)(ch.row0 + sr) * a.lddz;
    }
    f32x4 acc[2][2] = {};
    const int wm = (w & 1) * 32, wn = (w >> 1) * 32;
    for (int k0 = 0; k0 < kdim; k0 += MS_K) {
        f32x4 av = {0.0f, 0.0f, 0.0f, 0.0f}, bv = {0.0f, 0.0f, 0.0f, 0.0f};
        const int kr = k0 + tk;
        if constexpr (MODE == MM_WGRAD) {
            if (kr < kdim) {
                av = ms_ld4(dz + (size_t)(ch.row0 + kr) * a.lddz, m0 + tc, a.N);
                bv = ms_ld4(x + (size_t)mm_src(a, ch.row0 + kr) * a.ldx, tn + tc, a.K);
            }
        } else {
            if (arow) av = ms_ld4(arow, k0 + sc, kdim);
            if constexpr (MODE == MM_FWD) {
                if (brow) bv = ms_ld4(brow, k0 + sc, kdim);
            } else {
                if (kr < kdim) bv = ms_ld4(wg + (size_t)kr * a.ldw, tn + tc, a.K);
            }
        }
        __syncthreads();
        if constexpr (MODE == MM_WGRAD) {
#pragma unroll
            for (int i = 0; i < 4; ++i) As[tc + i][tk] = av[i];
        } else {
            *reinterpret_cast<f32x4*>(&As[sr][sc]) = av;
        }
        if constexpr (MODE == MM_FWD) {
            *reinterpret_cast<f32x4*>(&Bs[sr][sc]) = bv;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) Bs[tc + i][tk] = bv[i];
        }
        __syncthreads();
        // lane quarter q holds contraction columns 4q .. 4q+3; instruction j
        // takes column 4q + j of every quarter (the same for A and B)
        f32x4 af[2], bf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            af[i] = *reinterpret_cast<const f32x4*>(&As[wm + 16 * i + m16][4 * q]);
            bf[i] = *reinterpret_cast<const f32x4*>(&Bs[wn + 16 * i + m16][4 * q]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int l = 0; l < 2; ++l)
                    acc[i][l] = __builtin_amdgcn_mfma_f32_16x16x4f32(af[i][j], bf[l][j], acc[i][l], 0, 0, 0);
    }
    // lane: tile column m16, tile rows 4q + t of each 16 x 16 block
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int mr = wm + 16 * i + 4 * q + t;
            if constexpr (MODE == MM_FWD) {
                if (mr >= ch.n) continue;
                const int r = ch.row0 + mr;
                if (glu) {
                    const int f = mm_col(a, true, tn, wn + m16);
                    if (f >= 0) mm_out_glu<T>(a, ch.group, r, f, acc[i][0][t], acc[i][1][t]);
                } else {
#pragma unroll
                    for (int l = 0; l < 2; ++l) {
                        const int n = tn + wn + 16 * l + m16;
                        if (n < a.N) mm_out<T>(a, ch.group, r, n, acc[i][l][t]);
                    }
                }
            } else {
                if (MODE == MM_DGRAD ? mr >= ch.n : m0 + mr >= a.N) continue;
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    const int k = tn + wn + 16 * l + m16;
                    if (k >= a.K) continue;
                    if constexpr (MODE == MM_DGRAD)
                        mm_st(static_cast<T*>(a.dx) + (size_t)(ch.row0 + mr) * a.ldx + k, acc[i][l][t]);
                    else
                        mm_st(static_cast<G*>(a.dw) + ((size_t)ch.group * a.N + m0 + mr) * a.ldw + k, acc[i][l][t]);
                }
            }
        }
    }
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

}  // namespace

int mm_chunk_rows(bool f32, int mode, int P, int K, int N, int E) {
    if (!f32 && mode == MM_FWD && mr_takes(P, N, E)) return 0;
    return f32 ? MS_T : mt_chunk_rows(mode, P, K, N, E);
}

size_t mm_split_bytes(bool f32, int mode, int P, int K, int N, int E, bool exact) {
    if (f32 || (exact && mode == MM_FWD && mr_takes(P, N, E))) return 0;
    return mt_split_bytes(mode, P, K, N, E, exact);
}

hipError_t launch_mm_forward(const MmArgs& a, bool f32, hipStream_t s) {
    const int tm = a.chunks ? a.max_chunks : cdiv(a.P, MS_T), tn = cdiv(a.N, MS_T);
    const dim3 g((uint32_t)(tm * tn));
    if (f32)
        ms_kernel<float, MM_FWD, float><<<g, 256, 0, s>>>(a, tm, tn);
    else
        return mr_takes(a.P, a.N, a.E) ? launch_mr_forward(a, s) : launch_mt(a, MM_FWD, s);
    return hipGetLastError();
}

hipError_t launch_mm_dgrad(const MmArgs& a, bool f32, hipStream_t s) {
    const int tm = a.chunks ? a.max_chunks : cdiv(a.P, MS_T), tn = cdiv(a.K, MS_T);
    const dim3 g((uint32_t)(tm * tn));
    if (f32)
        ms_kernel<float, MM_DGRAD, float><<<g, 256, 0, s>>>(a, tm, tn);
    else
        return launch_mt(a, MM_DGRAD, s);
    return hipGetLastError();
}

hipError_t launch_mm_wgrad(const MmArgs& a, bool f32, hipStream_t s) {
    const int tm = cdiv(a.N, MS_T), tn = cdiv(a.K, MS_T);
    const dim3 g((uint32_t)(tm * tn), (uint32_t)a.E);
    if (f32)
        ms_kernel<float, MM_WGRAD, float><<<g, 256, 0, s>>>(a, tm, tn);
    else
        return launch_mt(a, MM_WGRAD, s);
    return hipGetLastError();
}

}  // namespace ds4
