// fp32 products at original precision on the fp32 matrix instructions
// (v_mfma_f32_16x16x4_f32), every mode in one kernel: 64 x 64 outputs per
// workgroup of 4 waves, stages of 32 contraction columns through two LDS
// buffers, the next stage's loads in flight (in registers) while one is
// worked on.  Tile rows of 36 floats: the 4-column fragment reads and the
// 16-byte writes then spread over the banks.  Sizes are those of parity runs
// and of small models; a stage's latency bounds the small ones.
#include "matmul.hpp"

namespace ds4 {

namespace {

constexpr int MS_T = 64;       // tile rows and columns
constexpr int MS_K = 32;       // contraction columns per stage
constexpr int MS_LD = MS_K + 4;

// Four consecutive elements of a row from element c on; zeros past n.
__device__ __forceinline__ f32x4 ms_ld4(const float* row, int c, int n) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c + 4 <= n) {
        v = *reinterpret_cast<const f32x4*>(row + c);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < n) v[i] = row[c + i];
    }
    return v;
}

template <int MODE>
__global__ __launch_bounds__(256) void ms_kernel(MmArgs a, int tiles_m) {
    __shared__ float As[2][MS_T][MS_LD], Bs[2][MS_T][MS_LD];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int m16 = lane & 15, q = lane >> 4;
    const bool glu = MODE == MM_FWD && a.act == MM_SWIGLU;
    MmChunk ch;
    int m0 = 0, kdim;
    const int tn = ((int)blockIdx.x / tiles_m) * MS_T;
    if constexpr (MODE == MM_WGRAD) {
        ch.group = blockIdx.y;
        mm_group_rows(a.offsets, ch.group, a.P, ch.row0, ch.n);
        m0 = ((int)blockIdx.x % tiles_m) * MS_T;
        kdim = ch.n;
    } else {
        if (!mm_chunk(a, (int)blockIdx.x % tiles_m, MS_T, ch)) return;
        kdim = MODE == MM_FWD ? a.K : a.N;
    }
    const float* wg = static_cast<const float*>(a.w) + (size_t)ch.group * a.N * a.ldw;
    const float* x = static_cast<const float*>(a.x);
    const float* dz = static_cast<const float*>(a.dz);

    // staging, two pieces of 4 elements per thread and operand.  Contiguous
    // along the contraction: rows tid/8 and tid/8 + 32, columns 4 * (tid % 8);
    // contiguous along the tile: contraction rows tid/16 and tid/16 + 16, tile
    // columns 4 * (tid % 16)
    const int sr = tid >> 3, sc = (tid & 7) * 4;
    const int tk = tid >> 4, tc = (tid & 15) * 4;
    const float* arow[2] = {nullptr, nullptr};
    const float* brow[2] = {nullptr, nullptr};
    if constexpr (MODE != MM_WGRAD) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = sr + 32 * i;
            if constexpr (MODE == MM_FWD) {
                if (r < ch.n) arow[i] = x + (size_t)mm_src(a, ch.row0 + r) * a.ldx;
                const int n = mm_col(a, glu, tn, r);
                if (n >= 0) brow[i] = wg + (size_t)n * a.ldw;
            } else {
                if (r < ch.n) arow[i] = dz + (size_t)(ch.row0 + r) * a.lddz;
            }
        }
    }
    f32x4 av[2], bv[2];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            av[i] = bv[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            const int kr = k0 + tk + 16 * i;
            if constexpr (MODE == MM_WGRAD) {
                if (kr < kdim) {
                    av[i] = ms_ld4(dz + (size_t)(ch.row0 + kr) * a.lddz, m0 + tc, a.N);
                    bv[i] = ms_ld4(x + (size_t)mm_src(a, ch.row0 + kr) * a.ldx, tn + tc, a.K);
                }
            } else {
                if (arow[i]) av[i] = ms_ld4(arow[i], k0 + sc, kdim);
                if constexpr (MODE == MM_FWD) {
                    if (brow[i]) bv[i] = ms_ld4(brow[i], k0 + sc, kdim);
                } else {
                    if (kr < kdim) bv[i] = ms_ld4(wg + (size_t)kr * a.ldw, tn + tc, a.K);
                }
            }
        }
    };
    auto store = [&](int b) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (MODE == MM_WGRAD) {
#pragma unroll
                for (int j = 0; j < 4; ++j) As[b][tc + j][tk + 16 * i] = av[i][j];
            } else {
                *reinterpret_cast<f32x4*>(&As[b][sr + 32 * i][sc]) = av[i];
            }
            if constexpr (MODE == MM_FWD) {
                *reinterpret_cast<f32x4*>(&Bs[b][sr + 32 * i][sc]) = bv[i];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) Bs[b][tc + j][tk + 16 * i] = bv[i][j];
            }
        }
    };
    f32x4 acc[2][2] = {};
    const int wm = (w & 1) * 32, wn = (w >> 1) * 32;
    load(0);
    int b = 0;
    for (int k0 = 0; k0 < kdim; k0 += MS_K, b ^= 1) {
        store(b);
        load(k0 + MS_K);   // (zeros past the end)
        __syncthreads();
        // lane quarter q holds 4 contraction columns of each half; instruction
        // j takes column j of every quarter (the same for A and B)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4 af[2], bf[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                af[i] = *reinterpret_cast<const f32x4*>(&As[b][wm + 16 * i + m16][16 * h + 4 * q]);
                bf[i] = *reinterpret_cast<const f32x4*>(&Bs[b][wn + 16 * i + m16][16 * h + 4 * q]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int l = 0; l < 2; ++l)
                        acc[i][l] = __builtin_amdgcn_mfma_f32_16x16x4f32(af[i][j], bf[l][j], acc[i][l], 0, 0, 0);
        }
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
                    if (f >= 0) mm_out_glu<float>(a, ch.group, r, f, acc[i][0][t], acc[i][1][t]);
                } else {
#pragma unroll
                    for (int l = 0; l < 2; ++l) {
                        const int n = tn + wn + 16 * l + m16;
                        if (n < a.N) mm_out<float>(a, ch.group, r, n, acc[i][l][t]);
                    }
                }
            } else {
                if (MODE == MM_DGRAD ? mr >= ch.n : m0 + mr >= a.N) continue;
#pragma unroll
                for (int l = 0; l < 2; ++l) {
                    const int k = tn + wn + 16 * l + m16;
                    if (k >= a.K) continue;
                    if constexpr (MODE == MM_DGRAD)
                        mm_st(static_cast<float*>(a.dx) + (size_t)(ch.row0 + mr) * a.ldx + k, acc[i][l][t]);
                    else
                        mm_st(static_cast<float*>(a.dw) + ((size_t)ch.group * a.N + m0 + mr) * a.ldw + k, acc[i][l][t]);
                }
            }
        }
    }
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

}  // namespace

int mm_chunk_rows(bool f32, int mode, int P, int K, int N, int E) {
    if (f32) return MS_T;
    return mode == MM_FWD && mr_takes(P, N, E) ? 0 : mt_chunk_rows(mode, P, K, N, E);
}

size_t mm_split_bytes(bool f32, int mode, int P, int K, int N, int E, bool exact) {
    if (f32 || (exact && mode == MM_FWD && mr_takes(P, N, E))) return 0;
    return mt_split_bytes(mode, P, K, N, E, exact);
}

hipError_t launch_mm_forward(const MmArgs& a, bool f32, hipStream_t s) {
    if (!f32) return mr_takes(a.P, a.N, a.E) ? launch_mr_forward(a, s) : launch_mt(a, MM_FWD, s);
    const int tm = a.chunks ? a.max_chunks : cdiv(a.P, MS_T), tn = cdiv(a.N, MS_T);
    ms_kernel<MM_FWD><<<dim3((uint32_t)(tm * tn)), 256, 0, s>>>(a, tm);
    return hipGetLastError();
}

hipError_t launch_mm_dgrad(const MmArgs& a, bool f32, hipStream_t s) {
    if (!f32) return launch_mt(a, MM_DGRAD, s);
    const int tm = a.chunks ? a.max_chunks : cdiv(a.P, MS_T), tn = cdiv(a.K, MS_T);
    ms_kernel<MM_DGRAD><<<dim3((uint32_t)(tm * tn)), 256, 0, s>>>(a, tm);
    return hipGetLastError();
}

hipError_t launch_mm_wgrad(const MmArgs& a, bool f32, hipStream_t s) {
    if (!f32) return launch_mt(a, MM_WGRAD, s);
    const int tm = cdiv(a.N, MS_T), tn = cdiv(a.K, MS_T);
    ms_kernel<MM_WGRAD><<<dim3((uint32_t)(tm * tn), (uint32_t)a.E), 256, 0, s>>>(a, tm);
    return hipGetLastError();
}

}  // namespace ds4
