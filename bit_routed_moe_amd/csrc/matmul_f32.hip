// fp32 products at original precision on the fp32 matrix instructions
// (v_mfma_f32_16x16x4_f32), every mode in one kernel: 64 x 64 outputs per
// workgroup of 4 waves, stages of 32 contraction columns through two LDS
// buffers, the loads of the two stages after it in flight (in registers) while
// one is worked on.  In LDS an operand lies as it comes: contiguous along the
// contraction, rows of 32 + 4 floats and fragments of 4 columns at once;
// contiguous along the tile, contraction rows of 64 + 4 floats and fragments
// element by element (written transposed, 16 lanes met in one bank).  Sizes
// are those of parity runs and of small models.  118 .. 122 TFLOP/s in both
// directions from 4096 x 7168 x 2048 on (the library's 8192^3 product 154), 67
// at 1000 x 1500 x 1500.  A stage's latency, about 1.2 us, bounds products of
// few outputs: the contraction is not split, so 16 rows of 1500 -> 200 take
// 35 us.
#include "matmul.hpp"

namespace ds4 {

namespace {

constexpr int MS_T = 64;       // tile rows and columns
constexpr int MS_K = 32;       // contraction columns per stage
constexpr int MS_LD = MS_K + 4;    // floats per LDS row, contraction along the row
constexpr int MS_LT = MS_T + 4;    // the same, tile along the row
constexpr int MS_BUF = MS_T * MS_LD > MS_K * MS_LT ? MS_T * MS_LD : MS_K * MS_LT;

template <int MODE>
__global__ __launch_bounds__(256) void ms_kernel(MmArgs a, int tiles_m) {
    __shared__ __attribute__((aligned(16))) float As[2][MS_BUF], Bs[2][MS_BUF];
    constexpr bool AT = MODE == MM_WGRAD, BT = MODE != MM_FWD;   // contiguous along the tile
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
    // (rows and columns past the tile's end read the last one: what they give
    // is not stored)
    const float* arow[2] = {nullptr, nullptr};
    const float* brow[2] = {nullptr, nullptr};
    if constexpr (MODE != MM_WGRAD) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = ch.row0 + min(sr + 32 * i, ch.n - 1);
            if constexpr (MODE == MM_FWD) {
                arow[i] = x + (size_t)mm_src(a, r) * a.ldx;
                const int n = mm_col(a, glu, tn, sr + 32 * i);
                brow[i] = wg + (size_t)(n < 0 ? a.N - 1 : n) * a.ldw;
            } else {
                arow[i] = dz + (size_t)r * a.lddz;
            }
        }
    }
    const int acol = min(m0 + tc, (a.N - 1) & ~3), bcol = min(tn + tc, (a.K - 1) & ~3), klast = (kdim - 1) & ~3;
    // two stages of pieces in flight; wgrad's x rows (through the pair ids) are
    // known a stage before their pieces are asked for
    f32x4 av[2][2], bv[2][2];
    int src[2] = {0, 0};
    auto rows_of = [&](int k0) {
        if constexpr (MODE == MM_WGRAD) {
#pragma unroll
            for (int i = 0; i < 2; ++i) src[i] = mm_src(a, ch.row0 + min(k0 + tk + 16 * i, kdim - 1));
        }
    };
    // whole 16-byte pieces without a branch (which would make the compiler wait
    // for the loads); store() puts zeros behind the contraction's end
    auto load = [&](int u, int k0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int kr = min(k0 + tk + 16 * i, kdim - 1), kc = min(k0 + sc, klast);
            const float *pa, *pb;
            if constexpr (MODE == MM_WGRAD) {
                pa = dz + (size_t)(ch.row0 + kr) * a.lddz + acol;
                pb = x + (size_t)src[i] * a.ldx + bcol;
            } else {
                pa = arow[i] + kc;
                pb = MODE == MM_FWD ? brow[i] + kc : wg + (size_t)kr * a.ldw + bcol;
            }
            av[u][i] = *reinterpret_cast<const f32x4*>(pa);
            bv[u][i] = *reinterpret_cast<const f32x4*>(pb);
        }
    };
    auto store = [&](int b, int k0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (k0 + MS_K > kdim) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool kc = k0 + sc + j < kdim, kr = k0 + tk + 16 * i < kdim;
                    av[b][i][j] = (AT ? kr : kc) ? av[b][i][j] : 0.0f;
                    bv[b][i][j] = (BT ? kr : kc) ? bv[b][i][j] : 0.0f;
                }
            }
            *reinterpret_cast<f32x4*>(&As[b][AT ? (tk + 16 * i) * MS_LT + tc : (sr + 32 * i) * MS_LD + sc]) = av[b][i];
            *reinterpret_cast<f32x4*>(&Bs[b][BT ? (tk + 16 * i) * MS_LT + tc : (sr + 32 * i) * MS_LD + sc]) = bv[b][i];
        }
    };
    // tile row r, contraction columns k .. k+3
    auto frag = [&](const float* buf, bool t, int r, int k) {
        if (!t) return *reinterpret_cast<const f32x4*>(buf + r * MS_LD + k);
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = buf[(k + j) * MS_LT + r];
        return v;
    };
    f32x4 acc[2][2] = {};
    const int wm = (w & 1) * 32, wn = (w >> 1) * 32;
    if (kdim > 0) {
        rows_of(0);
        load(0, 0);
        rows_of(MS_K);
        load(1, MS_K);
        rows_of(2 * MS_K);
    }
    auto stage = [&](int b, int k0) {
        store(b, k0);
        load(b, k0 + 2 * MS_K);
        rows_of(k0 + 3 * MS_K);
        __syncthreads();
        // lane quarter q holds 4 contraction columns of each half; instruction
        // j takes column j of every quarter (the same for A and B)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4 af[2], bf[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                af[i] = frag(As[b], AT, wm + 16 * i + m16, 16 * h + 4 * q);
                bf[i] = frag(Bs[b], BT, wn + 16 * i + m16, 16 * h + 4 * q);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int l = 0; l < 2; ++l)
                        acc[i][l] = __builtin_amdgcn_mfma_f32_16x16x4f32(af[i][j], bf[l][j], acc[i][l], 0, 0, 0);
        }
    };
    for (int k0 = 0; k0 < kdim; k0 += 2 * MS_K) {
        stage(0, k0);
        if (k0 + MS_K < kdim) stage(1, k0 + MS_K);
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
