// bf16 forward products of few rows (decoding): every weight is read once,
// straight into registers, and the time is that of reading them.
//
// A workgroup takes one chunk of at most 16 rows of a group and 16 * RT weight
// rows (SwiGLU: 16 gate rows and the 16 up rows they pair with); its 8 waves
// share the contraction KW ways (and weight rows 8 / KW ways where the
// contraction is short), so that a small product still has enough waves to
// keep the memory busy.  A step is 128 contraction columns, 4 loads of 64
// contiguous bytes of each of 16 weight rows, two steps in flight per wave
// (256 contiguous bytes as 4 pieces 64 bytes apart, each load touching twice
// the lines, took 136 us for one token's gate/up products instead of 80, and
// non-temporal loads 98).  Weights go first into the matrix instruction
// (v_mfma_f32_16x16x32_bf16), so a lane's results belong to one token.  The
// waves' partial sums are joined in LDS in wave order.  5.0 TB/s on one
// 7168 x 7168 product (20.4 us), 5.9 TB/s on one token's gate/up products of 8
// experts (79.5 us), 6.2 TB/s on a 131072 x 7168 head (301 us).
//
// The rows' group is found from the offsets in the kernel (a plan launch would
// cost more than the product): workgroup row p of the grid is sorted row p,
// and only the first row of each 16-row chunk of a group goes on.
#include "matmul.hpp"

namespace ds4 {

namespace {

constexpr int MR_WAVES = 8;
constexpr int MR_STEP = 128;   // contraction columns per step

// 16 bytes of a row from chunk c on; elements from column K on are zero.
__device__ __forceinline__ u32x4 mr_masked(const uint16_t* row, int c, int K) {
    u32x4 v = {0, 0, 0, 0};
    if (8 * c < K) {
        v = *reinterpret_cast<const u32x4*>(row + 8 * c);
        const int n = K - 8 * c;
        if (n < 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = 2 * i + 1 < n ? v[i] : (2 * i < n ? v[i] & 0xFFFFu : 0u);
        }
    }
    return v;
}

template <int RT, bool GLU>
__global__ __launch_bounds__(64 * MR_WAVES) void mr_kernel(MmArgs a, int kw) {
    __shared__ f32x4 red[MR_WAVES][RT][64];
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, q = lane >> 4;

    // the chunk: group, first row, rows
    int group = 0, row0 = blockIdx.y, n = 0;
    if (a.offsets) {
        if (tid == 0) found[2] = 0;
        __syncthreads();
        for (int e = tid; e < a.E; e += 64 * MR_WAVES) {
            int r0, cnt;
            mm_group_rows(a.offsets, e, a.P, r0, cnt);
            if (row0 >= r0 && row0 < r0 + cnt && (row0 - r0) % 16 == 0) {
                // (overlapping ranges of corrupt offsets: any one of them)
                found[0] = e;
                found[1] = min(16, r0 + cnt - row0);
                found[2] = 1;
            }
        }
        __syncthreads();
        if (!found[2]) return;
        group = __builtin_amdgcn_readfirstlane(found[0]);
        n = __builtin_amdgcn_readfirstlane(found[1]);
    } else {
        row0 = 16 * blockIdx.y;
        n = min(16, a.P - row0);
    }

    // this wave's weight rows and share of the contraction
    const int ng = MR_WAVES / kw, kpart = w % kw;
    const int rb = blockIdx.x * ng + w / kw;               // block of 16 * RT rows (GLU: 16 pairs)
    const int cols = GLU ? a.N >> 1 : a.N;
    const uint16_t* wg = static_cast<const uint16_t*>(a.w) + (size_t)group * a.N * a.ldw;
    const uint16_t* wr[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int c = GLU ? rb * 16 + m : rb * 16 * RT + 16 * t + m;
        wr[t] = wg + (size_t)(min(c, cols - 1) + (GLU && t ? cols : 0)) * a.ldw;
    }
    const bool has = m < n;
    const uint16_t* xr = static_cast<const uint16_t*>(a.x) + (size_t)mm_src(a, row0 + (has ? m : 0)) * a.ldx;

    const int full = a.K / MR_STEP;
    const int each = (full + kw - 1) / kw;
    const int s0 = min(full, kpart * each), s1 = min(full, s0 + each);
    f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 wv[2][RT][4], xv[2][4];
    auto load = [&](int b, int s) {
        const int c = s * MR_STEP + 8 * q;
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                wv[b][t][j] = reinterpret_cast<const u32x4*>(wr[t] + c)[4 * j];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            xv[b][j] = u32x4{0, 0, 0, 0};
            if (has) xv[b][j] = reinterpret_cast<const u32x4*>(xr + c)[4 * j];
        }
    };
    auto mma = [&](int b) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < RT; ++t)
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv[b][t][j]),
                                                                 __builtin_bit_cast(bf16x8, xv[b][j]), acc[t], 0, 0, 0);
    };
    if (rb * 16 * (GLU ? 1 : RT) < cols) {
        if (s0 < s1) load(0, s0);
        if (s0 + 1 < s1) load(1, s0 + 1);
        for (int s = s0; s < s1; s += 2) {
            mma(0);
            if (s + 2 < s1) load(0, s + 2);
            if (s + 1 < s1) {
                mma(1);
                if (s + 3 < s1) load(1, s + 3);
            }
        }
        if (kpart == kw - 1 && a.K % MR_STEP) {   // the last columns, masked
            const int c = full * (MR_STEP / 8) + q;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x4 xt = has ? mr_masked(xr, c + 4 * j, a.K) : u32x4{0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, mr_masked(wr[t], c + 4 * j, a.K)), __builtin_bit_cast(bf16x8, xt), acc[t],
                        0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) red[w][t][lane] = acc[t];
    __syncthreads();

    // one output per thread and turn: weight row rr (fastest) of row group g, token tok
    const int per = GLU ? 16 : 16 * RT;                    // outputs per row group and token
    for (int i = tid; i < ng * per * n; i += 64 * MR_WAVES) {
        const int rr = i % per, g = (i / per) % ng, tok = i / (per * ng);
        const int c = (blockIdx.x * ng + g) * per + rr;
        if (c >= cols) continue;
        float z[GLU ? 2 : 1];
#pragma unroll
        for (int t = 0; t < (GLU ? 2 : 1); ++t) {
            const int rt = GLU ? t : rr >> 4;
            const float* p = reinterpret_cast<const float*>(&red[g * kw][rt][((rr & 15) >> 2) * 16 + tok]) + (rr & 3);
            z[t] = 0.0f;
            for (int k = 0; k < kw; ++k) z[t] += p[(size_t)k * RT * 64 * 4];
        }
        if constexpr (GLU)
            mm_out_glu<uint16_t>(a, group, row0 + tok, c, z[0], z[1]);
        else
            mm_out<uint16_t>(a, group, row0 + tok, c, z[0]);
    }
}

// Waves of a workgroup along the contraction: all 8 from 8 steps on, fewer
// while a share would be empty.
int mr_kw(int K) {
    int kw = MR_WAVES;
    while (kw > 1 && kw > K / MR_STEP) kw >>= 1;
    return kw;
}

}  // namespace

// Products that take these kernels; "a / b": us here / with the tile kernels,
// weights read from memory each time (K -> N at some rows).
//   dense, up to 8 rows: 2048 -> 8192 10.9 / 16.0, 7168 -> 4096 14.8 / 16.8,
//     7168 -> 131072 310 / 309; at worst 7168 -> 1024 13.7 / 11.2 and 4096 ->
//     131072 200 / 175.
//   dense, 16 rows (the rows' own reads from L2 grow to half the weights'):
//     2048 -> 8192 12.3 / 16.1, 4096 -> 4096 11.7 / 13.5, 7168 -> 4096 17.0 /
//     17.3, but past about 2^24 weights the tiles win: 4096 -> 8192 19.4 / 17.8,
//     7168 -> 8192 30.8 / 26.1, 7168 -> 16384 57.5 / 44.9, and from 32768
//     columns on, where the rule leaves it to them, 7168 -> 32768 91 / 79.  A
//     rule on weights in place of columns would serve 9 to 16 rows better.
//   grouped, 256 experts: 7168 -> 4096 8 pairs 80 / 84, 64 499 / 519, 256 1515
//     / 1528; 2048 -> 1024 64 pairs 39 / 45, 256 125 / 124; 2048 -> 7168 64
//     pairs 267 / 264, 256 828 / 775.  64 experts: 7168 -> 4096 64 pairs 399 /
//     410, 128 505 / 500, 256 (tiles) 634 / 601.  8 experts: 7168 -> 4096 8
//     pairs 58 / 64, 16 74 / 68, 32 (tiles) 95 / 84.
bool mr_takes(int P, int N, int E) {
    if (E > 1) return P <= 16 || (P <= 256 && P <= 2 * E);
    return P <= 8 || (P <= 16 && N < 32768);
}

hipError_t launch_mr_forward(const MmArgs& a, hipStream_t s) {
    const int kw = mr_kw(a.K), ng = MR_WAVES / kw;
    const uint32_t gy = a.offsets ? (uint32_t)a.P : (uint32_t)((a.P + 15) / 16);
    const bool glu = a.act == MM_SWIGLU;
    // two row tiles per wave once there are 4 workgroups per CU with them
    const bool two = glu || (int64_t)((a.N + 31) / 32) * (a.offsets ? a.P : 1) >= 1024 * ng;
    const int per = glu ? 16 : (two ? 32 : 16), cols = glu ? a.N / 2 : a.N;
    const dim3 g((uint32_t)((cols + per * ng - 1) / (per * ng)), gy);
    if (glu)
        mr_kernel<2, true><<<g, 64 * MR_WAVES, 0, s>>>(a, kw);
    else if (two)
        mr_kernel<2, false><<<g, 64 * MR_WAVES, 0, s>>>(a, kw);
    else
        mr_kernel<1, false><<<g, 64 * MR_WAVES, 0, s>>>(a, kw);
    return hipGetLastError();
}

}  // namespace ds4
