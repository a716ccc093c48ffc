// 8-bit products of few rows (decoding): every weight is read once, straight
// into registers, and the time is that of reading them.
//
// A workgroup takes one chunk of at most 16 rows of a group and 16 * RT weight
// rows (SwiGLU: 16 gate rows and the 16 up rows they pair with); its 8 waves
// share the contraction KW ways (and weight rows 8 / KW ways where the
// contraction is short).  A step is 128 contraction columns, 2 loads of 64 contiguous bytes
// of each of 16 weight rows, four steps in flight per wave (steps of 256
// columns, two in flight: 12.1 against 11.3 us at one row of 7168 -> 7168, 4.2
// against 3.6 at 1024 -> 1024).
// Weights go first into the matrix instruction (v_mfma_i32_16x16x64_i8), so a
// lane's results belong to one row.  The waves' sums are joined in LDS.  One row
// of 7168 -> 7168: 11.3 us (weights at 4.5 TB/s, launch included); one token's
// gate/up products of 8 experts 7168 -> 4096 41.7 us (5.6 TB/s); 16 rows of
// 7168 -> 40000 59 us.
//
// The rows' group is found from the offsets in the kernel (a plan launch would
// cost more than the product), by a scan over the groups' numbers of chunks, or
// where there are fewer rows than chunks could be, by row: workgroup row p of
// the grid is sorted row p, and only the first row of each chunk goes on.
#include "matmul_int8.hpp"

namespace ds4 {

namespace {

constexpr int W8_WAVES = 8;
constexpr int W8_STEP = 128;   // contraction columns per step
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// 16 bytes of a row from chunk c on; bytes from column K on are zero.
__device__ __forceinline__ i32x4 w8_masked(const int8_t* row, int c, int K) {
    i32x4 v = {0, 0, 0, 0};
    const int n = K - 16 * c;
    if (n > 0) {
        v = *reinterpret_cast<const i32x4*>(row + 16 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = n - 4 * i;   // bytes of word i that exist
            v[i] = b >= 4 ? v[i] : (b > 0 ? (int32_t)((uint32_t)v[i] & (0xFFFFFFFFu >> (32 - 8 * b))) : 0);
        }
    }
    return v;
}

template <typename T, int RT, bool GLU>
__global__ __launch_bounds__(64 * W8_WAVES) void w8_kernel(M8Args a, int kw, int scan) {
    __shared__ i32x4 red[W8_WAVES][RT][64];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, q = lane >> 4;

    // the chunk: group, first row, rows
    int group = 0, row0, n;
    if (a.offsets) {
        __shared__ int found[4], tmp[32];
        if (tid == 0) found[0] = 0;
        if (scan) {   // chunk blockIdx.y of the groups' chunks
            int r0[2], cnt[2], total;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                r0[i] = cnt[i] = 0;
                if (2 * tid + i < a.E) mm_group_rows(a.offsets, 2 * tid + i, a.P, r0[i], cnt[i]);
            }
            const int n0 = (cnt[0] + 15) >> 4, n1 = (cnt[1] + 15) >> 4;
            int at = (int)blockIdx.y - block_exclusive_scan(n0 + n1, tmp, &total);   // (barriers inside)
            if (at >= 0 && at < n0 + n1) {
                const int i = at >= n0;
                at -= i ? n0 : 0;
                found[0] = 1;
                found[1] = 2 * tid + i;
                found[2] = r0[i] + 16 * at;
                found[3] = min(16, cnt[i] - 16 * at);
            }
        } else {      // the chunk that starts at row blockIdx.y, if one does
            __syncthreads();
            for (int e = tid; e < a.E; e += 64 * W8_WAVES) {
                int r0, cnt;
                mm_group_rows(a.offsets, e, a.P, r0, cnt);
                const int d = (int)blockIdx.y - r0;
                if (d >= 0 && d < cnt && d % 16 == 0) {
                    // (overlapping ranges of corrupt offsets: any of them)
                    found[0] = 1;
                    found[1] = e;
                    found[2] = blockIdx.y;
                    found[3] = min(16, cnt - d);
                }
            }
        }
        __syncthreads();
        if (!found[0]) return;
        group = __builtin_amdgcn_readfirstlane(found[1]);
        row0 = __builtin_amdgcn_readfirstlane(found[2]);
        n = min(__builtin_amdgcn_readfirstlane(found[3]), a.P - row0);
    } else {
        row0 = 16 * blockIdx.y;
        n = min(16, a.P - row0);
    }

    // this wave's weight rows and share of the contraction
    const int ng = W8_WAVES / kw, kpart = w % kw;
    const int rb = blockIdx.x * ng + w / kw;               // block of 16 * RT rows (GLU: 16 pairs)
    const int cols = GLU ? a.N >> 1 : a.N;
    const int8_t* const wg = static_cast<const int8_t*>(a.w) + (size_t)group * a.N * a.ldw;
    const int8_t* wr[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int c = GLU ? rb * 16 + m : rb * 16 * RT + 16 * t + m;
        wr[t] = wg + (size_t)(min(c, cols - 1) + (GLU && t ? cols : 0)) * a.ldw;
    }
    const bool has = m < n;
    const int8_t* const xr = static_cast<const int8_t*>(a.x) + (size_t)mm_src(a, row0 + (has ? m : 0)) * a.ldx;

    const int full = a.K / W8_STEP;
    const int each = (full + kw - 1) / kw;
    const int s0 = min(full, kpart * each), s1 = min(full, s0 + each);
    i32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = i32x4{0, 0, 0, 0};
    i32x4 wv[4][RT][2], xv[4][2];
    auto load = [&](int b, int s) {
        const int c = s * W8_STEP + 16 * q;
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) wv[b][t][j] = reinterpret_cast<const i32x4*>(wr[t] + c)[4 * j];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            xv[b][j] = i32x4{0, 0, 0, 0};
            if (has) xv[b][j] = reinterpret_cast<const i32x4*>(xr + c)[4 * j];
        }
    };
    auto mma = [&](int b) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int t = 0; t < RT; ++t)
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[b][t][j], xv[b][j], acc[t], 0, 0, 0);
    };
    if (rb * 16 * (GLU ? 1 : RT) < cols) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
            if (s0 + d < s1) load(d, s0 + d);
        for (int s = s0; s < s1; s += 4) {
#pragma unroll
            for (int d = 0; d < 4; ++d)
                if (s + d < s1) {
                    mma(d);
                    if (s + d + 4 < s1) load(d, s + d + 4);
                }
        }
        if (kpart == kw - 1 && a.K % W8_STEP) {   // the last columns, masked
            const int c = full * (W8_STEP / 16) + q;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const i32x4 xt = has ? w8_masked(xr, c + 4 * j, a.K) : i32x4{0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w8_masked(wr[t], c + 4 * j, a.K), xt, acc[t], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) red[w][t][lane] = acc[t];
    __syncthreads();

    // one output per thread and turn: weight row rr (fastest) of row group g, row tok
    const int per = GLU ? 16 : 16 * RT;                    // outputs per row group and row
    for (int i = tid; i < ng * per * n; i += 64 * W8_WAVES) {
        const int rr = i % per, g = (i / per) % ng, tok = i / (per * ng);
        const int c = (blockIdx.x * ng + g) * per + rr;
        if (c >= cols) continue;
        const int r = row0 + tok;
        const M8RowScale rs = m8_row_scale(a.xs[mm_src(a, r)]);
        float z[GLU ? 2 : 1];
#pragma unroll
        for (int t = 0; t < (GLU ? 2 : 1); ++t) {
            const int rt = GLU ? t : rr >> 4;
            const int32_t* p = reinterpret_cast<const int32_t*>(&red[g * kw][rt][((rr & 15) >> 2) * 16 + tok]) + (rr & 3);
            int32_t sum = 0;
            for (int k = 0; k < kw; ++k) sum += p[(size_t)k * RT * 64 * 4];
            const size_t o = (size_t)group * a.N + c + (t ? cols : 0);
            z[t] = (float)sum * rs.s * a.ws[o] * (rs.far ? 0x1p64f : 1.0f);
            if (a.bias) z[t] += mm_ld(static_cast<const T*>(a.bias) + o);
        }
        float v;
        if constexpr (GLU)
            v = z[0] / (1.0f + expf(-z[0])) * z[1];
        else
            v = mm_act(z[0], a.act);
        const size_t o = (size_t)r * a.ldy + c;
        if (a.residual) v += mm_ld(static_cast<const T*>(a.residual) + o);
        mm_st(static_cast<T*>(a.y) + o, v);
    }
}

// Waves of a workgroup along the contraction: all 8 from 8 steps on, fewer
// while a share would be empty.
int w8_kw(int K) {
    int kw = W8_WAVES;
    while (kw > 1 && kw > K / W8_STEP) kw >>= 1;
    return kw;
}

// Workgroup rows of a grouped call: one per chunk that there can be, or per row
// where that is fewer.
int w8_rows_of_grid(int P, int E) {
    const int most = P / 16 + (E < P ? E : P);
    return most < P ? most : P;
}

// Two row tiles per wave once that leaves nearly a workgroup per CU: x is read
// half as often (16 rows of 7168 -> 7168 13.4 against 16.2 us, one row 11.3
// against 11.9).
bool w8_two(int N, int gy, int ng) { return (int64_t)((N + 31) / 32) * gy >= 200 * ng; }

template <typename T>
hipError_t w8_run(const M8Args& a, hipStream_t s) {
    const int kw = w8_kw(a.K), ng = W8_WAVES / kw;
    const int most = a.offsets ? w8_rows_of_grid(a.P, a.E) : 1;
    const int scan = a.offsets && most < a.P;
    const uint32_t gy = a.offsets ? (uint32_t)most : (uint32_t)((a.P + 15) / 16);
    const bool glu = a.act == MM_SWIGLU;
    const bool two = glu || w8_two(a.N, most, ng);
    const int per = glu ? 16 : (two ? 32 : 16), cols = glu ? a.N / 2 : a.N;
    const dim3 g((uint32_t)((cols + per * ng - 1) / (per * ng)), gy);
    if (glu)
        w8_kernel<T, 2, true><<<g, 64 * W8_WAVES, 0, s>>>(a, kw, scan);
    else if (two)
        w8_kernel<T, 2, false><<<g, 64 * W8_WAVES, 0, s>>>(a, kw, scan);
    else
        w8_kernel<T, 1, false><<<g, 64 * W8_WAVES, 0, s>>>(a, kw, scan);
    return hipGetLastError();
}

}  // namespace

// Products that take these kernels.  Up to 8 rows (16 below 32768 columns, and
// of groups) the weights come from memory once in either kernel, and these read
// them faster: 9 rows of 7168 -> 7168 13.3 us against 16.0 on the tiles, 16 of
// 7168 -> 131072 176 / 162; at worst 12 rows of 4096 -> 16384 17.0 / 16.0.  More
// rows read small weights again from L2 for each 16, which the tiles' latency
// outlasts for a while (301 x 1459 -> 331 4.8 / 8.3, 1200 10.4 / 8.5; 903 rows
// of 7 groups 459 -> 331 7.0 / 9.3), and few rows of many groups read them once
// here too (64 of 256 groups 7168 -> 4096 269 / 300, 256 of 256 807 / 817):
// there an estimate decides, of the time for all workgroups, for a wave's steps
// and for the bytes read, fitted together with the tiles'.
bool m8_rows_takes(int P, int K, int N, int E, double tile_us) {
    if (E > 1 ? P <= 16 : P <= 8 || (P <= 16 && N < 32768)) return true;
    if (P > 1 << 19) return false;   // (chunks are a dimension of the grid, at most 65535)
    const int kw = w8_kw(K), ng = W8_WAVES / kw;
    const double chunks = E == 1 ? (P + 15) / 16 : P / 16.0 + (E < P ? E : P) / 2.0;
    const bool two = w8_two(N, E == 1 ? 1 : w8_rows_of_grid(P, E), ng);
    const int per = (two ? 32 : 16) * ng;
    const double wgs = chunks * ((N + per - 1) / per) / 256.0;   // per CU
    const int steps = ((K / W8_STEP + kw - 1) / kw + (K % W8_STEP != 0)) * (two ? 2 : 1);
    const double mb = chunks * N * K / (1 << 20);
    if (E == 1) return 1.75 + 0.565 * wgs + 0.274 * steps + 0.12 * mb < tile_us;
    return 2.15 + 0.795 * wgs + 0.032 * steps + 0.204 * mb < tile_us + 3.0;   // (a plan, or scans, on top)
}

hipError_t launch_m8_rows(const M8Args& a, bool f32, hipStream_t s) {
    return f32 ? w8_run<float>(a, s) : w8_run<uint16_t>(a, s);
}

}  // namespace ds4
