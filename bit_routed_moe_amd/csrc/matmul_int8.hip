// Products in 8-bit integers on the matrix cores (v_mfma_i32_16x16x64_i8).
//
// A workgroup computes BR x BC outputs in stages of 128 or 64 contraction
// columns (as many bytes of every tile row), which global_load_lds_dwordx4
// brings into a ring of LDS buffers without passing through registers.  Of a
// row of 128 bytes the 16-byte chunk c lies in slot c ^ ((r >> 1) & 7), of 64
// bytes in c ^ (-(r >> 2) & 3): a fragment read (ds_read_b128 of 16 rows at one
// chunk per lane quarter) then meets no bank twice (counter: 0 conflicts; 46%
// of the LDS cycles with c ^ ((r >> 2) & 3)).  One barrier per stage.  In the
// tiles that have a CU to themselves fragments are read one step of 64 columns
// ahead of the matrix instructions that take them; workgroups that share a CU
// cover each other's waits, and skip the row tiles that a group's last chunk
// lacks.  The column operand goes first into the matrix instruction, so a lane
// holds 4 consecutive columns of one row; results leave through LDS in whole
// rows, after the epilogue.
//
// 4096 x 7168 -> 4096: 104 to 108 us by run, 2.2 to 2.3 POP/s (2.4 at 8192^3,
// where the library's plain product reaches 2.1).  The matrix cores are busy 57%
// of the cycles at 1.84 GHz: what switches sets the clock (all codes 1: 2.9
// POP/s).  Variants with fewer LDS reads (4 waves of 128 x 128 outputs, 2.2 POP/s
// at 2.07 GHz and 48% busy) or larger matrix instructions (32x32x32: 3.1 POP/s on
// equal codes, 2.2 on random ones) gain nothing there.  Groups of few rows are
// bound by their weights: 4096 tokens' down products of 256 experts (3.9 GB read,
// 0.47 GB written) take 986 to 1026 us, 4.3 TB/s; 16 rows for each expert 700 us,
// 5.5 TB/s.
// Of those, 128 x 256 tiles of 64-column stages, two workgroups per CU, take 3
// to 10% less than one of three 128-column stages.
#include <type_traits>

#include "matmul_int8.hpp"
#include "tile.hpp"

namespace ds4 {

namespace {

constexpr int M8_K = 128;          // contraction columns that the estimate counts as a stage
constexpr int M8_MAX_SPLITS = 16;  // of the contraction
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// One operand of BT tile rows of KB bytes staged by NW waves.
template <int BT, int NW, int KB>
struct M8Operand {
    static constexpr int CPR = KB / 16, RPD = 1024 / KB;   // 16-byte chunks per row, rows per DMA
    static constexpr int BYTES = BT * KB;
    static constexpr int ND = BYTES / 1024 / NW;   // DMAs per wave and stage
    static_assert(ND * NW * 1024 == BYTES, "whole DMAs per wave");
    // tile row and chunk that DMA i of wave w brings for this lane
    static __device__ __forceinline__ int row(int i, int w, int lane) { return (i * NW + w) * RPD + lane / CPR; }
    // what a row's chunks are moved by
    static __device__ __forceinline__ int place(int row) { return KB == 128 ? (row >> 1) & 7 : -(row >> 2) & 3; }
    static __device__ __forceinline__ int chunk(int row, int lane) { return (lane % CPR) ^ place(row); }
    // Fragment t (16 tile rows from t0 + 16 * t on) of k-step ks.
    static __device__ __forceinline__ i32x4 frag(const uint8_t* buf, int t0, int t, int ks, int lane) {
        const int m = lane & 15, q = lane >> 4, r = t0 + 16 * t + m;
        return *reinterpret_cast<const i32x4*>(buf + r * KB + (((ks * 4 + q) ^ place(m)) << 4));
    }
    // Zeros from contraction column krem of the stage on (of one operand: the
    // other's bytes there are then multiplied by zero).
    static __device__ __forceinline__ void clear_tail(uint8_t* buf, int krem, int tid) {
        for (int i = tid; i < BT * CPR; i += NW * 64) {
            const int r = i / CPR, c = i % CPR;
            uint8_t* p = buf + r * KB + ((c ^ place(r)) << 4);
            if (16 * c >= krem)
                *reinterpret_cast<u32x4*>(p) = u32x4{0, 0, 0, 0};
            else
                for (int j = krem - 16 * c; j < 16; ++j) p[j] = 0;
        }
    }
};

// 8 sums of a row from a wave's LDS region: rows of CW values, 16-byte chunk c
// of row r at c ^ r (modulo the row's chunks).
template <int CW>
__device__ __forceinline__ void m8_get8(const uint8_t* reg, int r, int col, int32_t (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const i32x4 x = *reinterpret_cast<const i32x4*>(reg + r * (CW * 4) + ((((col >> 2) + h) ^ (r & (CW / 4 - 1))) << 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = x[i];
    }
}

__device__ __forceinline__ void m8_part8(int32_t* p, const int32_t (&v)[8], int n, bool vec) {
    if (vec) {
        reinterpret_cast<i32x4*>(p)[0] = i32x4{v[0], v[1], v[2], v[3]};
        reinterpret_cast<i32x4*>(p)[1] = i32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}

// WR x WC waves, each (BR / WR) x (BC / WC) outputs; ST stage buffers of KB
// contraction columns; PIPE: fragments read a step ahead (where workgroups
// share a CU they cover each other's waits); WPS waves per SIMD.
template <int BR, int BC, int WR, int WC, int KB, int ST, bool PIPE, int WPS, typename T>
__global__ __launch_bounds__(64 * WR * WC, WPS) void m8_kernel(M8Args a, int tr, int tc) {
    constexpr int NW = WR * WC;
    using RowOp = M8Operand<BR, NW, KB>;
    using ColOp = M8Operand<BC, NW, KB>;
    constexpr int STB = RowOp::BYTES + ColOp::BYTES;
    constexpr int MI = BR / WR / 16, NI = BC / WC / 16;
    constexpr int LPS = RowOp::ND + ColOp::ND;   // DMAs per wave and stage
    static_assert(KB == 128 || (KB == 64 && !PIPE), "PIPE has two steps of 64 columns");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[ST * STB];
    const uint32_t lds32 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);

    // this workgroup's tile: each of the 8 XCDs (workgroup id modulo 8) takes
    // a contiguous eighth of the tiles that exist
    const int slot = (int)blockIdx.x >> 3;
    auto tile_of = [&](int ntr, int& t) {
        const int total = ntr * tc, per = (total + 7) >> 3;
        t = ((int)blockIdx.x & 7) * per + slot;
        return slot < per && t < total;
    };
    int t, rt, ct;
    MmChunk ch;
    if (a.E > 1 && !a.chunks) {
        // without a plan: a scan over the groups' numbers of chunks (a group's
        // tiles follow one another, so that its weights are read once)
        __shared__ int tmp[32], found[4];
        constexpr int G = 1024 / (64 * NW);
        int r0[G], cnt[G], sum = 0, total;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            r0[i] = cnt[i] = 0;
            if (G * tid + i < a.E) mm_group_rows(a.offsets, G * tid + i, a.P, r0[i], cnt[i]);
            sum += (cnt[i] + BR - 1) / BR;
        }
        int first = block_exclusive_scan(sum, tmp, &total);
        if (!tile_of(min(total, a.max_chunks), t)) return;
        const int c = t / tc;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int n = (cnt[i] + BR - 1) / BR;
            if (c >= first && c < first + n) {
                found[0] = G * tid + i;
                found[1] = r0[i];
                found[2] = cnt[i];
                found[3] = first;
            }
            first += n;
        }
        __syncthreads();
        const int n = __builtin_amdgcn_readfirstlane(found[2]);
        mt_tile(t - __builtin_amdgcn_readfirstlane(found[3]) * tc, (n + BR - 1) / BR, tc, rt, ct);
        ch.group = __builtin_amdgcn_readfirstlane(found[0]);
        ch.row0 = __builtin_amdgcn_readfirstlane(found[1]) + rt * BR;
        ch.n = min(BR, n - rt * BR);
    } else {
        const int ntr = a.chunks ? a.n_chunks[0] : tr;
        if (!tile_of(ntr, t)) return;
        if (a.chunks) {
            const int c = t / tc;
            const MmChunk o = a.chunks[c];
            int r0, n;
            mm_group_rows(a.offsets, o.group, a.P, r0, n);
            const int first = c - o.index;
            mt_tile(t - first * tc, (n + BR - 1) / BR, tc, rt, ct);
            rt += first;
        } else {
            mt_tile(t, ntr, tc, rt, ct);
        }
        if (!mm_chunk(a, rt, BR, ch)) return;
    }
    const int c0 = ct * BC;
    const bool glu = a.act == MM_SWIGLU;
    const int8_t* const wg = static_cast<const int8_t*>(a.w) + (size_t)ch.group * a.N * a.ldw;

    // the DMAs' source rows; a lane's chunk is the same in all of a wave's
    // DMAs, whose rows differ by a multiple of 16
    static_assert((NW * RowOp::RPD) % 16 == 0, "one chunk per lane");
    const int rrow = RowOp::row(0, w, lane), crow = ColOp::row(0, w, lane);
    const int chunk = RowOp::chunk(rrow, lane);   // (rrow == crow)
    const int8_t* rsrc[RowOp::ND];
    const int8_t* csrc[ColOp::ND];
#pragma unroll
    for (int i = 0; i < RowOp::ND; ++i)
        rsrc[i] = static_cast<const int8_t*>(a.x) +
                  (size_t)mm_src(a, ch.row0 + min(rrow + i * NW * RowOp::RPD, ch.n - 1)) * a.ldx;
#pragma unroll
    for (int i = 0; i < ColOp::ND; ++i) {
        const int n = mm_col(a, glu, c0, crow + i * NW * ColOp::RPD);
        csrc[i] = wg + (size_t)(n < 0 ? a.N - 1 : n) * a.ldw;
    }
    const int kchunk = (a.K - 1) / 16;
    auto issue1 = [&](int st, int i) {   // DMA i (0 .. LPS-1) of stage st
        const uint32_t buf = lds32 + (uint32_t)(st % ST) * STB;
        const int off = 16 * min(st * (KB / 16) + chunk, kchunk);
        if (i < RowOp::ND)
            mt_dma16(rsrc[i] + off, buf + (uint32_t)(i * NW + w) * 1024u);
        else
            mt_dma16(csrc[i - RowOp::ND] + off, buf + RowOp::BYTES + (uint32_t)((i - RowOp::ND) * NW + w) * 1024u);
    };
    auto issue = [&](int st) {
#pragma unroll
        for (int i = 0; i < LPS; ++i) issue1(st, i);
    };

    i32x4 acc[NI][MI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    // a wave's first row and column of the tile; its row tiles of 16 follow one
    // another with PIPE, else they alternate with the other waves' (who then
    // share the rows of a chunk that does not fill the tile)
    constexpr int RT = PIPE ? 1 : WR;
    const int wr0 = (w % WR) * (PIPE ? BR / WR : 16), wc0 = (w / WR) * (BC / WC);
    // stages [sb, ns) of the contraction: all, or this split's share
    const int nall = (a.K + KB - 1) / KB;
    const int each = (nall + a.ksplits - 1) / a.ksplits;
    const int sb = min(nall, (int)blockIdx.z * each), ns = min(nall, sb + each);
    auto clear_tail = [&](int st) {   // behind the contraction's end, in the last stage
        if (st == nall - 1 && a.K % KB) {
            RowOp::clear_tail(lds + (st % ST) * STB, a.K % KB, tid);
            __syncthreads();
        }
    };
    // Matrix instructions on fragments rf, cf while the next ones are read
    // from step ks of stage st (and, with more, stage `more`'s DMAs issued),
    // spread over the row tiles.
    auto step = [&](const i32x4 (&rf)[MI], const i32x4 (&cf)[NI], i32x4 (&rn)[MI], i32x4 (&cn)[NI], int st, int ks,
                    int more) {
        const uint8_t* buf = lds + (st % ST) * STB;
#pragma unroll
        for (int j = 0; j < MI; ++j) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (i * MI / NI == j) cn[i] = ColOp::frag(buf + RowOp::BYTES, wc0, i, ks, lane);
            rn[j] = RowOp::frag(buf, wr0, RT * j, ks, lane);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(cf[i], rf[j], acc[i][j], 0, 0, 0);
            if (more >= 0) {
#pragma unroll
                for (int i = 0; i < LPS; ++i)
                    if (i * MI / LPS == j) issue1(more, i);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if constexpr (PIPE) {
        if (sb < ns) {
#pragma unroll
            for (int s = 0; s < ST; ++s)
                if (sb + s < ns) issue(sb + s);
            if (sb + ST <= ns)
                mt_wait_vm<(ST - 1) * LPS>();
            else
                mt_wait_vm<0>();
            mt_barrier();
            clear_tail(sb);
            i32x4 rf[2][MI], cf[2][NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) cf[0][i] = ColOp::frag(lds + (sb % ST) * STB + RowOp::BYTES, wc0, i, 0, lane);
#pragma unroll
            for (int j = 0; j < MI; ++j) rf[0][j] = RowOp::frag(lds + (sb % ST) * STB, wr0, RT * j, 0, lane);
            for (int st = sb; st < ns; ++st) {
                step(rf[0], cf[0], rf[1], cf[1], st, 1, -1);
                // stage st is read; stage st + 1 has to have landed
                if (ST > 2 && st + ST - 1 < ns)
                    mt_wait_vm<(ST - 2) * LPS>();
                else
                    mt_wait_vm<0>();
                mt_barrier();
                if (st + 1 < ns) clear_tail(st + 1);
                // (past the last stage the fragments read are not used)
                step(rf[1], cf[1], rf[0], cf[0], st + 1, 0, st + ST < ns ? st + ST : -1);
            }
        }
    } else {
        if (sb < ns) {
#pragma unroll
            for (int s = 0; s < ST - 1; ++s)
                if (sb + s < ns) issue(sb + s);
        }
        // Of a chunk with fewer rows than the tile (the end of a group) only
        // the row tiles that exist are multiplied.
        auto stages = [&](auto whole) {
            for (int st = sb; st < ns; ++st) {
                if (ST > 2 && st + ST - 2 < ns)
                    mt_wait_vm<(ST - 2) * LPS>();
                else
                    mt_wait_vm<0>();
                mt_barrier();
                if (st + ST - 1 < ns) issue(st + ST - 1);
                clear_tail(st);
                const uint8_t* buf = lds + (st % ST) * STB;
#pragma unroll
                for (int ks = 0; ks < KB / 64; ++ks) {
                    i32x4 rf[MI], cf[NI];
#pragma unroll
                    for (int i = 0; i < NI; ++i) cf[i] = ColOp::frag(buf + RowOp::BYTES, wc0, i, ks, lane);
                    if constexpr (decltype(whole)::value) {
#pragma unroll
                        for (int j = 0; j < MI; ++j) rf[j] = RowOp::frag(buf, wr0, RT * j, ks, lane);
                    }
#pragma unroll
                    for (int j = 0; j < MI; ++j) {
                        if (decltype(whole)::value || wr0 + 16 * RT * j < ch.n) {
                            if constexpr (!decltype(whole)::value) rf[j] = RowOp::frag(buf, wr0, RT * j, ks, lane);
#pragma unroll
                            for (int i = 0; i < NI; ++i)
                                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(cf[i], rf[j], acc[i][j], 0, 0, 0);
                        }
                    }
                }
            }
        };
        if (ch.n > BR - 16)
            stages(std::true_type{});
        else
            stages(std::false_type{});
    }

    // Out through LDS, RP rows of the wave's tile at a time.  In the
    // accumulators a lane holds columns 4q .. 4q+3 of row m of each 16 x 16
    // block.
    constexpr int CW = BC / WC, WROWS = BR / WR;
    constexpr int FIT = ST * STB / NW / (CW * 4);   // rows of the wave's region
    constexpr int RP = FIT >= WROWS ? WROWS : (FIT >= WROWS / 2 ? WROWS / 2 : WROWS / 4);
    static_assert(RP >= 16 && RP % 16 == 0 && RP <= FIT && (CW & (CW - 1)) == 0 && CW >= 32, "passes of whole row tiles");
    int32_t* const part = a.ksplits > 1 ? a.ipart + (size_t)blockIdx.z * a.kpart_stride : nullptr;
    uint8_t* reg = lds + w * (RP * CW * 4);
    auto row_of = [&](int i) { return wr0 + 16 * RT * (i >> 4) + (i & 15); };   // tile row of the wave's row i
    __syncthreads();
#pragma unroll
    for (int p = 0; p < WROWS / RP; ++p) {
        const int m = lane & 15, q = lane >> 4;
#pragma unroll
        for (int j = 0; j < RP / 16; ++j)
#pragma unroll
            for (int i = 0; i < NI; ++i)
                *reinterpret_cast<i32x4*>(reg + (16 * j + m) * (CW * 4) + (((4 * i + q) ^ (m & (CW / 4 - 1))) << 4)) =
                    acc[i][p * (RP / 16) + j];
        if (glu) {
            // 16 gate columns, then the 16 up columns they pair with
            constexpr int LR = CW / 16;   // lanes per row
            const int half = a.N >> 1;
            const int c8 = lane & (LR - 1), col = 32 * (c8 >> 1) + 8 * (c8 & 1);
            const int f = ((c0 + wc0) >> 1) + 8 * c8, cnt = half - f;
#pragma unroll 1
            for (int rr = lane / LR; rr < RP; rr += 64 / LR) {
                int32_t g[8], u[8];
                m8_get8<CW>(reg, rr, col, g);
                m8_get8<CW>(reg, rr, col + 16, u);
                const int at = row_of(p * RP + rr);
                if (at >= ch.n || cnt <= 0) continue;
                const int r = ch.row0 + at;
                if (part) {
                    int32_t* o = part + (size_t)r * a.ldp + f;
                    m8_part8(o, g, cnt, cnt >= 8);
                    m8_part8(o + half, u, cnt, cnt >= 8 && (half & 3) == 0);
                } else {
                    const float xs = a.xs[mm_src(a, r)];
                    float zg[8], zu[8];
                    m8_z8<T>(a, ch.group, xs, f, cnt, g, zg);
                    m8_z8<T>(a, ch.group, xs, half + f, cnt, u, zu);
                    m8_out8<T, true>(a, r, f, cnt, zg, zu);
                }
            }
        } else {
            constexpr int LR = CW / 8;
            const int col = 8 * (lane & (LR - 1)), n = c0 + wc0 + col, cnt = a.N - n;
#pragma unroll 1
            for (int rr = lane / LR; rr < RP; rr += 64 / LR) {
                int32_t v[8];
                m8_get8<CW>(reg, rr, col, v);
                const int at = row_of(p * RP + rr);
                if (at >= ch.n || cnt <= 0) continue;
                const int r = ch.row0 + at;
                if (part) {
                    m8_part8(part + (size_t)r * a.ldp + n, v, cnt, cnt >= 8);
                } else {
                    float z[8];
                    m8_z8<T>(a, ch.group, a.xs[mm_src(a, r)], n, cnt, v, z);
                    m8_out8<T, false>(a, r, n, cnt, z, nullptr);
                }
            }
        }
    }
}

// Joins the splits of a product and finishes the rows as the tile kernel
// would: 8 rows of 256 columns per workgroup, rows 8 * blockIdx.z on of one
// chunk.
template <typename T>
__global__ __launch_bounds__(256) void m8_join_kernel(M8Args a, int bm) {
    MmChunk ch;
    if (!mm_chunk(a, blockIdx.y, bm, ch)) return;
    const int rr = blockIdx.z * 8 + (threadIdx.x >> 5);
    if (rr >= ch.n) return;
    const int r = ch.row0 + rr, half = a.N >> 1;
    const bool glu = a.act == MM_SWIGLU;
    const int n = blockIdx.x * 256 + 8 * (threadIdx.x & 31), cnt = (glu ? half : a.N) - n;
    if (cnt <= 0) return;
    auto sum8 = [&](int c, bool vec, int32_t (&v)[8]) {
        const int32_t* p = a.ipart + (size_t)r * a.ldp + c;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0;
        if (vec) {
#pragma unroll 4
            for (int s = 0; s < a.ksplits; ++s) {
                const i32x4* x = reinterpret_cast<const i32x4*>(p + s * a.kpart_stride);
                const i32x4 lo = x[0], hi = x[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] += lo[i];
                    v[4 + i] += hi[i];
                }
            }
        } else {
            for (int s = 0; s < a.ksplits; ++s)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < cnt) v[i] += p[s * a.kpart_stride + i];
        }
    };
    const float xs = a.xs[mm_src(a, r)];
    int32_t v[8];
    float z[8];
    sum8(n, cnt >= 8, v);
    m8_z8<T>(a, ch.group, xs, n, cnt, v, z);
    if (glu) {
        float u[8];
        sum8(half + n, cnt >= 8 && (half & 3) == 0, v);
        m8_z8<T>(a, ch.group, xs, half + n, cnt, v, u);
        m8_out8<T, true>(a, r, n, cnt, z, u);
    } else {
        m8_out8<T, false>(a, r, n, cnt, z, nullptr);
    }
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Tile shapes, with the times that the estimate takes (us): lat per stage of
// 128 contraction columns and end for its start and writing, of a workgroup by
// itself on its CU; the same per workgroup and CU when the chip is full, where
// workgroups that share a CU (`one`: none do) hide each other's ends.  The
// numbers are fitted to 842 products (10 .. 37000 rows, dense and of 2 .. 256
// groups, 64 .. 8192 x 64 .. 8192), each timed in every shape and split and, up
// to 2000 rows, on the few-row kernel: what m8_pick takes is 1.2% off the best
// in the mean, over 10% off in 5% of them, at most 43%.  Of 320 products that
// the fit had not seen it is 1.8% off in the mean and over 10% in 25 (at worst
// 4115 rows of 109 groups 86 -> 269, 16.2 us against 10.1).
struct M8Shape {
    int br, bc;
    double lat, end, full_lat, full_end;
    bool one;
};
constexpr M8Shape M8_SHAPES[] = {{256, 256, 0.926, 1.34, 1.58, 8.0, true},
                                 {128, 256, 0.738, 1.41, 0.842, 6.31, true},
                                 {128, 256, 0.937, 2.82, 1.108, 1.92, false},
                                 {128, 128, 0.434, 2.73, 0.54, 0.85, false},
                                 {64, 64, 0.363, 2.65, 0.143, 0.93, false}};
constexpr int M8_NSHAPES = 5;
constexpr double M8_JOIN = 1.5;     // us of a join launch
constexpr double M8_MEM = 2.1e6;    // bytes per us of partial sums
constexpr double M8_READ = 18.5e6;  // bytes per us of both operands into LDS, of groups whose weights
constexpr double M8_FAR = 13.6e6;   // the 256 MB of the memory-side cache hold, or not
// Workgroups per CU up to which each scans for its chunk: 256 rows of 8 groups
// 2048 -> 2048 13.2 us against 14.9 with a plan launch, 4096 of 8 41.8 / 42.3,
// but 32768 of 64 256 -> 4096 290 / 249, 16000 of 1000 512 -> 512 78 / 63.
constexpr double M8_SCANS = 4.0;

// Tile shape and contraction splits of the least estimated time.
M8Pick m8_tile_pick(int P, int K, int N, int E) {
    const int live = E < P ? E : P;
    const int all = cdiv(K, M8_K);
    M8Pick best{0, 1, 1e300};
    for (int i = 0; i < M8_NSHAPES; ++i) {
        const M8Shape& t = M8_SHAPES[i];
        double tr = cdiv(P, t.br);   // row tiles; of ragged groups about half a tile each is not filled
        if (E > 1) tr = (double)P / t.br + 0.5 * live > live ? (double)P / t.br + 0.5 * live : live;
        const double tiles = tr * cdiv(N, t.bc);
        for (int s = 1; s <= M8_MAX_SPLITS && (s == 1 || (i >= 3 && all / s >= 4 && tiles * s <= 512.0)); s *= 2) {
            const int stages = cdiv(all, s);
            double per_cu = tiles * s / 256.0;
            if (t.one) per_cu = (double)(int64_t)(per_cu + 0.999);
            const double alone = t.lat * stages + t.end, full = per_cu * (t.full_lat * stages + t.full_end);
            double us = alone > full ? alone : full;
            if (E > 1) {
                const double read = tiles * (t.br + t.bc) * K /
                                    ((double)live * N * K < (double)(1 << 28) ? M8_READ : M8_FAR);
                us = us > read ? us : read;
            }
            if (s > 1) us += M8_JOIN + tiles * s * t.br * t.bc * 8.0 / M8_MEM;
            if (us < best.us) best = M8Pick{i, s, us};
        }
    }
    return best;
}

template <int BR, int BC, int WR, int WC, int KB, int ST, bool PIPE, int WPS, typename T>
hipError_t m8_launch(const M8Args& a, hipStream_t s) {
    const int tr = a.E > 1 ? a.max_chunks : cdiv(a.P, BR), tc = cdiv(a.N, BC);
    const int64_t total = (int64_t)tr * tc;
    const dim3 g((uint32_t)((total + 7) / 8 * 8), 1, (uint32_t)a.ksplits);
    m8_kernel<BR, BC, WR, WC, KB, ST, PIPE, WPS, T><<<g, 64 * WR * WC, 0, s>>>(a, tr, tc);
    if (a.ksplits > 1) {
        const dim3 j((uint32_t)cdiv(a.act == MM_SWIGLU ? a.N / 2 : a.N, 256), (uint32_t)tr, BR / 8u);
        m8_join_kernel<T><<<j, 256, 0, s>>>(a, BR);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t m8_run(const M8Args& a, int shape, hipStream_t s) {
    switch (shape) {
        case 0: return m8_launch<256, 256, 2, 4, 128, 2, true, 2, T>(a, s);
        case 1: return m8_launch<128, 256, 2, 4, 128, 3, true, 2, T>(a, s);
        case 2: return m8_launch<128, 256, 2, 4, 64, 3, false, 4, T>(a, s);
        case 3: return m8_launch<128, 128, 2, 4, 128, 2, false, 4, T>(a, s);
        default: return m8_launch<64, 64, 2, 2, 128, 3, false, 2, T>(a, s);
    }
}

}  // namespace

M8Pick m8_pick(int P, int K, int N, int E) {
    const M8Pick tile = m8_tile_pick(P, K, N, E);
    return m8_rows_takes(P, K, N, E, tile.us) ? M8Pick{-1, 1, 0.0} : tile;
}

int m8_chunk_rows(const M8Pick& pick) { return pick.shape < 0 ? 0 : M8_SHAPES[pick.shape].br; }

bool m8_wants_plan(const M8Pick& pick, int P, int N, int E) {
    const M8Shape& t = M8_SHAPES[pick.shape];
    const double tiles = ((double)P / t.br + 0.5 * (E < P ? E : P)) * cdiv(N, t.bc);
    return pick.splits > 1 || tiles > M8_SCANS * 256.0;
}

size_t m8_split_bytes(const M8Pick& pick, int P, int N) {
    return pick.splits > 1 ? (size_t)pick.splits * P * ((N + 7) / 8 * 8) * 4 : 0;
}

size_t m8_split_bound(int P, int K, int N) {
    // at most 512 tiles of up to 128 x 128 in all splits together, and at most
    // M8_MAX_SPLITS splits
    if (cdiv(K, M8_K) < 8) return 0;
    const int64_t all = M8_MAX_SPLITS * (int64_t)P * ((N + 7) / 8 * 8), cap = (int64_t)512 * 128 * 128;
    return (size_t)(all < cap ? all : cap) * 4;
}

hipError_t launch_m8(const M8Args& a0, const M8Pick& pick, bool f32, hipStream_t s) {
    if (pick.shape < 0) return launch_m8_rows(a0, f32, s);
    M8Args a = a0;
    a.ksplits = pick.splits;
    a.ldp = (a.N + 7) / 8 * 8;
    a.kpart_stride = (size_t)a.P * a.ldp;
    return f32 ? m8_run<float>(a, pick.shape, s) : m8_run<uint16_t>(a, pick.shape, s);
}

}  // namespace ds4
