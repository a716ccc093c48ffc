// bf16 products at original precision on the matrix cores
// (v_mfma_f32_16x16x32_bf16, fp32 accumulation), for forward, dgrad and wgrad.
//
// Every mode is C[row][col] = sum_k R(row, k) Q(col, k), where an operand is
// either contiguous along the contraction (x and w forward, dz in dgrad) or
// along the tile (w in dgrad, dz and x in wgrad):
//   forward  rows: token rows (gathered), cols: weight rows, k: in_dim
//   dgrad    rows: dz rows,               cols: in_dim,      k: out_dim
//   wgrad    rows: out_dim,               cols: in_dim,      k: the group's rows
//
// A workgroup computes BR x BC outputs in stages of 64 contraction columns,
// which global_load_lds_dwordx4 brings into a ring of LDS buffers without
// passing through registers.  One barrier per stage: behind it the stage's
// buffer may be filled again, and a later stage has landed.  In the 256-wide
// tiles, one workgroup per CU, fragments are read one step of 32 columns ahead
// of the matrix instructions that take them and the barrier stands in the
// stage's middle (dgrad 129 -> 113 us, wgrad 134 -> 117 us at 4096 x 7168 x
// 2048); of the smaller ones several share a CU and cover each other's waits.
//   Contiguous along k: tile row r is 128 bytes, its 16-byte chunk c in slot
//     c ^ ((r >> 1) & 7), so a fragment read (16 rows at one chunk per lane
//     quarter, ds_read_b128) covers all 64 banks.
//   Contiguous along the tile: contraction row k is one LDS row, its 32-byte
//     granule g (16 columns) in place g ^ (k & 3 | (k >> 3 & 1) << 2) (64
//     columns: g ^ (k >> 1 & 1 | (k >> 3 & 1) << 1)); the fragment is read
//     transposed (ds_read_b64_tr_b16: 16 lanes take 4 contraction rows x 16
//     columns, and a lane gets its column's 4 values).
// Counters: no LDS bank conflicts in any mode; at 256 x 256 matrix cores busy
// 61% (forward), 49% (dgrad) and 46% (wgrad) of the cycles.  1.2 PFLOP/s at 4096
// x 7168 -> 4096 with SwiGLU (201 us; the library's plain product 169), 1.07
// over dx and dW of 4096 rows, 7168 -> 2048 (109 + 115 us).  Groups of few rows
// are bound by their weights (4096 tokens' down products of 256 experts at 4.1
// TB/s), their dW by each tile's start and writing (25% busy).
// The column operand goes first into the matrix instruction, so a lane holds 4
// consecutive columns of one row of C; they leave through LDS in whole rows.
#include "matmul.hpp"
#include "tile.hpp"

namespace ds4 {

namespace {

constexpr int MT_K = 64;            // contraction columns per stage
constexpr int MT_MAX_SPLITS = 16;   // of the contraction
constexpr int MT_RING = 2048;       // wgrad: row numbers kept in LDS
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// One operand of BT tile rows (or columns) staged by NW waves.
template <bool STRIDED, int BT, int NW>
struct MtOperand {
    static constexpr int BYTES = BT * MT_K * 2;
    static constexpr int ND = BYTES / 1024 / NW;   // DMAs per wave and stage
    static_assert(ND * NW * 1024 == BYTES, "whole DMAs per wave");
    static constexpr int CPR = STRIDED ? BT / 8 : 8;   // 16-byte chunks per LDS row
    static constexpr int RPD = 64 / CPR;               // LDS rows per DMA

    // what a strided operand's granules of LDS row k are moved by
    static __device__ __forceinline__ int place(int k) {
        if constexpr (BT >= 128) return (k & 3) | ((k >> 1) & 4);
        return ((k >> 1) & 1) | ((k >> 2) & 2);   // (two rows per 64 banks)
    }
    // LDS row and chunk that DMA i of wave w brings for this lane
    static __device__ __forceinline__ int lds_row(int i, int w, int lane) { return (i * NW + w) * RPD + lane / CPR; }
    static __device__ __forceinline__ int chunk(int row, int lane) {
        const int s = lane % CPR;
        if constexpr (STRIDED) return s ^ (place(row) << 1);
        return s ^ ((row >> 1) & 7);
    }
    // Fragment t (16 tile rows from t0 + 16 * t on) of k-step ks.
    static __device__ __forceinline__ bf16x8 frag(const uint8_t* buf, int t0, int t, int ks, int lane) {
        const int m = lane & 15, q = lane >> 4;
        if constexpr (STRIDED) {
            const int k = 8 * q + (m >> 2), g = (t0 >> 4) + t;   // (the step's 32 and the half's 4 do not move place)
            const uint8_t* p = buf + (ks * 32 + k) * (BT * 2) + ((g ^ place(k)) << 5) + (m & 3) * 8;
            typedef __attribute__((address_space(3))) s16x4 lds4;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * BT * 2));
            return __builtin_bit_cast(bf16x8, s16x8(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)));
        } else {
            const int r = t0 + 16 * t + m;
            return *reinterpret_cast<const bf16x8*>(buf + r * 128 + (((ks * 4 + q) ^ (m >> 1)) << 4));
        }
    }
    // Zeros from contraction column krem of the stage on.
    static __device__ __forceinline__ void clear_tail(uint8_t* buf, int krem, int tid) {
        if constexpr (STRIDED) {
            for (int i = krem * (BT / 8) + tid; i < MT_K * (BT / 8); i += NW * 64)
                *reinterpret_cast<u32x4*>(buf + i * 16) = u32x4{0, 0, 0, 0};
        } else {
            for (int i = tid; i < BT * 8; i += NW * 64) {
                const int r = i >> 3, c = i & 7;
                uint8_t* p = buf + r * 128 + ((c ^ ((r >> 1) & 7)) << 4);
                if (8 * c >= krem)
                    *reinterpret_cast<u32x4*>(p) = u32x4{0, 0, 0, 0};
                else
                    for (int j = krem - 8 * c; j < 8; ++j) reinterpret_cast<uint16_t*>(p)[j] = 0;
            }
        }
    }
};

// 8 values of a row (vec: the address is 16-byte aligned and all 8 exist).
__device__ __forceinline__ void mt_st8(uint16_t* p, const float (&v)[8], int n, bool vec) {
    if (vec) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<u32x4*>(p) = o;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint16_t)f32_to_bf16(v[i]);
    }
}
__device__ __forceinline__ void mt_st8(float* p, const float (&v)[8], int n, bool vec) {
    if (vec) {
        reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
        reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}
__device__ __forceinline__ void mt_add8(float (&v)[8], const uint16_t* p, int n, bool vec) {
    if (vec) {
        const u32x4 o = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] += __uint_as_float(o[i] << 16);
            v[2 * i + 1] += __uint_as_float(o[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) v[i] += bf16_to_f32(p[i]);
    }
}

// A wave's outputs pass through its own LDS region on their way out, so that
// the activation code exists once and rows leave in whole 16-byte pieces:
// rows of CW floats, 16-byte chunk c of row r at c ^ r (modulo the row's chunks).
template <int CW>
__device__ __forceinline__ void mt_get8(const uint8_t* reg, int r, int col, float (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(reg + r * (CW * 4) + ((((col >> 2) + h) ^ (r & (CW / 4 - 1))) << 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = x[i];
    }
}

// Forward epilogue of 8 columns from n on (cnt of them exist) of row r.
__device__ __forceinline__ void mt_out8(const MmArgs& a, const uint16_t* bias, int r, int n, int cnt, float (&v)[8]) {
    const bool vec = cnt >= 8;
    if (bias) mt_add8(v, bias + n, cnt, vec && (a.N & 7) == 0);
    if (a.z) mt_st8(static_cast<uint16_t*>(a.z) + (size_t)r * a.ldz + n, v, cnt, vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mm_act(v[i], a.act);
    const size_t o = (size_t)r * a.ldy + n;
    if (a.residual) mt_add8(v, static_cast<const uint16_t*>(a.residual) + o, cnt, vec);
    mt_st8(static_cast<uint16_t*>(a.y) + o, v, cnt, vec);
}

__device__ __forceinline__ void mt_out8_glu(const MmArgs& a, const uint16_t* bias, int r, int f, int cnt,
                                            float (&g)[8], float (&u)[8]) {
    const int half = a.N >> 1;
    const bool vec = cnt >= 8, vecu = vec && (half & 7) == 0;
    if (bias) {
        mt_add8(g, bias + f, cnt, vecu);   // (expert rows of an odd N start anywhere)
        mt_add8(u, bias + half + f, cnt, vecu);
    }
    if (a.z) {
        uint16_t* zr = static_cast<uint16_t*>(a.z) + (size_t)r * a.ldz;
        mt_st8(zr + f, g, cnt, vec);
        mt_st8(zr + half + f, u, cnt, vecu);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = g[i] / (1.0f + expf(-g[i])) * u[i];
    const size_t o = (size_t)r * a.ldy + f;
    if (a.residual) mt_add8(g, static_cast<const uint16_t*>(a.residual) + o, cnt, vec);
    mt_st8(static_cast<uint16_t*>(a.y) + o, g, cnt, vec);
}

// WR x WC waves, each (BR / WR) x (BC / WC) outputs; ST stage buffers.
template <int MODE, int BR, int BC, int WR, int WC, int ST, typename G>
__global__ __launch_bounds__(64 * WR * WC) void mt_kernel(MmArgs a, int tr, int tc) {
    constexpr int NW = WR * WC;
    using RowOp = MtOperand<MODE == MM_WGRAD, BR, NW>;
    using ColOp = MtOperand<MODE != MM_FWD, BC, NW>;
    constexpr int STB = RowOp::BYTES + ColOp::BYTES;
    constexpr int MI = BR / WR / 16, NI = BC / WC / 16;
    constexpr int LPS = RowOp::ND + ColOp::ND;   // DMAs per wave and stage
    constexpr bool PIPE = BC == 256;   // fragments a step ahead (smaller tiles' workgroups cover each other's waits)
    __shared__ __attribute__((aligned(1024))) uint8_t lds[ST * STB];
    const uint32_t lds32 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);

    // this workgroup's tile: each of the 8 XCDs (workgroup id modulo 8) takes
    // a contiguous eighth of the tiles that exist
    int ntr = tr;
    if (MODE != MM_WGRAD && a.chunks) ntr = a.n_chunks[0];
    const int total = ntr * tc, per = (total + 7) >> 3, slot = (int)blockIdx.x >> 3;
    const int t = ((int)blockIdx.x & 7) * per + slot;
    if (slot >= per || t >= total) return;
    int rt, ct;
    mt_tile(t, ntr, tc, rt, ct);
    const int c0 = ct * BC;
    int r0 = 0, kdim;
    MmChunk ch;
    if constexpr (MODE == MM_WGRAD) {
        ch.group = blockIdx.y;
        mm_group_rows(a.offsets, ch.group, a.P, ch.row0, ch.n);
        r0 = rt * BR;
        kdim = ch.n;
    } else {
        if (!mm_chunk(a, rt, BR, ch)) return;
        kdim = MODE == MM_FWD ? a.K : a.N;
    }
    const bool glu = MODE == MM_FWD && a.act == MM_SWIGLU;
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const uint16_t* dz = static_cast<const uint16_t*>(a.dz);
    const uint16_t* wg = static_cast<const uint16_t*>(a.w) + (size_t)ch.group * a.N * a.ldw;

    // fixed parts of the DMAs' source addresses.  The chunk that a lane brings
    // is the same in all of a wave's DMAs (their rows differ by a multiple of
    // 16, or of 8 times an even number of waves), so operands contiguous along
    // the tile need one pointer, the others one per row
    static_assert(NW % 2 == 0 && (NW * RowOp::RPD) % 16 == 0 && (NW * ColOp::RPD) % 16 == 0, "one chunk per lane");
    const int rrow = RowOp::lds_row(0, w, lane), crow = ColOp::lds_row(0, w, lane);
    constexpr int RSTEP = NW * RowOp::RPD, CSTEP = NW * ColOp::RPD;   // rows from DMA to DMA
    const int rchunk = RowOp::chunk(rrow, lane), cchunk = ColOp::chunk(crow, lane);
    constexpr int NR = MODE == MM_WGRAD ? 1 : RowOp::ND, NC = MODE == MM_FWD ? ColOp::ND : 1;
    const uint16_t* rsrc[NR];
    const uint16_t* csrc[NC];
    if constexpr (MODE == MM_WGRAD) {
        rsrc[0] = dz + (size_t)ch.row0 * a.lddz + 8 * min(r0 / 8 + rchunk, (a.N - 1) / 8);
    } else {
#pragma unroll
        for (int i = 0; i < RowOp::ND; ++i) {
            const int r = ch.row0 + min(rrow + i * RSTEP, ch.n - 1);
            rsrc[i] = MODE == MM_FWD ? x + (size_t)mm_src(a, r) * a.ldx : dz + (size_t)r * a.lddz;
        }
    }
    if constexpr (MODE == MM_FWD) {
#pragma unroll
        for (int i = 0; i < ColOp::ND; ++i) {
            const int n = mm_col(a, glu, c0, crow + i * CSTEP);
            csrc[i] = wg + (size_t)(n < 0 ? a.N - 1 : n) * a.ldw;
        }
    } else {
        csrc[0] = (MODE == MM_DGRAD ? wg : x) + 8 * min(c0 / 8 + cchunk, (a.K - 1) / 8);
    }
    const int kchunk = (kdim - 1) / 8;
    // wgrad's x rows: a ring of 32 stages' row numbers in LDS, 16 stages filled
    // at a time (pair ids loaded a stage ahead into registers put their latency
    // into every stage's wait: 3.4 us a stage, 1.7 without them)
    __shared__ int src_rows[MODE == MM_WGRAD ? MT_RING : 1];
    auto fill_rows = [&](int st) {
        if (MODE == MM_WGRAD && a.sorted_pair) {
            for (int i = st * MT_K + tid; i < (st + MT_RING / MT_K / 2) * MT_K && i < kdim; i += NW * 64)
                src_rows[i % MT_RING] = mm_src(a, ch.row0 + i);
        }
    };
    // DMA i (0 .. LPS-1) of stage st
    auto issue1 = [&](int st, int i) {
        const uint32_t buf = lds32 + (uint32_t)(st % ST) * STB;
        const uint16_t* p;
        if (i < RowOp::ND) {
            if constexpr (MODE == MM_WGRAD)
                p = rsrc[0] + (size_t)min(st * MT_K + rrow + i * RSTEP, kdim - 1) * a.lddz;
            else
                p = rsrc[i] + 8 * min(st * (MT_K / 8) + rchunk, kchunk);
            mt_dma16(p, buf + (uint32_t)(i * NW + w) * 1024u);
        } else {
            const int c = i - RowOp::ND;
            if constexpr (MODE == MM_FWD) {
                p = csrc[c] + 8 * min(st * (MT_K / 8) + cchunk, kchunk);
            } else {
                const int k = min(st * MT_K + crow + c * CSTEP, kdim - 1);
                if constexpr (MODE == MM_DGRAD)
                    p = csrc[0] + (size_t)k * a.ldw;
                else
                    p = csrc[0] + (size_t)(a.sorted_pair ? src_rows[k % MT_RING] : ch.row0 + k) * a.ldx;
            }
            mt_dma16(p, buf + RowOp::BYTES + (uint32_t)(c * NW + w) * 1024u);
        }
    };
    auto issue = [&](int st) {
#pragma unroll
        for (int i = 0; i < LPS; ++i) issue1(st, i);
    };

    f32x4 acc[NI][MI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int wr0 = (w % WR) * (BR / WR), wc0 = (w / WR) * (BC / WC);
    // stages [sb, ns) of the contraction: all, or this split's share
    const int nall = (kdim + MT_K - 1) / MT_K;
    const int each = (nall + a.ksplits - 1) / a.ksplits;
    const int sb = min(nall, (int)blockIdx.z * each), ns = min(nall, sb + each);
    auto clear_tail = [&](int st) {   // behind the contraction's end, in the last stage
        if (st == nall - 1 && kdim % MT_K) {
            RowOp::clear_tail(lds + (st % ST) * STB, kdim % MT_K, tid);
            ColOp::clear_tail(lds + (st % ST) * STB + RowOp::BYTES, kdim % MT_K, tid);
            __syncthreads();
        }
    };
    // Matrix instructions on fragments rf, cf while the next ones are read
    // from step ks of stage st (and, with more, stage `more`'s DMAs issued),
    // spread over the row tiles.
    auto step = [&](const bf16x8 (&rf)[MI], const bf16x8 (&cf)[NI], bf16x8 (&rn)[MI], bf16x8 (&cn)[NI], int st, int ks,
                    int more) {
        const uint8_t* buf = lds + (st % ST) * STB;
#pragma unroll
        for (int j = 0; j < MI; ++j) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (i * MI / NI == j) cn[i] = ColOp::frag(buf + RowOp::BYTES, wc0, i, ks, lane);
            rn[j] = RowOp::frag(buf, wr0, j, ks, lane);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cf[i], rf[j], acc[i][j], 0, 0, 0);
            if (more >= 0) {
#pragma unroll
                for (int i = 0; i < LPS; ++i)
                    if (i * MI / LPS == j) issue1(more, i);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr int HALF = MT_RING / MT_K / 2;   // stages per filling of the ring
    if (MODE == MM_WGRAD && a.sorted_pair && sb < ns) {
        fill_rows(sb / HALF * HALF);
        fill_rows(sb / HALF * HALF + HALF);
        __syncthreads();
    }
    // in stage st, behind its barrier: the half of the ring behind stage st has
    // been read; what it then holds, stage st + 8 on, is needed first by the
    // DMAs that are issued up to ST stages ahead, so in 5 stages at the earliest
    auto refill = [&](int st) {
        if (MODE == MM_WGRAD && st % HALF == HALF / 2 && st / HALF > sb / HALF) fill_rows((st / HALF + 1) * HALF);
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
            bf16x8 rf[2][MI], cf[2][NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) cf[0][i] = ColOp::frag(lds + (sb % ST) * STB + RowOp::BYTES, wc0, i, 0, lane);
#pragma unroll
            for (int j = 0; j < MI; ++j) rf[0][j] = RowOp::frag(lds + (sb % ST) * STB, wr0, j, 0, lane);
            for (int st = sb; st < ns; ++st) {
                step(rf[0], cf[0], rf[1], cf[1], st, 1, -1);
                // stage st is read; stage st + 1 has to have landed
                if (ST > 2 && st + ST - 1 < ns)
                    mt_wait_vm<(ST - 2) * LPS>();
                else
                    mt_wait_vm<0>();
                mt_barrier();
                if (st + 1 < ns) clear_tail(st + 1);
                refill(st);
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
        for (int st = sb; st < ns; ++st) {
            if (ST > 2 && st + ST - 2 < ns)
                mt_wait_vm<(ST - 2) * LPS>();
            else
                mt_wait_vm<0>();
            mt_barrier();
            if (st + ST - 1 < ns) issue(st + ST - 1);
            refill(st);
            clear_tail(st);
            const uint8_t* buf = lds + (st % ST) * STB;
#pragma unroll
            for (int ks = 0; ks < MT_K / 32; ++ks) {
                bf16x8 rf[MI], cf[NI];
#pragma unroll
                for (int i = 0; i < NI; ++i) cf[i] = ColOp::frag(buf + RowOp::BYTES, wc0, i, ks, lane);
#pragma unroll
                for (int j = 0; j < MI; ++j) rf[j] = RowOp::frag(buf, wr0, j, ks, lane);
#pragma unroll
                for (int j = 0; j < MI; ++j)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cf[i], rf[j], acc[i][j], 0, 0, 0);
            }
        }
    }

    // Out through LDS, RP rows of the wave's tile at a time.  In the
    // accumulators a lane holds columns 4q .. 4q+3 of row m of each 16 x 16
    // block.
    constexpr int CW = BC / WC, WROWS = BR / WR;
    constexpr int FIT = ST * STB / NW / (CW * 4);   // rows of the wave's region
    constexpr int RP = FIT >= WROWS ? WROWS : (FIT >= WROWS / 2 ? WROWS / 2 : WROWS / 4);
    static_assert(RP >= 16 && RP % 16 == 0 && RP <= FIT && (CW & (CW - 1)) == 0 && CW >= 32, "passes of whole row tiles");
    const uint16_t* bias = nullptr;
    if (MODE == MM_FWD && a.bias) bias = static_cast<const uint16_t*>(a.bias) + (size_t)ch.group * a.N;
    const int rows = MODE == MM_WGRAD ? a.N - r0 : ch.n;
    const size_t row0 = MODE == MM_WGRAD ? (size_t)ch.group * a.N + r0 : (size_t)ch.row0;   // first output row
    float* part = a.ksplits > 1 ? a.kpart + (size_t)blockIdx.z * a.kpart_stride : nullptr;
    uint8_t* reg = lds + w * (RP * CW * 4);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < WROWS / RP; ++p) {
        const int m = lane & 15, q = lane >> 4;
#pragma unroll
        for (int j = 0; j < RP / 16; ++j)
#pragma unroll
            for (int i = 0; i < NI; ++i)
                *reinterpret_cast<f32x4*>(reg + (16 * j + m) * (CW * 4) + (((4 * i + q) ^ (m & (CW / 4 - 1))) << 4)) =
                    acc[i][p * (RP / 16) + j];
        const int rbase = wr0 + p * RP;
        if (MODE == MM_FWD && glu) {
            // 16 gate columns, then the 16 up columns they pair with
            constexpr int LR = CW / 16;   // lanes per row
            const int c8 = lane & (LR - 1), col = 32 * (c8 >> 1) + 8 * (c8 & 1);
            const int f = ((c0 + wc0) >> 1) + 8 * c8, cnt = (a.N >> 1) - f;
#pragma unroll 1
            for (int rr = lane / LR; rr < RP; rr += 64 / LR) {
                float g[8], u[8];
                mt_get8<CW>(reg, rr, col, g);
                mt_get8<CW>(reg, rr, col + 16, u);
                if (rbase + rr >= rows || cnt <= 0) continue;
                if (part) {
                    float* o = part + (row0 + rbase + rr) * a.ldp + f;
                    mt_st8(o, g, cnt, cnt >= 8);
                    mt_st8(o + (a.N >> 1), u, cnt, cnt >= 8 && (a.N & 7) == 0);
                } else {
                    mt_out8_glu(a, bias, ch.row0 + rbase + rr, f, cnt, g, u);
                }
            }
        } else {
            constexpr int LR = CW / 8;
            const int col = 8 * (lane & (LR - 1)), n = c0 + wc0 + col, cnt = (MODE == MM_FWD ? a.N : a.K) - n;
#pragma unroll 1
            for (int rr = lane / LR; rr < RP; rr += 64 / LR) {
                float v[8];
                mt_get8<CW>(reg, rr, col, v);
                if (rbase + rr >= rows || cnt <= 0) continue;
                const size_t r = row0 + rbase + rr;
                if (part)
                    mt_st8(part + r * a.ldp + n, v, cnt, cnt >= 8);
                else if constexpr (MODE == MM_FWD)
                    mt_out8(a, bias, (int)r, n, cnt, v);
                else if constexpr (MODE == MM_DGRAD)
                    mt_st8(static_cast<G*>(a.dx) + r * a.ldx + n, v, cnt, cnt >= 8);
                else
                    mt_st8(static_cast<G*>(a.dw) + r * a.ldw + n, v, cnt, cnt >= 8);
            }
        }
    }
}

// Joins the splits of a product, in split order, and finishes the rows as the
// tile kernel would: 8 rows of 256 columns per workgroup, rows 8 * blockIdx.z
// on of one chunk (forward, dgrad), or 8 * blockIdx.y on of dw.
template <int MODE, typename G>
__global__ __launch_bounds__(256) void mt_join_kernel(MmArgs a, int bm) {
    MmChunk ch;
    size_t r;
    if constexpr (MODE == MM_WGRAD) {
        ch.group = 0;
        r = (size_t)blockIdx.y * 8 + (threadIdx.x >> 5);
        if (r >= (size_t)a.E * a.N) return;
    } else {
        if (!mm_chunk(a, blockIdx.y, bm, ch)) return;
        const int rr = blockIdx.z * 8 + (threadIdx.x >> 5);
        if (rr >= ch.n) return;
        r = (size_t)(ch.row0 + rr);
    }
    const bool glu = MODE == MM_FWD && a.act == MM_SWIGLU;
    const int cols = MODE != MM_FWD ? a.K : (glu ? a.N >> 1 : a.N);
    const int n = blockIdx.x * 256 + 8 * (threadIdx.x & 31), cnt = cols - n;
    if (cnt <= 0) return;
    const uint16_t* bias = nullptr;
    if (MODE == MM_FWD && a.bias) bias = static_cast<const uint16_t*>(a.bias) + (size_t)ch.group * a.N;
    auto sum8 = [&](int c, bool vec, float (&v)[8]) {
        const float* p = a.kpart + r * a.ldp + c;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (vec) {
#pragma unroll 4
            for (int s = 0; s < a.ksplits; ++s) {
                const f32x4* x = reinterpret_cast<const f32x4*>(p + s * a.kpart_stride);
                const f32x4 lo = x[0], hi = x[1];
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
    float v[8];
    sum8(n, cnt >= 8, v);
    if (MODE == MM_FWD && glu) {
        float u[8];
        sum8((a.N >> 1) + n, cnt >= 8 && (a.N & 7) == 0, u);
        mt_out8_glu(a, bias, (int)r, n, cnt, v, u);
    } else if constexpr (MODE == MM_FWD) {
        mt_out8(a, bias, (int)r, n, cnt, v);
    } else if constexpr (MODE == MM_DGRAD) {
        mt_st8(static_cast<G*>(a.dx) + r * a.ldx + n, v, cnt, cnt >= 8);
    } else {
        mt_st8(static_cast<G*>(a.dw) + r * a.ldw + n, v, cnt, cnt >= 8);
    }
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Tile shapes, with the times that the estimate takes from measurement (us per
// stage of 64 contraction columns): lat of a workgroup by itself on its CU, thr
// per workgroup and CU when the chip is full; wgs that share a CU, so that one's
// start and end hide behind another's stages.  Of 66 products (24 .. 16384 rows,
// dense and of 8 .. 64 groups, 300 .. 8192 x 512 .. 8192, three modes), timed in
// every shape and split, the choice is within 15% of the best in 65; the other
// is 2048 rows of 8 groups, 1024 -> 1024, at 24.8 us against 19.0.
struct MtShape {
    int br, bc;
    double lat, thr;
    int wgs;
};
constexpr MtShape MT_SHAPES[] = {
    {256, 256, 1.1, 1.6, 1}, {128, 256, 0.68, 0.95, 1}, {128, 128, 0.55, 0.55, 2}, {64, 64, 0.25, 0.18, 3}};
constexpr int MT_NSHAPES = 4;
constexpr double MT_ENDS = 3.0;    // us to fill a workgroup's first stages and to write its tile
constexpr double MT_WENDS = 0.9;   // the same of wgrad's, without the writing
constexpr double MT_JOIN = 4.0;    // us of a join launch
constexpr double MT_MEM = 4.5e6;   // bytes per us, of outputs and partial sums
constexpr double MT_RAGGED = 1.25; // small tiles of groups read their weights more often

// Tile shape and contraction splits of the least estimated time: a CU's
// workgroups times their stages, plus what does not overlap.
MtPick mt_pick_(int mode, int P, int K, int N, int E) {
    const int live = E < P ? E : P;
    const int kdim = mode == MM_FWD ? K : (mode == MM_DGRAD ? N : (P + E - 1) / E);
    const int ns = cdiv(kdim, MT_K);
    MtPick best{0, 1};
    double least = 1e300;
    for (int i = 0; i < MT_NSHAPES; ++i) {
        const MtShape& t = MT_SHAPES[i];
        double tr;   // row tiles; of ragged groups about half a tile each is not filled
        if (mode == MM_WGRAD)
            tr = (double)cdiv(N, t.br) * E;
        else if (E == 1)
            tr = cdiv(P, t.br);
        else
            tr = (double)P / t.br + 0.5 * live > live ? (double)P / t.br + 0.5 * live : live;
        const double tiles = tr * cdiv(mode == MM_FWD ? N : K, t.bc);
        const double out = tiles * t.br * t.bc * 2.0 / MT_MEM;
        for (int s = 1; s <= MT_MAX_SPLITS && (s == 1 || (i >= 2 && ns / s >= 4 && tiles * s <= 512.0)); s *= 2) {
            const double wgs = tiles * s, per_cu = wgs <= 256.0 ? wgs / 256.0 : (double)(int64_t)(wgs / 256.0 + 0.999);
            const double thr = t.thr * (t.wgs > 1 && E > 1 && mode != MM_WGRAD ? MT_RAGGED : 1.0);
            const double stage = thr * per_cu > t.lat ? thr * per_cu : t.lat;
            double us = stage * cdiv(ns, s);
            if (mode == MM_WGRAD)   // (few stages: the writing does not hide)
                us += MT_WENDS * (per_cu < 1.0 ? 1.0 : per_cu) + out;
            else if (t.wgs == 1)
                us += MT_ENDS * (per_cu < 1.0 ? 1.0 : per_cu) + out;
            else
                us = (us > out ? us : out) + MT_ENDS;
            if (s > 1) us += MT_JOIN + (double)wgs * t.br * t.bc * 8.0 / MT_MEM;
            if (us < least) {
                least = us;
                best = MtPick{i, s};
            }
        }
    }
    return best;
}

template <int MODE, int BR, int BC, int WR, int WC, int ST, typename G>
hipError_t mt_launch(const MmArgs& a, hipStream_t s) {
    const int tr = MODE == MM_WGRAD ? cdiv(a.N, BR) : (a.chunks ? a.max_chunks : cdiv(a.P, BR));
    const int tc = cdiv(MODE == MM_FWD ? a.N : a.K, BC);
    const int64_t total = (int64_t)tr * tc;
    const dim3 g((uint32_t)((total + 7) / 8 * 8), MODE == MM_WGRAD ? (uint32_t)a.E : 1u, (uint32_t)a.ksplits);
    mt_kernel<MODE, BR, BC, WR, WC, ST, G><<<g, 64 * WR * WC, 0, s>>>(a, tr, tc);
    if (a.ksplits > 1) {
        const int cols = MODE != MM_FWD ? a.K : (a.act == MM_SWIGLU ? a.N / 2 : a.N);
        const dim3 j((uint32_t)cdiv(cols, 256),
                     (uint32_t)(MODE == MM_WGRAD ? cdiv((int64_t)a.E * a.N, 8) : tr), MODE == MM_WGRAD ? 1u : BR / 8u);
        mt_join_kernel<MODE, G><<<j, 256, 0, s>>>(a, BR);
    }
    return hipGetLastError();
}

template <int MODE, typename G>
hipError_t mt_run(const MmArgs& a, int shape, hipStream_t s) {
    constexpr int DEEP = 3;
    switch (shape) {
        case 0: return mt_launch<MODE, 256, 256, 2, 4, 2, G>(a, s);
        case 1: return mt_launch<MODE, 128, 256, 2, 4, DEEP, G>(a, s);
        case 2: return mt_launch<MODE, 128, 128, 2, 2, 2, G>(a, s);
        default: return mt_launch<MODE, 64, 64, 2, 2, DEEP, G>(a, s);
    }
}

}  // namespace

MtPick mt_pick(int mode, int P, int K, int N, int E) { return mt_pick_(mode, P, K, N, E); }
int mt_chunk_rows(int mode, int P, int K, int N, int E) { return MT_SHAPES[mt_pick(mode, P, K, N, E).shape].br; }

size_t mt_split_bytes(int mode, int P, int K, int N, int E, bool exact) {
    // the bound: at most 512 tiles of up to 128 x 128 in all splits together,
    // and at most MT_MAX_SPLITS splits
    const int64_t kdim = mode == MM_FWD ? K : (mode == MM_DGRAD ? N : P);
    if (cdiv(kdim, MT_K) < 8) return 0;
    const int64_t rows = mode == MM_WGRAD ? (int64_t)E * N : P, cols = mode == MM_FWD ? N : K;
    const int64_t one = rows * ((cols + 7) / 8 * 8);
    if (exact) {
        const int splits = mt_pick(mode, P, K, N, E).splits;
        return splits > 1 ? (size_t)splits * one * 4 : 0;
    }
    const int64_t all = MT_MAX_SPLITS * one;
    const int64_t cap = (int64_t)512 * 128 * 128;
    return (size_t)(all < cap ? all : cap) * 4;
}

hipError_t launch_mt(const MmArgs& a0, int mode, hipStream_t s) {
    MmArgs a = a0;
    const MtPick pick = mt_pick(mode, a.P, a.K, a.N, a.E);
    a.ksplits = pick.splits;
    a.ldp = ((mode == MM_FWD ? a.N : a.K) + 7) / 8 * 8;
    a.kpart_stride = (size_t)(mode == MM_WGRAD ? (int64_t)a.E * a.N : (int64_t)a.P) * a.ldp;
    if (mode == MM_FWD) return mt_run<MM_FWD, uint16_t>(a, pick.shape, s);
    if (mode == MM_DGRAD) return mt_run<MM_DGRAD, uint16_t>(a, pick.shape, s);
    if (a.grad_f32) return mt_run<MM_WGRAD, float>(a, pick.shape, s);
    return mt_run<MM_WGRAD, uint16_t>(a, pick.shape, s);
}

}  // namespace ds4
