// Rules on logits before sampling: penalties for tokens said before, biases,
// and a grammar's mask.  For token v of row b, with c and n the numbers of its
// occurrences in the row's history and in the generated part of it:
//   l = c > 0 ? (l > 0 ? l / repetition : l * repetition) : l
//   l = l - frequency * n - presence * (n > 0)
//   l = l + bias of v
//   l = -infinity unless v's bit is set in the row's mask
//
// Bound by memory: each logit is read and written once.  A workgroup takes one
// segment of a row.  It requests the row's lists and its logits (those in
// 16-byte pieces that the mask leaves something of) before it waits for any,
// then notes the history's and the biases' tokens of its segment in LDS (a count
// per token, the generated ones added and the prompt's in the top bit; the place
// of its last bias): integer atomics, whose order changes nothing.  64 rows of 131072 fp32 under all rules
// (histories of 2000 tokens, half of the rows masked; 68 MB) 14.6 us, 4.6 TB/s;
// 256 rows of 50003 bf16 to fp32 with counts (77 MB) 16.9 us, 4.6 TB/s; one row
// of 131072 5.6 us, the latency of its lists and of LDS.  With the lists
// requested behind the logits, both tables always and 4096-token segments of
// 256 threads: 23.7, 19.4 and 8.4 us.
#include "common.hpp"
#include "launch.hpp"

namespace ds4 {

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
// 16 bytes of a row that starts anywhere.
typedef u32x4 lg_f32x4 __attribute__((aligned(4)));
typedef u32x4 lg_bf16x8 __attribute__((aligned(2)));

template <typename T>
struct LgVec;
template <>
struct LgVec<float> {
    static constexpr int N = 4;
    typedef lg_f32x4 Piece;
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ void get(u32x4 r, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
    }
};
template <>
struct LgVec<uint16_t> {
    static constexpr int N = 8;
    typedef lg_bf16x8 Piece;
    static __device__ __forceinline__ float get(uint16_t v) { return bf16_to_f32(v); }
    static __device__ __forceinline__ void get(u32x4 r, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
};

template <int N>
__device__ __forceinline__ void lg_store(float* p, const float (&v)[N]) {
#pragma unroll
    for (int h = 0; h < N / 4; ++h) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[4 * h + i]);
        reinterpret_cast<lg_f32x4*>(p)[h] = r;
    }
}
template <int N>
__device__ __forceinline__ void lg_store(uint16_t* p, const float (&v)[N]) {
    if constexpr (N == 8) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<lg_bf16x8*>(p) = r;
    } else {
        typedef u32x2 half __attribute__((aligned(2)));
        *reinterpret_cast<half*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}
__device__ __forceinline__ void lg_store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void lg_store1(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16(v); }

// Entries [first, first + n) of row b in a list of `total`; none where the
// offsets are not ascending within it.
__device__ __forceinline__ void lg_range(const int32_t* offsets, int b, int total, int& first, int& n) {
    first = offsets[b];
    const int end = offsets[b + 1];
    n = first >= 0 && end <= total && end >= first ? end - first : 0;
}

constexpr uint32_t LG_PROMPT = 0x80000000u;

// NT threads, C pieces of 16 bytes of logits each; HIST, BIAS: rows have a
// history, a list of biases (LDS for one table only lets twice the workgroups
// share a CU).
template <typename TI, typename TO, int NT, int C, bool HIST, bool BIAS>
__global__ __launch_bounds__(NT) void lg_kernel(LogitArgs a) {
    constexpr int N = LgVec<TI>::N, S = NT * C * N;
    __shared__ __attribute__((aligned(16))) uint32_t count[HIST ? S : 4], place[BIAS ? S : 4];
    const int tid = threadIdx.x, b = blockIdx.y, v0 = blockIdx.x * S;
    const TI* const in = static_cast<const TI*>(a.logits) + (size_t)b * a.ld;
    TO* const out = static_cast<TO*>(a.out) + (size_t)b * a.ld_out;

    // where the row's lists lie, and the first of its history
    int h0 = 0, nh = 0, made = 0, b0 = 0, nb = 0;
    typedef i32x4 tokens4 __attribute__((aligned(4)));
    i32x4 said[2];
    if constexpr (BIAS) lg_range(a.bias_offsets, b, a.n_bias, b0, nb);
    if constexpr (HIST) {
        lg_range(a.history_offsets, b, a.n_history, h0, nh);
        made = a.prompt_len ? a.prompt_len[b] : 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = 4 * (j * NT + tid);
            if (i + 4 <= nh) said[j] = *reinterpret_cast<const tokens4*>(a.history + (size_t)h0 + i);
        }
    }
    // the mask's bits of this thread's pieces (all set without a mask)
    uint32_t bits[C];
    const uint32_t* words = nullptr;
    if (a.mask) {
        const int g = a.mask_row ? a.mask_row[b] : b;
        if (g >= 0 && g < a.mask_rows) words = a.mask + (size_t)g * a.mask_ld;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int v = v0 + (i * NT + tid) * N;
        bits[i] = (1u << N) - 1;
        if (words && v < a.V) bits[i] &= words[v >> 5] >> (v & 31);
    }
    u32x4 piece[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int v = v0 + (i * NT + tid) * N;
        if (bits[i] && v + N <= a.V) piece[i] = *reinterpret_cast<const typename LgVec<TI>::Piece*>(in + v);
    }

    if constexpr (HIST || BIAS) {
        for (int i = tid; i < S / 4; i += NT) {
            if constexpr (HIST) reinterpret_cast<u32x4*>(count)[i] = u32x4{0, 0, 0, 0};
            if constexpr (BIAS) reinterpret_cast<u32x4*>(place)[i] = u32x4{0, 0, 0, 0};
        }
        __syncthreads();
    }
    if constexpr (HIST) {
        auto note = [&](int i, int token) {   // token i of the history
            const uint32_t d = (uint32_t)token - (uint32_t)v0;
            if (d < (uint32_t)S) {
                if (i >= made)
                    atomicAdd(&count[d], 1u);
                else
                    atomicOr(&count[d], LG_PROMPT);
            }
        };
        auto note4 = [&](int i, i32x4 t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) note(i + e, t[e]);
        };
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = 4 * (j * NT + tid);
            if (i + 4 <= nh) note4(i, said[j]);
        }
#pragma unroll 2
        for (uint32_t i = 4 * (2 * NT + tid); i + 4 <= (uint32_t)nh; i += 4 * NT)   // (beyond 31 bits at most by a step)
            note4((int)i, *reinterpret_cast<const tokens4*>(a.history + (size_t)h0 + i));
        if (tid < (nh & 3)) note((nh & ~3) + tid, a.history[(size_t)h0 + (nh & ~3) + tid]);
    }
    if constexpr (BIAS) {
        for (uint32_t i = tid; i < (uint32_t)nb; i += NT) {
            const uint32_t d = (uint32_t)a.bias_token[(size_t)b0 + i] - (uint32_t)v0;
            if (d < (uint32_t)S) atomicMax(&place[d], i + 1);
        }
    }
    if constexpr (HIST || BIAS) __syncthreads();
    const float rep = a.repetition ? a.repetition[b] : 1.0f;
    const float pres = a.presence ? a.presence[b] : 0.0f, freq = a.frequency ? a.frequency[b] : 0.0f;
    // token d of the segment
    auto rule = [&](float l, uint32_t c, uint32_t at) {
        if (c) {
            if (a.repetition) l = l > 0.0f ? l / rep : l * rep;
            const uint32_t n = c & ~LG_PROMPT;
            if (n) l = l - freq * (float)n - pres;
        }
        if (at) l += a.bias_value[(size_t)b0 + at - 1];
        return l;
    };
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int d = (i * NT + tid) * N, v = v0 + d;
        if (v >= a.V) break;
        if (v + N <= a.V) {
            float l[N];
            if (bits[i]) LgVec<TI>::get(piece[i], l);
            if constexpr (HIST || BIAS) {
                if (bits[i]) {
#pragma unroll
                    for (int h = 0; h < N / 4; ++h) {
                        u32x4 c = {0, 0, 0, 0}, p = {0, 0, 0, 0};
                        if constexpr (HIST) c = reinterpret_cast<const u32x4*>(count + d)[h];
                        if constexpr (BIAS) p = reinterpret_cast<const u32x4*>(place + d)[h];
                        if (c[0] | c[1] | c[2] | c[3] | p[0] | p[1] | p[2] | p[3]) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) l[4 * h + e] = rule(l[4 * h + e], c[e], p[e]);
                        }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < N; ++e) l[e] = (bits[i] >> e) & 1 ? l[e] : -INFINITY;
            lg_store<N>(out + v, l);
        } else {   // the row's end
            for (int e = 0; v + e < a.V; ++e) {
                float l = LgVec<TI>::get(in[v + e]);
                if constexpr (HIST || BIAS) l = rule(l, HIST ? count[d + e] : 0u, BIAS ? place[d + e] : 0u);
                lg_store1(out + v + e, (bits[i] >> e) & 1 ? l : -INFINITY);
            }
        }
    }
}

template <typename TI, typename TO, int NT, int C>
hipError_t lg_launch(const LogitArgs& a, hipStream_t s) {
    constexpr int S = NT * C * LgVec<TI>::N;
    const dim3 g((uint32_t)((a.V + S - 1) / S), (uint32_t)a.B);
    if (a.history && a.bias_token)
        lg_kernel<TI, TO, NT, C, true, true><<<g, NT, 0, s>>>(a);
    else if (a.history)
        lg_kernel<TI, TO, NT, C, true, false><<<g, NT, 0, s>>>(a);
    else if (a.bias_token)
        lg_kernel<TI, TO, NT, C, false, true><<<g, NT, 0, s>>>(a);
    else
        lg_kernel<TI, TO, NT, C, false, false><<<g, NT, 0, s>>>(a);
    return hipGetLastError();
}

// Segments of 8192 tokens (1024 threads) once there are rows and tokens enough
// for about two of their workgroups per CU; else short ones, that the row's
// history is read by more workgroups matters less than idle CUs.  us with 1024
// threads of 8 tokens / 512 of 8 / 256 of 16 / 1024 of 16: 64 rows of 131072,
// history and biases of 2000 and 30 each 16.0 / 16.2 / 19.3 / 16.7, histories
// of 32000 25.8 / 31.7 / - / 25.3; 256 rows of 50003, histories of 700 19.0 /
// 19.3 / - / 20.4, with biases 21.6 / 22.0 / - / 29.1.
template <typename TI, typename TO>
hipError_t lg_run(const LogitArgs& a, hipStream_t s) {
    if (a.V <= 4096 || (int64_t)a.B * a.V < (int64_t)512 * 8192) return lg_launch<TI, TO, 256, 1>(a, s);
    return lg_launch<TI, TO, 1024, 8 / LgVec<TI>::N>(a, s);
}

}  // namespace

hipError_t launch_adjust_logits(const LogitArgs& a, bool f32_in, bool f32_out, hipStream_t s) {
    if (f32_in) return f32_out ? lg_run<float, float>(a, s) : lg_run<float, uint16_t>(a, s);
    return f32_out ? lg_run<uint16_t, float>(a, s) : lg_run<uint16_t, uint16_t>(a, s);
}

}  // namespace ds4
