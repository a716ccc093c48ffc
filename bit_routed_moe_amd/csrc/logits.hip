// Rules on logits before sampling: penalties for tokens said before, biases,
// and a grammar's mask.  For token v of row b, with c and n the numbers of its
// occurrences in the row's history and in the generated part of it:
//   l = c > 0 ? (l > 0 ? l / repetition : l * repetition) : l
//   l = l - frequency * n - presence * (n > 0)
//   l = l + bias of v
//   l = -infinity unless v's bit is set in the row's mask
//
// Bound by memory: each logit is read and written once.  A workgroup takes one
// segment of a row.  It requests its logits first (those in 16-byte pieces that
// the mask leaves something of), then reads the row's whole history and biases
// and notes those of its segment in LDS (a count per token, the generated ones
// added and the prompt's in the top bit; the place of its last bias): integer
// atomics, whose order changes nothing.
#include "common.hpp"
#include "launch.hpp"

namespace ds4 {

namespace {

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

// NT threads, C pieces of 16 bytes of logits each; TABLE: there is a history
// or a bias.
template <typename TI, typename TO, int NT, int C, bool TABLE>
__global__ __launch_bounds__(NT) void lg_kernel(LogitArgs a) {
    constexpr int N = LgVec<TI>::N, S = NT * C * N;
    __shared__ __attribute__((aligned(16))) uint32_t count[TABLE ? S : 4], place[TABLE ? S : 4];
    const int tid = threadIdx.x, b = blockIdx.y, v0 = blockIdx.x * S;
    const TI* const in = static_cast<const TI*>(a.logits) + (size_t)b * a.ld;
    TO* const out = static_cast<TO*>(a.out) + (size_t)b * a.ld_out;

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

    int b0 = 0;
    if constexpr (TABLE) {
        for (int i = tid; i < S / 4; i += NT) {
            reinterpret_cast<u32x4*>(count)[i] = u32x4{0, 0, 0, 0};
            reinterpret_cast<u32x4*>(place)[i] = u32x4{0, 0, 0, 0};
        }
        __syncthreads();
        if (a.history) {
            int h0, n;
            lg_range(a.history_offsets, b, a.n_history, h0, n);
            const int made = a.prompt_len ? a.prompt_len[b] : 0;
#pragma unroll 4
            for (int i = tid; i < n; i += NT) {
                const uint32_t d = (uint32_t)a.history[(size_t)h0 + i] - (uint32_t)v0;
                if (d < (uint32_t)S) {
                    if (i >= made)
                        atomicAdd(&count[d], 1u);
                    else
                        atomicOr(&count[d], LG_PROMPT);
                }
            }
        }
        if (a.bias_token) {
            int n;
            lg_range(a.bias_offsets, b, a.n_bias, b0, n);
            for (int i = tid; i < n; i += NT) {
                const uint32_t d = (uint32_t)a.bias_token[(size_t)b0 + i] - (uint32_t)v0;
                if (d < (uint32_t)S) atomicMax(&place[d], (uint32_t)i + 1);
            }
        }
        __syncthreads();
    }
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
            if constexpr (TABLE) {
                if (bits[i]) {
                    uint32_t any = 0;
#pragma unroll
                    for (int h = 0; h < N / 4; ++h) {
                        const u32x4 c = reinterpret_cast<const u32x4*>(count + d)[h];
                        const u32x4 p = reinterpret_cast<const u32x4*>(place + d)[h];
                        any = c[0] | c[1] | c[2] | c[3] | p[0] | p[1] | p[2] | p[3];
                        if (any) {
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
                if constexpr (TABLE) l = rule(l, count[d + e], place[d + e]);
                lg_store1(out + v + e, (bits[i] >> e) & 1 ? l : -INFINITY);
            }
        }
    }
}

template <typename TI, typename TO, int NT, int C>
hipError_t lg_launch(const LogitArgs& a, hipStream_t s) {
    constexpr int S = NT * C * LgVec<TI>::N;
    const dim3 g((uint32_t)((a.V + S - 1) / S), (uint32_t)a.B);
    if (a.history || a.bias_token)
        lg_kernel<TI, TO, NT, C, true><<<g, NT, 0, s>>>(a);
    else
        lg_kernel<TI, TO, NT, C, false><<<g, NT, 0, s>>>(a);
    return hipGetLastError();
}

template <typename TI, typename TO>
hipError_t lg_run(const LogitArgs& a, hipStream_t s) {
    constexpr int C = 16 / LgVec<TI>::N;   // pieces that make 16 tokens
    if ((int64_t)a.B * a.V < (int64_t)1024 * 4096) return lg_launch<TI, TO, 256, 1>(a, s);
    return lg_launch<TI, TO, 256, C>(a, s);
}

}  // namespace

hipError_t launch_adjust_logits(const LogitArgs& a, bool f32_in, bool f32_out, hipStream_t s) {
    if (f32_in) return f32_out ? lg_run<float, float>(a, s) : lg_run<float, uint16_t>(a, s);
    return f32_out ? lg_run<uint16_t, float>(a, s) : lg_run<uint16_t, uint16_t>(a, s);
}

}  // namespace ds4
