// Rows between the tokens' order and the experts' order, with the router's
// weights applied, and the gradients of both directions.  With pos =
// pair_pos[t * k + j] the sorted row of token t's slot j (none outside
// [0, rows)) and w its weight (1 without weights):
//   to rows    out[pos]  = w src[t]                        (dispatch; collect's gradient)
//   to tokens  out[t]    = base[t] + sum_j w src[pos]      (collect; dispatch's gradient)
//   weights    dw[t][j]  = sum_h src[pos][h] v[t][h]       (v: the token's row)
// Both directions go token by token, so that a token's row is read or written
// once and only the k sorted rows move k times, and the weights' gradients are
// sums over a row that its wave or workgroup has in hand.  They are bound by
// memory: 4096 tokens top-8 of 7168 bf16 by expert (529 MB) 92 us, 5.7 TB/s;
// 2048 tokens' collected rows, gradients of rows and weights (500 MB) 100 us,
// 5.0 TB/s; 4096 tokens collected (587 MB) 116 us, 5.1 TB/s.  Sorted row by row
// in place of token by token, a token's row would be read k times.
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace ds4 {

namespace {

template <typename T>
struct TkVec;
template <>
struct TkVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(u32x4 r, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
    }
    static __device__ __forceinline__ u32x4 put(const float (&v)[4]) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[i]);
        return r;
    }
};
template <>
struct TkVec<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(u32x4 r, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ u32x4 put(const float (&v)[8]) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        return r;
    }
};

// 16-byte chunk c of a row; the elements behind column H, which may hold
// anything, read as zero.
template <typename T>
__device__ __forceinline__ u32x4 tk_load(const T* row, int c, int H) {
    constexpr int N = TkVec<T>::N, W = sizeof(T) / 2;   // (halves of 16 bits per element)
    u32x4 r = *reinterpret_cast<const u32x4*>(row + (size_t)c * N);
    const int n = H - c * N;
    if (n < N) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int h = 2 * i;                        // first half of word i
            r[i] = h + 1 < n * W ? r[i] : (h < n * W ? r[i] & 0xFFFFu : 0u);
        }
    }
    return r;
}

template <bool NT = false, typename T>
__device__ __forceinline__ void tk_store(T* row, int c, int H, u32x4 r) {
    constexpr int N = TkVec<T>::N;
    const int n = H - c * N;
    if (n >= N) {
        u32x4* p = reinterpret_cast<u32x4*>(row + (size_t)c * N);
        if constexpr (NT)
            __builtin_nontemporal_store(r, p);
        else
            *p = r;
    } else {
        const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) row[(size_t)c * N + i] = e[i];
    }
}

// One wave per pair, the waves of a workgroup share a token; blockIdx.y: a
// share of the columns (chunks [y * span, ..), none with DOTS).  Workgroups
// from T on clear the rows that no pair names, 64 of them per wave.
template <typename T, bool DOTS, bool NT>
__global__ __launch_bounds__(512) void tk_rows_kernel(TokenArgs a, int span) {
    using V = TkVec<T>;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
    const int chunks = (a.H + V::N - 1) / V::N;
    const int c0 = blockIdx.y * span, c1 = min(chunks, c0 + span);
    T* const out = static_cast<T*>(a.out);
    if ((int)blockIdx.x >= a.T) {
        const int64_t r0 = ((int64_t)((int)blockIdx.x - a.T) * nw + w) * 64;
        const int64_t r = r0 + lane;
        const bool none = r < a.rows && (uint32_t)a.sorted_pair[r] >= (uint32_t)a.T * (uint32_t)a.k;
        uint64_t left = __ballot(none);
        while (left) {
            const int i = __builtin_ctzll(left);
            left &= left - 1;
            T* row = out + (r0 + i) * a.ldr;
            for (int c = c0 + lane; c < c1; c += 64) tk_store<NT>(row, c, a.H, u32x4{0, 0, 0, 0});
        }
        return;
    }
    const int t = blockIdx.x;
    const T* const src = static_cast<const T*>(a.src) + (size_t)t * a.ldx;
    for (int j = w; j < a.k; j += nw) {
        const size_t p = (size_t)t * a.k + j;
        const int pos = __builtin_amdgcn_readfirstlane(a.pair_pos[p]);
        const bool there = (uint32_t)pos < (uint32_t)a.rows;
        float dot = 0.0f;
        if (there) {
            const float wt = a.topk_w ? a.topk_w[p] : 1.0f;
            T* const row = out + (size_t)pos * a.ldr;
            const T* const theirs = static_cast<const T*>(a.theirs) + (DOTS ? (size_t)pos * a.ldr : 0);
            constexpr int U = 4;
            for (int c = c0 + lane; c < c1; c += 64 * U) {
                u32x4 x[U], o[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    x[u] = u32x4{0, 0, 0, 0};
                    if (c + 64 * u < c1) x[u] = tk_load(src, c + 64 * u, a.H);
                    if constexpr (DOTS) {
                        o[u] = u32x4{0, 0, 0, 0};
                        if (c + 64 * u < c1) o[u] = tk_load(theirs, c + 64 * u, a.H);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float v[V::N];
                    V::get(x[u], v);
                    if constexpr (DOTS) {
                        float q[V::N];
                        V::get(o[u], q);
#pragma unroll
                        for (int i = 0; i < V::N; ++i) dot += v[i] * q[i];
                    }
                    if (a.topk_w) {
#pragma unroll
                        for (int i = 0; i < V::N; ++i) v[i] *= wt;
                        x[u] = V::put(v);
                    }
                    if (out && c + 64 * u < c1) tk_store<NT>(row, c + 64 * u, a.H, x[u]);
                }
            }
        }
        if constexpr (DOTS) {
            dot = wave_sum(dot);
            if (lane == 0) a.dw[p] = there ? dot : 0.0f;
        }
    }
}

// Sums of M values (a power of 2, at most 64) over the wave, together: each
// step halves the values that a lane holds, so 8 sums take 10 exchanges, not
// 48.  Value i's sum ends in the lanes whose low bits spell i.
template <int M>
__device__ __forceinline__ float tk_sums(float (&v)[M], int lane) {
    int o = 1;
#pragma unroll
    for (int n = M / 2; n >= 1; n >>= 1, o <<= 1) {
        const bool up = lane & o;
        // keep the odd values where the lane's bit is set, else the even ones
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? v[2 * i + 1] : v[2 * i], give = up ? v[2 * i] : v[2 * i + 1];
            v[i] = keep + __shfl_xor(give, o, WAVE);
        }
    }
#pragma unroll
    for (; o < 64; o <<= 1) v[0] += __shfl_xor(v[0], o, WAVE);
    return v[0];
}

// One workgroup per token (and share of the columns, as above), a chunk of
// columns per thread and turn; the k rows are read 8, 4, 2 or 1 at a time.
template <typename T, bool DOTS>
__global__ __launch_bounds__(512) void tk_tokens_kernel(TokenArgs a, int span) {
    using V = TkVec<T>;
    __shared__ int pos[64];
    __shared__ float wt[64], dots[8][64];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63, w = tid >> 6, t = blockIdx.x;
    const int chunks = (a.H + V::N - 1) / V::N;
    const int c0 = blockIdx.y * span, c1 = min(chunks, c0 + span);
    for (int j = tid; j < a.k; j += nt) {
        const size_t p = (size_t)t * a.k + j;
        const int at = a.pair_pos[p];
        const bool there = (uint32_t)at < (uint32_t)a.rows;
        pos[j] = there ? at : -1;
        wt[j] = !there ? 0.0f : (a.topk_w ? a.topk_w[p] : 1.0f);
    }
    if constexpr (DOTS)
        for (int i = tid; i < 8 * 64; i += nt) (&dots[0][0])[i] = 0.0f;
    __syncthreads();
    const T* const src = static_cast<const T*>(a.src);
    const T* const base = a.base ? static_cast<const T*>(a.base) + (size_t)t * a.ldx : nullptr;
    const T* const tok = DOTS ? static_cast<const T*>(a.theirs) + (size_t)t * a.ldx : nullptr;
    T* const out = a.out ? static_cast<T*>(a.out) + (size_t)t * a.ldx : nullptr;
    // (all threads of a wave take part in the sums of DOTS)
    for (int first = c0; first < c1; first += nt) {
        const int c = first + tid;
        const bool mine = c < c1;
        float acc[V::N], x[V::N];
#pragma unroll
        for (int i = 0; i < V::N; ++i) acc[i] = x[i] = 0.0f;
        if (base && mine) V::get(tk_load(base, c, a.H), acc);
        if constexpr (DOTS)
            if (mine) V::get(tk_load(tok, c, a.H), x);
        auto block = [&](int j, auto count) {
            constexpr int JB = decltype(count)::value;
            u32x4 r[JB];
            if (mine) {
#pragma unroll
                for (int i = 0; i < JB; ++i) r[i] = tk_load(src + (size_t)max(pos[j + i], 0) * a.ldr, c, a.H);
            }
            float dot[JB];
#pragma unroll
            for (int i = 0; i < JB; ++i) {
                const bool there = mine && pos[j + i] >= 0;
                const float wj = wt[j + i];
                if (!there) r[i] = u32x4{0, 0, 0, 0};
                float v[V::N];
                V::get(r[i], v);
                dot[i] = 0.0f;
#pragma unroll
                for (int e = 0; e < V::N; ++e) {
                    acc[e] += wj * v[e];
                    if constexpr (DOTS) dot[i] += x[e] * v[e];
                }
            }
            if constexpr (DOTS) {
                const float sum = tk_sums<JB>(dot, lane);
                if (lane < JB) dots[w][j + lane] += sum;
            }
        };
        int j = 0;
        for (; j + 8 <= a.k; j += 8) block(j, std::integral_constant<int, 8>{});
        if (j + 4 <= a.k) {
            block(j, std::integral_constant<int, 4>{});
            j += 4;
        }
        if (j + 2 <= a.k) {
            block(j, std::integral_constant<int, 2>{});
            j += 2;
        }
        if (j < a.k) block(j, std::integral_constant<int, 1>{});
        if (out && mine) tk_store(out, c, a.H, V::put(acc));
    }
    if constexpr (DOTS) {
        __syncthreads();
        for (int j = tid; j < a.k; j += nt) {
            float s = 0.0f;
            for (int i = 0; i < (nt >> 6); ++i) s += dots[i][j];
            a.dw[(size_t)t * a.k + j] = pos[j] >= 0 ? s : 0.0f;
        }
    }
}

// dlogits[t] = w_j (dw_j - sum_i w_i dw_i) at the chosen experts, 0 elsewhere
// (the weights are the softmax of the chosen logits).  A wave per token; the
// row is put together in LDS, so that it leaves in whole pieces.
__global__ __launch_bounds__(256) void tk_route_backward_kernel(int T, int E, int k, const int32_t* __restrict__ idx,
                                                                const float* __restrict__ w,
                                                                const float* __restrict__ dw,
                                                                float* __restrict__ dlogits) {
    __shared__ float rows[4][1024];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int t = blockIdx.x * 4 + wv;
    float* const row = rows[wv];
    if (t < T) {
        const size_t p = (size_t)t * k + lane;
        const float wj = lane < k ? w[p] : 0.0f, dj = lane < k ? dw[p] : 0.0f;
        const int e = lane < k ? idx[p] : -1;
        const float s = wave_sum(lane < k ? wj * dj : 0.0f);
        for (int i = lane; i < E; i += 64) row[i] = 0.0f;
        __builtin_amdgcn_wave_barrier();
        if ((uint32_t)e < (uint32_t)E) row[e] = wj * (dj - s);
    }
    __syncthreads();
    if (t >= T) return;
    float* const out = dlogits + (size_t)t * E;
    for (int i = lane; i < E; i += 64) out[i] = row[i];
}

int tk_chunks(const TokenArgs& a, bool f32) { return f32 ? (a.H + 3) / 4 : (a.H + 7) / 8; }

// Chunks of a row per workgroup: all of them, or a share of whole waves where
// tokens alone leave CUs without a workgroup (sums over a row need all of it).
int tk_span(const TokenArgs& a, int chunks) {
    if (a.dw || a.T >= 256) return chunks;
    const int waves = (chunks + 63) / 64, want = 256 / a.T;
    const int parts = want < waves ? want : waves;
    return (waves + parts - 1) / parts * 64;
}

}  // namespace

hipError_t launch_tokens_to_rows(const TokenArgs& a, bool f32, hipStream_t s) {
    const int chunks = tk_chunks(a, f32);
    const int nw = a.k < 8 ? a.k : 8;
    const uint32_t clear = a.sorted_pair && a.out ? (uint32_t)(((int64_t)a.rows + 64 * nw - 1) / (64 * nw)) : 0u;
    const int span = tk_span(a, chunks);
    const dim3 g((uint32_t)a.T + clear, (uint32_t)((chunks + span - 1) / span));
    // Rows that do not fit the 256 MB of the memory-side cache pass it by, others
    // stay there for their reader: 4096 tokens top-8 of 7168 bf16 (470 MB) 92
    // against 121 us, but 2048 (235 MB) 48 against 41, 1024 24 against 22.5.
    const int64_t moved = (int64_t)a.rows * a.H * (f32 ? 4 : 2) * ((a.out ? 1 : 0) + (a.dw ? 1 : 0));
    const uint32_t threads = 64 * nw;
    auto run = [&](auto nt) {
        constexpr bool NT = decltype(nt)::value;
        if (f32) {
            if (a.dw)
                tk_rows_kernel<float, true, NT><<<g, threads, 0, s>>>(a, span);
            else
                tk_rows_kernel<float, false, NT><<<g, threads, 0, s>>>(a, span);
        } else {
            if (a.dw)
                tk_rows_kernel<uint16_t, true, NT><<<g, threads, 0, s>>>(a, span);
            else
                tk_rows_kernel<uint16_t, false, NT><<<g, threads, 0, s>>>(a, span);
        }
    };
    if (moved > ((int64_t)1 << 28))
        run(std::true_type{});
    else
        run(std::false_type{});
    return hipGetLastError();
}

hipError_t launch_rows_to_tokens(const TokenArgs& a, bool f32, hipStream_t s) {
    const int chunks = tk_chunks(a, f32);
    const int span = tk_span(a, chunks);
    // as many waves as leave the last turn full: 14 waves of columns go in 2 turns of 7
    const int waves = (span + 63) / 64, turns = (waves + 7) / 8;
    const uint32_t nt = 64 * ((waves + turns - 1) / turns);
    const dim3 g((uint32_t)a.T, (uint32_t)((chunks + span - 1) / span));
    if (f32) {
        if (a.dw)
            tk_tokens_kernel<float, true><<<g, nt, 0, s>>>(a, span);
        else
            tk_tokens_kernel<float, false><<<g, nt, 0, s>>>(a, span);
    } else {
        if (a.dw)
            tk_tokens_kernel<uint16_t, true><<<g, nt, 0, s>>>(a, span);
        else
            tk_tokens_kernel<uint16_t, false><<<g, nt, 0, s>>>(a, span);
    }
    return hipGetLastError();
}

hipError_t launch_route_backward(int T, int E, int k, const int32_t* idx, const float* w, const float* dw,
                                 float* dlogits, hipStream_t s) {
    tk_route_backward_kernel<<<(uint32_t)((T + 3) / 4), 256, 0, s>>>(T, E, k, idx, w, dw, dlogits);
    return hipGetLastError();
}

}  // namespace ds4
