// Token sampling: temperature, top-k, top-p, min-p and one given random number
// per row.
//
// The tokens of a row in (logit descending, index ascending) order have
// weights w_i = exp((l_i - max) / T).  Each filter keeps a prefix of that
// order, so the kept set is the shortest of three prefixes, its mass the least
// of three masses, and the sampled token is the one at which the running sum
// first exceeds u times that mass.  The vocabulary is never sorted: each
// question is "where does a running count or sum cross a value", answered by a
// histogram over (max - l) / T (64 bins per unit or more) and then among the tokens of
// the few bins that the crossings can lie in, which are collected and sorted.
//
// Weights are held as integers, round(w * 2^43) in 64 bits, from 64-bit
// arithmetic: integer sums do not depend on the order of additions, so the
// histogram's atomics and every sum below are reproducible, and a border moves
// by at most 2^-43 of the largest weight per token.  Tokens below e^-31 of the
// largest are never chosen.
//
// Four launches for rows of a long vocabulary, S workgroups per row in the
// first three: the row's maximum; the histogram (LDS, then integer atomics
// into the row's); the collection; the answer, one workgroup per row.  Where
// more tokens than fit lie in the bins of a crossing (nearly flat rows, or
// many equal logits) the last launch narrows each crossing down by itself,
// pass by pass over the row: 64 rows of 131072 with top-p take 79 us where flat
// rows fill fine bins, 381 us where a mask of -1e4 keeps the bins wide (42 us
// and 346 us at one row), 1.1 ms where all logits are equal.
//
// 64 rows of 131072 are bound by waiting: vector units are busy for 53%, 40%,
// 22% and 4% of the four launches, LDS for 12%, 21%, 9% and 3%; each workgroup
// has its scans, searches and barriers once, however few tokens it reads.  256
// rows of 50003 in bf16: 49%, 57%, 45% and 25%, LDS 8%, 37% (most of it
// conflicts of the histogram's atomics), 10% and 22%.
#include "common.hpp"
#include "launch.hpp"

namespace ds4 {

namespace {

constexpr int SP_BINS = 2048;                // bin b: b <= per (max - l) / T < b + 1
constexpr double SP_REACH = 31.0;            // (max - l) / T from which a token has no weight
constexpr int SP_CAP = 2048;                 // tokens sorted at once
constexpr double SP_ONE = 8796093022208.0;   // 2^43
constexpr uint64_t SP_ONE_I = (uint64_t)1 << 43;
constexpr int SP_THREADS = 512;              // of the launches that split a row
constexpr int SP_FOUND = 1024;               // tokens one of their workgroups may collect
constexpr int SP_LAST = 512;                 // of the answering launch
constexpr int SP_KEYS = SP_CAP / SP_LAST;

struct SpArgs {
    const void* logits;
    int64_t ld;
    int V, S;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t* top_k;
    int32_t* token;
    float* prob;
    // workspace, per row
    uint64_t* best;    // [SP_MAX_SPLITS] largest route_key of each split
    uint32_t* low;     // [SP_MAX_SPLITS] lowest logit (order-preserving bits)
    uint64_t* mass;    // [SP_BINS]
    uint32_t* cnt;     // [SP_BINS]
    uint64_t* list;    // [SP_CAP] collected keys
    uint32_t* n;       // [64] (first: tokens collected)
};

// Weight of a token t = per (max - l) / T bins below the largest, in bin b:
// e^(-(b + 1/2)/per) (table or exp) times the series of e^x for the rest
// x = (b + 1/2 - t)/per, |x| <= 1/128; the first omitted term is below 2^-51.
// The rounding to an integer is that of adding 2^52.
__device__ __forceinline__ double sp_bin_exp(int b, double unit) { return SP_ONE * exp(-((double)b + 0.5) * unit); }
__device__ __forceinline__ uint64_t sp_weight(double t, double ebin, double unit) {
    const double x = (0.5 - __builtin_amdgcn_fract(t)) * unit;
    double s = fma(x, 1.0 / 120.0, 1.0 / 24.0);
    s = fma(x, s, 1.0 / 6.0);
    s = fma(x, s, 0.5);
    s = fma(x, s, 1.0);
    s = fma(x, s, 1.0);
    return (uint64_t)(__double_as_longlong(fma(ebin, s, 4503599627370496.0)) & 0xFFFFFFFFFFFFFll);
}

__device__ __forceinline__ uint32_t sp_k32(float l) { return (uint32_t)(route_key(l, 0) >> 32); }
__device__ __forceinline__ int sp_key_index(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

// Up to four ranges of bins.
struct SpBins {
    int lo[4], hi[4];
    __device__ __forceinline__ bool has(int b) const {
        return (b >= lo[0] && b <= hi[0]) || (b >= lo[1] && b <= hi[1]) || (b >= lo[2] && b <= hi[2]) ||
               (b >= lo[3] && b <= hi[3]);
    }
};

// A row's logits and what its weights are relative to.
template <typename T>
struct SpRow {
    const T* row;
    int V;
    float mx;
    double per;     // bins per unit of (max - l) / T, a power of two
    double unit;    // 1 / per
    double scale;   // per / T
    double limit;   // bins of tokens with weight

    // per (max - l) / T; 0 for the largest logits themselves, also infinite ones
    __device__ __forceinline__ double dist(float l) const {
        return l == mx ? 0.0 : ((double)mx - (double)l) * scale;
    }
    // Bin of a distance, SP_BINS for tokens of no weight
    __device__ __forceinline__ int bin(double t) const { return t < limit ? (int)t : SP_BINS; }
    __device__ __forceinline__ uint64_t weight(float l) const {
        const double t = dist(l);
        const int b = bin(t);
        return b < SP_BINS ? sp_weight(t, sp_bin_exp(b, unit), unit) : 0;
    }

    // Logits outside [least, most] lie in none of the bins (the bounds are a
    // bin and a part in 2^20 wide of them, far beyond the roundings of bin()).
    __device__ __forceinline__ void logits_of(const SpBins& s, float& least, float& most) const {
        int lo = SP_BINS, hi = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (s.hi[i] < s.lo[i]) continue;
            lo = min(lo, s.lo[i]);
            hi = max(hi, s.hi[i]);
        }
        least = (float)((double)mx - (double)(hi + 2) / scale);
        most = (float)((double)mx - (double)(lo - 1) / scale);
        least -= fabsf(least) * 0x1p-20f;
        most += fabsf(most) * 0x1p-20f;
        if (!(least > -INFINITY) || !(fabsf(mx) < INFINITY)) least = -INFINITY;   // (infinite or NaN: no bound)
        if (!(most < INFINITY) || !(fabsf(mx) < INFINITY)) most = INFINITY;
    }

    // f(logit, index) for the tokens of split s of n that are above -infinity
    // and not NaN, a thread's own in ascending order; NT threads.
    template <int NT, typename F>
    __device__ __forceinline__ void each(int s, int n, const F& f) const {
        constexpr int N = 16 / sizeof(T);
        constexpr int UN = 8 / N;      // 8 tokens per lane and step, the next step's loads in flight (16: 7% slower,
                                       // 32: 20%; each launch fetches its code afresh)
        const uintptr_t p = reinterpret_cast<uintptr_t>(row);
        const int skip = (int)(p & 15) / (int)sizeof(T);    // elements of the first 16 bytes before the row
        const u32x4* base = reinterpret_cast<const u32x4*>(p & ~(uintptr_t)15);
        const int nch = (skip + V + N - 1) / N;
        const int per = (nch + n - 1) / n;
        const int cb = min(nch, s * per), ce = min(nch, cb + per);
        if (cb >= ce) return;
        u32x4 nx[UN];
#pragma unroll
        for (int j = 0; j < UN; ++j) nx[j] = base[min(cb + (int)threadIdx.x + j * NT, ce - 1)];
#pragma unroll 1
        for (int c0 = cb + threadIdx.x; c0 < ce; c0 += NT * UN) {
            u32x4 v[UN];
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                v[j] = nx[j];
                nx[j] = base[min(c0 + (UN + j) * NT, ce - 1)];
            }
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                const int c = c0 + j * NT, i0 = c * N - skip;
                if (c >= ce || i0 < 0 || i0 + N > V) {   // what is not the row's becomes -infinity
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (c < ce && i0 + i >= 0 && i0 + i < V) continue;
                        if constexpr (sizeof(T) == 4)
                            v[j][i] = 0xFF800000u;
                        else
                            v[j][i >> 1] = (i & 1) ? (v[j][i >> 1] & 0xFFFFu) | 0xFF800000u
                                                   : (v[j][i >> 1] & 0xFFFF0000u) | 0xFF80u;
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float l;
                    if constexpr (sizeof(T) == 4)
                        l = __uint_as_float(v[j][i]);
                    else
                        l = __uint_as_float((i & 1) ? v[j][i >> 1] & 0xFFFF0000u : v[j][i >> 1] << 16);
                    if (l > -INFINITY) f(l, i0 + i);
                }
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ SpRow<T> sp_row(const SpArgs& a, int r) {
    SpRow<T> row;
    row.row = static_cast<const T*>(a.logits) + (size_t)r * a.ld;
    row.V = a.V;
    row.mx = 0.0f;
    row.per = row.unit = row.scale = row.limit = 1.0;
    return row;
}

// The row's reference from its largest key and its lowest logit above
// -infinity (as order-preserving bits); false when nothing is left to choose
// or the choice is greedy.  64 bins per unit reach all weights; a row of narrow
// range takes finer bins, 2, 4, ... times as many per unit while all of it
// still fits, so that few tokens share one.
template <typename T>
__device__ __forceinline__ bool sp_reference(const SpArgs& a, int r, uint64_t best, uint32_t low, SpRow<T>& row) {
    const float temp = a.temperature ? a.temperature[r] : 1.0f;
    if (best == 0 || !(temp > 0.0f)) return false;
    row.mx = key_value(best);
    const double inv_t = 1.0 / (double)temp;
    const double range = ((double)row.mx - (double)key_value((uint64_t)low << 32)) * inv_t;
    row.per = 64.0;
    if (range < SP_REACH)
        while (row.per < 16384.0 && range * row.per * 2.0 < SP_BINS - 1) row.per *= 2.0;
    row.unit = 1.0 / row.per;
    row.scale = row.per * inv_t;
    row.limit = SP_REACH * row.per < SP_BINS ? SP_REACH * row.per : (double)SP_BINS;
    return true;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const uint64_t k = __shfl_xor(v, o, WAVE);
        v = v > k ? v : k;
    }
    return v;
}

__device__ __forceinline__ uint32_t wave_min_u32(uint32_t v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = min(v, (uint32_t)__shfl_xor((int)v, o, WAVE));
    return v;
}

// The row's largest key and lowest logit from its splits' (at most 64: one per
// lane).
constexpr int SP_MAX_SPLITS = 64;
__device__ __forceinline__ uint64_t sp_row_best(const SpArgs& a, int r, uint32_t& low) {
    const int lane = threadIdx.x & 63;
    const bool has = lane < a.S;
    const size_t at = (size_t)r * SP_MAX_SPLITS + lane;
    low = wave_min_u32(has ? a.low[at] : 0xFFFFFFFFu);
    return wave_max_u64(has ? a.best[at] : 0);
}

// The same of split sp of n (every thread receives them); tmp, tmpl: NT / 64
// words.
template <int NT, typename T>
__device__ __forceinline__ uint64_t sp_largest(const SpRow<T>& row, int sp, int n, uint64_t* tmp, uint32_t* tmpl,
                                               uint32_t& low) {
    float lo = INFINITY, hi = -INFINITY;
    int at = 0;
    row.template each<NT>(sp, n, [&](float l, int idx) {   // (a thread's indices ascend: ties keep the lowest)
        at = l > hi ? idx : at;
        hi = fmaxf(hi, l);
        lo = fminf(lo, l);
    });
    uint64_t best = wave_max_u64(hi > -INFINITY ? route_key(hi, at) : 0);
    low = wave_min_u32(sp_k32(lo));
    if ((threadIdx.x & 63) == 0) {
        tmp[threadIdx.x >> 6] = best;
        tmpl[threadIdx.x >> 6] = low;
    }
    __syncthreads();
    for (int i = 0; i < NT / WAVE; ++i) {
        best = best > tmp[i] ? best : tmp[i];
        low = min(low, tmpl[i]);
    }
    __syncthreads();
    return best;
}

// Adds a token to a histogram in LDS.  Lanes that all meet in one bin (equal
// logits) add up first: same-address LDS atomics take one lane after the other.
__device__ __forceinline__ void sp_count(uint32_t* cnt, uint64_t* mass, int bin, uint64_t w) {
    const int first = __builtin_amdgcn_readfirstlane(bin);
    if (__builtin_expect(__ballot(bin != first) == 0 && __popcll(__ballot(1)) == WAVE, 0)) {
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) w += __shfl_xor(w, o, WAVE);
        if ((threadIdx.x & 63) == 0) {
            atomicAdd(cnt + bin, (uint32_t)WAVE);
            atomicAdd(reinterpret_cast<unsigned long long*>(mass + bin), (unsigned long long)w);
        }
    } else {
        atomicAdd(cnt + bin, 1u);
        atomicAdd(reinterpret_cast<unsigned long long*>(mass + bin), (unsigned long long)w);
    }
}

// Inclusive running counts and sums over the block, NT threads with P
// consecutive entries each.
template <int NT, int P>
__device__ __forceinline__ void sp_scan(uint32_t (&c)[P], uint64_t (&m)[P], uint32_t* redc, uint64_t* red) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
    for (int i = 1; i < P; ++i) {
        c[i] += c[i - 1];
        m[i] += m[i - 1];
    }
    uint32_t ct = c[P - 1];
    uint64_t mt = m[P - 1];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t cu = __shfl_up(ct, o, WAVE);
        const uint64_t mu = __shfl_up(mt, o, WAVE);
        if (lane >= o) {
            ct += cu;
            mt += mu;
        }
    }
    if (lane == 63) {
        redc[wv] = ct;
        red[wv] = mt;
    }
    __syncthreads();
    ct -= c[P - 1];
    mt -= m[P - 1];
    for (int i = 0; i < wv; ++i) {
        ct += redc[i];
        mt += red[i];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        c[i] += ct;
        m[i] += mt;
    }
    __syncthreads();
}

// A histogram (in global memory or LDS) -> its running counts and sums in LDS.
template <int NT>
__device__ __forceinline__ void sp_running(const uint32_t* cnt, const uint64_t* mass, uint32_t* C, uint64_t* M,
                                           uint32_t* redc, uint64_t* red) {
    constexpr int P = SP_BINS / NT;
    uint32_t c[P];
    uint64_t m[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        c[i] = cnt[P * threadIdx.x + i];
        m[i] = mass[P * threadIdx.x + i];
    }
    sp_scan<NT, P>(c, m, redc, red);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        C[P * threadIdx.x + i] = c[i];
        M[P * threadIdx.x + i] = m[i];
    }
    __syncthreads();
}

// First entry of an ascending array of SP_BINS that reaches t (which the last
// one does).
template <typename U>
__device__ __forceinline__ int sp_find(const U* v, uint64_t t) {
    int b = -1;
#pragma unroll
    for (int o = SP_BINS / 2; o >= 1; o >>= 1)
        if (v[b + o] < t) b += o;
    return b + 1;
}

__device__ __forceinline__ uint64_t sp_top_p(float p, uint64_t mass) {
    const double want = ceil((double)p * (double)mass);
    const uint64_t t = want < 1.0 ? 1 : (uint64_t)want;
    return t < mass ? t : mass;
}
__device__ __forceinline__ uint64_t sp_target(float u, uint64_t mass) {
    const double at = u > 0.0f ? floor((double)u * (double)mass) : 0.0;
    const uint64_t t = at < (double)mass ? (uint64_t)at + 1 : mass;
    return t < mass ? t : mass;
}
// Smallest weight that min-p keeps, and the bins it can lie in (q <= 1).
__device__ __forceinline__ uint64_t sp_min_weight(float q) { return (uint64_t)ceil((double)q * SP_ONE); }
__device__ __forceinline__ void sp_min_bins(float q, double per, int& lo, int& hi) {
    const int b = (int)fmin(-log((double)q) * per, (double)(SP_BINS - 1));
    lo = max(b - 1, 0);
    hi = min(b + 1, SP_BINS - 1);
}

struct SpFilters {
    int k;       // 0: off
    float p, q, u;
};
__device__ __forceinline__ SpFilters sp_filters(const SpArgs& a, int r, uint32_t tokens) {
    SpFilters f;
    const int k = a.top_k ? a.top_k[r] : 0;
    f.k = k > 0 && (uint32_t)k < tokens ? k : 0;    // (tokens past the bins weigh nothing)
    const float p = a.top_p ? a.top_p[r] : 1.0f;
    f.p = p < 1.0f ? p : 1.0f;
    const float q = a.min_p ? a.min_p[r] : 0.0f;
    f.q = q > 0.0f ? q : 0.0f;
    f.u = a.u[r];
    return f;
}

// The bins in which the crossings can lie, from the running counts C and sums
// M alone: every mass below is known to lie between two values, and the bins
// between their crossings are taken.  The kept mass is never below the first
// token's.
__device__ __forceinline__ SpBins sp_bins(const SpFilters& f, double per, const uint32_t* C, const uint64_t* M) {
    SpBins s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s.lo[i] = 0;
        s.hi[i] = -1;
    }
    uint64_t least = M[SP_BINS - 1], most = least;
    if (f.k) {
        const int b = sp_find(C, (uint64_t)f.k);
        s.lo[0] = s.hi[0] = b;
        if (C[b] <= SP_CAP) {   // the first k tokens hold every answer: take all of them
            s.lo[0] = 0;
            return s;
        }
        least = b ? M[b - 1] : 0;
        most = M[b];
    }
    least = least > SP_ONE_I ? least : SP_ONE_I;
    if (f.p < 1.0f) {
        s.lo[1] = sp_find(M, sp_top_p(f.p, least));
        s.hi[1] = sp_find(M, sp_top_p(f.p, most));
        least = s.lo[1] ? M[s.lo[1] - 1] : 0;
        least = least > SP_ONE_I ? least : SP_ONE_I;
        most = most < M[s.hi[1]] ? most : M[s.hi[1]];
    }
    if (f.q > 1.0f) {
        least = most = SP_ONE_I;
    } else if (f.q > 0.0f) {
        sp_min_bins(f.q, per, s.lo[2], s.hi[2]);
        uint64_t m = s.lo[2] ? M[s.lo[2] - 1] : 0;
        m = m > SP_ONE_I ? m : SP_ONE_I;
        least = least < m ? least : m;
        most = most < M[s.hi[2]] ? most : M[s.hi[2]];
    }
    s.lo[3] = sp_find(M, sp_target(f.u, least));
    s.hi[3] = sp_find(M, sp_target(f.u, most));
    return s;
}

// A split's tokens into a histogram in LDS (counts for top-k only).
template <int NT, typename T>
__device__ __forceinline__ void sp_histogram(const SpArgs& a, int r, const SpRow<T>& row, int sp, int n, uint32_t* cnt,
                                             uint64_t* mass, const double* table) {
    const bool counts = a.top_k && a.top_k[r] > 0;
    row.template each<NT>(sp, n, [&](float l, int) {
        const double d = row.dist(l);
        const int b = row.bin(d);
        if (b < SP_BINS) {
            if (counts) atomicAdd(cnt + b, 1u);
            atomicAdd(reinterpret_cast<unsigned long long*>(mass + b), (unsigned long long)sp_weight(d, table[b], row.unit));
        }
    });
    __syncthreads();
}

// ---- launches that split a row -----------------------------------------------

template <typename T>
__global__ __launch_bounds__(SP_THREADS) void sp_max_kernel(SpArgs a) {
    __shared__ uint64_t tmp[SP_THREADS / WAVE];
    __shared__ uint32_t tmpl[SP_THREADS / WAVE];
    const int sp = blockIdx.x, r = blockIdx.y;
    const SpRow<T> row = sp_row<T>(a, r);
    uint32_t low;
    const uint64_t best = sp_largest<SP_THREADS>(row, sp, a.S, tmp, tmpl, low);
    if (threadIdx.x == 0) {
        a.best[(size_t)r * SP_MAX_SPLITS + sp] = best;
        a.low[(size_t)r * SP_MAX_SPLITS + sp] = low;
    }
    // the row's histogram and list start empty
    for (int i = sp * SP_THREADS + threadIdx.x; i < SP_BINS; i += a.S * SP_THREADS) {
        a.cnt[(size_t)r * SP_BINS + i] = 0;
        a.mass[(size_t)r * SP_BINS + i] = 0;
    }
    if (sp == 0 && threadIdx.x == 0) a.n[(size_t)r * 64] = 0;
}

template <typename T>
__global__ __launch_bounds__(SP_THREADS) void sp_hist_kernel(SpArgs a) {
    __shared__ uint32_t cnt[SP_BINS];
    __shared__ uint64_t mass[SP_BINS];
    __shared__ double table[SP_BINS];
    const int sp = blockIdx.x, r = blockIdx.y;
    SpRow<T> row = sp_row<T>(a, r);
    uint32_t low;
    const uint64_t best = sp_row_best(a, r, low);
    if (!sp_reference(a, r, best, low, row)) return;
    for (int i = threadIdx.x; i < SP_BINS; i += SP_THREADS) {
        cnt[i] = 0;
        mass[i] = 0;
        table[i] = sp_bin_exp(i, row.unit);
    }
    __syncthreads();
    sp_histogram<SP_THREADS>(a, r, row, sp, a.S, cnt, mass, table);
    for (int i = threadIdx.x; i < SP_BINS; i += SP_THREADS) {
        if (cnt[i]) atomicAdd(a.cnt + (size_t)r * SP_BINS + i, cnt[i]);
        if (mass[i])
            atomicAdd(reinterpret_cast<unsigned long long*>(a.mass + (size_t)r * SP_BINS + i),
                      (unsigned long long)mass[i]);
    }
}

template <typename T>
__global__ __launch_bounds__(SP_THREADS) void sp_collect_kernel(SpArgs a) {
    __shared__ uint32_t C[SP_BINS];
    __shared__ uint64_t M[SP_BINS];
    __shared__ uint64_t found[SP_FOUND];
    __shared__ uint32_t redc[SP_THREADS / WAVE];
    __shared__ uint64_t red[SP_THREADS / WAVE];
    __shared__ uint32_t n, at;
    const int sp = blockIdx.x, r = blockIdx.y;
    SpRow<T> row = sp_row<T>(a, r);
    uint32_t low;
    const uint64_t best = sp_row_best(a, r, low);
    if (!sp_reference(a, r, best, low, row)) return;
    if (threadIdx.x == 0) n = 0;
    sp_running<SP_THREADS>(a.cnt + (size_t)r * SP_BINS, a.mass + (size_t)r * SP_BINS, C, M, redc, red);
    const SpBins bins = sp_bins(sp_filters(a, r, C[SP_BINS - 1]), row.per, C, M);
    float lmin, lmax;
    row.logits_of(bins, lmin, lmax);
    row.template each<SP_THREADS>(sp, a.S, [&](float l, int idx) {
        if (!(l >= lmin && l <= lmax)) return;   // (most tokens end here)
        const int b = row.bin(row.dist(l));
        if (b < SP_BINS && bins.has(b)) {
            const uint32_t i = atomicAdd(&n, 1u);
            if (i < SP_FOUND) found[i] = route_key(l, idx);
        }
    });
    __syncthreads();
    // (a count past SP_CAP says that they do not fit)
    if (threadIdx.x == 0) at = n ? atomicAdd(a.n + (size_t)r * 64, n <= SP_FOUND ? n : SP_CAP + 1) : 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < n && i < SP_FOUND && at + i < SP_CAP; i += SP_THREADS)
        a.list[(size_t)r * SP_CAP + at + i] = found[i];
}

// ---- the answer ----------------------------------------------------------------

struct SpShared {
    uint32_t C[SP_BINS];         // running counts and sums of the histogram
    uint64_t M[SP_BINS];
    uint32_t scnt[SP_BINS];      // histogram of a piece of one bin
    uint64_t smass[SP_BINS];     // (and the sorted tokens' weights)
    uint64_t key[SP_CAP];        // collected tokens, sorted: keys,
    uint32_t rank[SP_CAP];       // running counts and sums up to and with each
    uint64_t sum[SP_CAP];
    uint64_t red[SP_LAST / WAVE];
    uint32_t redc[SP_LAST / WAVE];
    uint32_t n;
    int at;
};

// Sorts more than SP_LAST collected keys descending: a bitonic network over
// SP_KEYS keys per thread in registers (key h of a thread is element
// tid + h * SP_LAST), exchanged by lane shuffles (distances below 64), LDS
// (below SP_LAST) or within the thread.
__device__ __forceinline__ void sp_sort_network(SpShared& s) {
    const int tid = threadIdx.x, n = (int)s.n;
    int size = 64;
    while (size < n) size <<= 1;
    uint64_t v[SP_KEYS];
#pragma unroll
    for (int h = 0; h < SP_KEYS; ++h) v[h] = tid + h * SP_LAST < n ? s.key[tid + h * SP_LAST] : 0;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1) {
#pragma unroll
        for (int hx = SP_KEYS / 2; hx >= 1; hx >>= 1) {
            if ((k >> 1) < hx * SP_LAST) continue;
#pragma unroll
            for (int h = 0; h < SP_KEYS; ++h) {
                if (h & hx) continue;
                const bool down = ((tid + h * SP_LAST) & k) == 0;
                const uint64_t x = v[h], y = v[h | hx];
                if (down ? x < y : x > y) {
                    v[h] = y;
                    v[h | hx] = x;
                }
            }
        }
        for (int j = min(k >> 1, SP_LAST / 2); j >= WAVE; j >>= 1) {
#pragma unroll
            for (int h = 0; h < SP_KEYS; ++h)
                if (tid + h * SP_LAST < size) s.key[tid + h * SP_LAST] = v[h];
            __syncthreads();
#pragma unroll
            for (int h = 0; h < SP_KEYS; ++h) {
                const int i = tid + h * SP_LAST;
                if ((i & ~63) >= size) continue;   // (whole waves past the end)
                const uint64_t o = s.key[i ^ j];
                const bool want_max = ((i & k) == 0) == ((i & j) == 0);
                v[h] = want_max ? (v[h] > o ? v[h] : o) : (v[h] < o ? v[h] : o);
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = WAVE / 2; j >= 1; j >>= 1) {
            if (j >= k) continue;
#pragma unroll
            for (int h = 0; h < SP_KEYS; ++h) {
                const int i = tid + h * SP_LAST;
                if ((i & ~63) >= size) continue;
                const uint64_t o = (uint64_t)__shfl_xor(v[h], j, WAVE);
                const bool want_max = ((i & k) == 0) == ((i & j) == 0);
                v[h] = want_max ? (v[h] > o ? v[h] : o) : (v[h] < o ? v[h] : o);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < SP_KEYS; ++h) s.key[tid + h * SP_LAST] = v[h];
    __syncthreads();
}

// Sorts the s.n collected keys descending.  Up to one per thread: a key's
// place is the number of greater ones, counted by as many threads per key as
// there are (109 keys 14,200 cycles with the network, whose 28 steps are one
// LDS round trip each).
__device__ __forceinline__ void sp_sort(SpShared& s) {
    const int tid = threadIdx.x, n = (int)s.n;
    if (n > SP_LAST) {
        sp_sort_network(s);
        return;
    }
    const int nr = max(WAVE, (n + WAVE - 1) & ~(WAVE - 1));   // (whole waves share a part of the comparisons)
    const int parts = SP_LAST / nr, part = tid / nr, i = tid - part * nr;
    if (tid < n) s.rank[tid] = 0;
    __syncthreads();
    uint64_t k = 0;
    if (part < parts && i < n) {
        k = s.key[i];
        const int each = (n + parts - 1) / parts, jb = part * each, je = min(n, jb + each);
        uint32_t greater = 0;
#pragma unroll 8
        for (int j = jb; j < je; ++j) greater += s.key[j] > k;
        if (greater) atomicAdd(&s.rank[i], greater);
    }
    __syncthreads();
    if (part == 0 && i < n) s.key[s.rank[i]] = k;
    __syncthreads();
}

// Weights (into smass), running counts and sums of the sorted tokens, which
// continue c0 and m0.
// gaps: between tokens of different bins stand the bins that were not
// collected, whose counts and masses C and M have.
template <typename T>
__device__ __forceinline__ void sp_sums(SpShared& s, const SpRow<T>& row, bool gaps, uint32_t c0, uint64_t m0) {
    const int n = (int)s.n;
    for (int i = threadIdx.x; i < n; i += SP_LAST) s.smass[i] = row.weight(key_value(s.key[i]));
    __syncthreads();
    uint32_t c[SP_KEYS];
    uint64_t m[SP_KEYS];
#pragma unroll
    for (int h = 0; h < SP_KEYS; ++h) {
        const int i = SP_KEYS * threadIdx.x + h;
        c[h] = 0;
        m[h] = 0;
        if (i >= n) continue;
        c[h] = 1;
        m[h] = s.smass[i];
        if (gaps) {
            const int b = row.bin(row.dist(key_value(s.key[i])));
            const int pb = i ? row.bin(row.dist(key_value(s.key[i - 1]))) : -1;
            if (b != pb && b) {
                c[h] += s.C[b - 1] - (pb >= 0 ? s.C[pb] : 0);
                m[h] += s.M[b - 1] - (pb >= 0 ? s.M[pb] : 0);
            }
        }
    }
    sp_scan<SP_LAST, SP_KEYS>(c, m, s.redc, s.red);
#pragma unroll
    for (int h = 0; h < SP_KEYS; ++h) {
        const int i = SP_KEYS * threadIdx.x + h;
        s.rank[i] = c0 + c[h];
        s.sum[i] = m0 + m[h];
    }
    __syncthreads();
}

// Position of the sorted token at which the running count (by_rank) or sum
// reaches t.
__device__ __forceinline__ int sp_cross(const SpShared& s, bool by_rank, uint64_t t) {
    int lo = 0, hi = (int)s.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((by_rank ? (uint64_t)s.rank[mid] : s.sum[mid]) < t)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// A crossing: the running sum up to and with the token, its weight and index.
struct SpHit {
    uint64_t mass, w;
    int index;
};
__device__ __forceinline__ SpHit sp_hit(const SpShared& s, bool by_rank, uint64_t t) {
    const int i = sp_cross(s, by_rank, t);
    SpHit h;
    h.mass = s.sum[i];
    h.w = s.smass[i];
    h.index = sp_key_index(s.key[i]);
    return h;
}

// Collects the tokens for which in(bin, k32) holds (at most SP_CAP exist).
template <typename T, typename F>
__device__ __forceinline__ void sp_gather(SpShared& s, const SpRow<T>& row, const F& in) {
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    row.template each<SP_LAST>(0, 1, [&](float l, int idx) {
        const int b = row.bin(row.dist(l));
        if (b < SP_BINS && in(b, sp_k32(l))) {
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < SP_CAP) s.key[at] = route_key(l, idx);
        }
    });
    __syncthreads();
}

// The crossing at running count or sum t, in a bin with more tokens than can
// be sorted at once: the range [lo, hi] of order-preserving logit bits is
// narrowed by histograms of up to 2048 pieces.
template <typename T>
__device__ SpHit sp_narrow(SpShared& s, const SpRow<T>& row, bool by_rank, uint64_t t) {
    const int b = by_rank ? sp_find(s.C, t) : sp_find(s.M, t);
    uint32_t c0 = b ? s.C[b - 1] : 0;
    uint64_t m0 = b ? s.M[b - 1] : 0;
    uint32_t n = SP_CAP + 1;   // (rows without top-k are not counted)
    uint32_t lo = 0, hi = 0xFFFFFFFFu;
    while (n > SP_CAP && lo < hi) {   // (each round divides the range by 2048)
        int shift = 0;
        while (((hi - lo) >> shift) >= SP_BINS) ++shift;
        for (int i = threadIdx.x; i < SP_BINS; i += SP_LAST) {
            s.scnt[i] = 0;
            s.smass[i] = 0;
        }
        __syncthreads();
        row.template each<SP_LAST>(0, 1, [&](float l, int) {
            const uint32_t k = sp_k32(l);
            if (k >= lo && k <= hi && row.bin(row.dist(l)) == b)
                sp_count(s.scnt, s.smass, (int)((hi - k) >> shift), row.weight(l));
        });
        __syncthreads();
        sp_running<SP_LAST>(s.scnt, s.smass, s.scnt, s.smass, s.redc, s.red);
        const int p = by_rank ? sp_find(s.scnt, t - c0) : sp_find(s.smass, t - m0);
        const uint32_t before = p ? s.scnt[p - 1] : 0;
        n = s.scnt[p] - before;
        c0 += before;
        m0 += p ? s.smass[p - 1] : 0;
        const uint32_t top = hi - ((uint32_t)p << shift);
        const uint32_t width = ((uint32_t)1 << shift) - 1;
        lo = top - lo > width ? top - width : lo;
        hi = top;
        __syncthreads();
    }
    if (n <= SP_CAP) {
        sp_gather(s, row, [&](int bb, uint32_t k) { return bb == b && k >= lo && k <= hi; });
        sp_sort(s);
        sp_sums(s, row, false, c0, m0);
        return sp_hit(s, by_rank, t);
    }
    // equal logits: the j-th of them in index order
    SpHit h;
    h.w = row.weight(key_value((uint64_t)hi << 32));
    const uint64_t j = by_rank ? t - c0 : (t - m0 + h.w - 1) / h.w;
    h.mass = m0 + j * h.w;
    h.index = -1;
    uint64_t seen = 0;
    for (int i0 = 0; i0 < row.V && h.index < 0; i0 += SP_LAST) {
        const int i = i0 + threadIdx.x;
        bool eq = false;
        if (i < row.V) {
            float l;
            if constexpr (sizeof(T) == 4)
                l = row.row[i];
            else
                l = bf16_to_f32(row.row[i]);
            eq = l > -INFINITY && sp_k32(l) == hi;
        }
        const uint64_t vote = __ballot(eq);
        if ((threadIdx.x & 63) == 0) s.redc[threadIdx.x >> 6] = (uint32_t)__popcll(vote);
        if (threadIdx.x == 0) s.at = -1;
        __syncthreads();
        uint64_t at = seen;
        for (int k = 0; k < (int)(threadIdx.x >> 6); ++k) at += s.redc[k];
        at += __popcll(vote & (((uint64_t)1 << (threadIdx.x & 63)) - 1));
        if (eq && at + 1 == j) s.at = i;
        __syncthreads();
        for (int k = 0; k < SP_LAST / WAVE; ++k) seen += s.redc[k];
        h.index = s.at;
        __syncthreads();
    }
    return h;
}

// The mass of all weights >= min-p's, at least the first token's, when the
// tokens around the border were not collected.
template <typename T>
__device__ __forceinline__ uint64_t sp_mass_from(SpShared& s, const SpRow<T>& row, float q) {
    const uint64_t wq = sp_min_weight(q);
    int lo, hi;
    sp_min_bins(q, row.per, lo, hi);
    uint64_t part = 0;
    row.template each<SP_LAST>(0, 1, [&](float l, int) {
        const int b = row.bin(row.dist(l));
        if (b >= lo && b <= hi) {
            const uint64_t w = row.weight(l);
            if (w >= wq) part += w;
        }
    });
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) part += __shfl_xor(part, o, WAVE);
    if ((threadIdx.x & 63) == 0) s.red[threadIdx.x >> 6] = part;
    __syncthreads();
    uint64_t m = lo ? s.M[lo - 1] : 0;
    for (int i = 0; i < SP_LAST / WAVE; ++i) m += s.red[i];
    __syncthreads();
    return m;
}

// The same from the sorted tokens, whose weights smass holds: they are all
// those of the border's bins, or all of the first k; below: the mass of the
// bins before the border's.
__device__ __forceinline__ uint64_t sp_mass_from_sorted(const SpShared& s, float q, uint64_t below) {
    // weights fall along the order: the last sorted token of enough weight
    const uint64_t wq = sp_min_weight(q);
    int lo = -1, hi = (int)s.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const uint64_t w = s.smass[mid];
        if (w >= wq)
            lo = mid;
        else
            hi = mid - 1;
    }
    const uint64_t m = lo >= 0 ? s.sum[lo] : 0;
    return m > below ? m : below;
}

// One workgroup per row, after the launches above; whole: without them (short
// rows), reading the row three times itself.
template <typename T>
__global__ __launch_bounds__(SP_LAST) void sp_final_kernel(SpArgs a, bool whole) {
    __shared__ SpShared s;
    const int tid = threadIdx.x, r = blockIdx.x;
    SpRow<T> row = sp_row<T>(a, r);
    uint32_t low;
    const uint64_t best = whole ? sp_largest<SP_LAST>(row, 0, 1, s.red, s.redc, low) : sp_row_best(a, r, low);
    if (!sp_reference(a, r, best, low, row)) {
        if (tid == 0) {
            a.token[r] = best == 0 ? -1 : sp_key_index(best);
            if (a.prob) a.prob[r] = best == 0 ? 0.0f : 1.0f;
        }
        return;
    }
    const uint32_t* cnt = s.scnt;
    const uint64_t* mass = s.smass;
    if (whole) {
        static_assert(SP_CAP >= SP_BINS, "the table fits");
        double* table = reinterpret_cast<double*>(s.sum);
        for (int i = tid; i < SP_BINS; i += SP_LAST) {
            s.scnt[i] = 0;
            s.smass[i] = 0;
            table[i] = sp_bin_exp(i, row.unit);
        }
        __syncthreads();
        sp_histogram<SP_LAST>(a, r, row, 0, 1, s.scnt, s.smass, table);
    } else {
        cnt = a.cnt + (size_t)r * SP_BINS;
        mass = a.mass + (size_t)r * SP_BINS;
    }
    sp_running<SP_LAST>(cnt, mass, s.C, s.M, s.redc, s.red);
    const SpFilters f = sp_filters(a, r, s.C[SP_BINS - 1]);
    if (whole) {
        const SpBins bins = sp_bins(f, row.per, s.C, s.M);
        sp_gather(s, row, [&](int b, uint32_t) { return bins.has(b); });
    } else {
        if (tid == 0) s.n = a.n[(size_t)r * 64];
        __syncthreads();
        for (uint32_t i = tid; i < s.n && i < SP_CAP; i += SP_LAST) s.key[i] = a.list[(size_t)r * SP_CAP + i];
        __syncthreads();
    }
    const bool fits = s.n <= SP_CAP;
    if (fits) {
        sp_sort(s);
        sp_sums(s, row, true, 0, 0);
    }
    // mass kept so far: of all tokens, of the first k, of top-p's prefix and
    // (a nested prefix too) of min-p's; then the token
    uint64_t kept = s.M[SP_BINS - 1];
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
        uint64_t t;
        if (step == 0) {
            if (!f.k) continue;
            t = (uint64_t)f.k;
        } else if (step == 1) {
            if (!(f.p < 1.0f)) continue;
            t = sp_top_p(f.p, kept);
        } else {
            if (f.q > 1.0f) {
                kept = SP_ONE_I;
            } else if (f.q > 0.0f) {
                int lo, hi;
                sp_min_bins(f.q, row.per, lo, hi);
                uint64_t m;
                if (fits)
                    m = sp_mass_from_sorted(s, f.q, lo ? s.M[lo - 1] : 0);
                else
                    m = sp_mass_from(s, row, f.q);
                kept = kept < m ? kept : m;
            }
            t = sp_target(f.u, kept);
        }
        const SpHit h = fits ? sp_hit(s, step == 0, t) : sp_narrow(s, row, step == 0, t);
        if (step < 2) {
            kept = h.mass;
        } else if (tid == 0) {
            a.token[r] = h.index;
            if (a.prob) a.prob[r] = (float)((double)h.w / (double)kept);
        }
    }
}

// Rows of at most this many tokens take one launch (8192 tokens: 1 row 22.8 us
// against 29.8 with four launches, 256 rows 24.4 against 41.3; 32000 tokens: 1
// row 43 against 30, 64 rows 46 against 41, 512 rows 103 against 101).
constexpr int SP_WHOLE = 16384;

// Workgroups per row: 4096 tokens each, but about 512 in all (64 rows of 131072
// 58.7 us, 256 of 50003 80.0; with 1024 61.7 and 83.5, with 2048 77.6 and 96.5:
// each has the row's histogram to scan).
int sp_splits(int B, int V) {
    const int by_len = (V + 4095) / 4096, by_rows = 512 / B;
    const int s = by_len < by_rows ? by_len : by_rows;
    return s < 1 ? 1 : (s > SP_MAX_SPLITS ? SP_MAX_SPLITS : s);
}

template <typename T>
hipError_t sp_launch(SpArgs& a, int B, hipStream_t s) {
    const bool whole = a.V <= SP_WHOLE;
    if (!whole) {
        const dim3 g((uint32_t)a.S, (uint32_t)B);
        sp_max_kernel<T><<<g, SP_THREADS, 0, s>>>(a);
        sp_hist_kernel<T><<<g, SP_THREADS, 0, s>>>(a);
        sp_collect_kernel<T><<<g, SP_THREADS, 0, s>>>(a);
    }
    sp_final_kernel<T><<<B, SP_LAST, 0, s>>>(a, whole);
    return hipGetLastError();
}

size_t sp_align(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

size_t sample_workspace_bytes(int B, int V) {
    if (V <= SP_WHOLE) return 0;
    const size_t b = (size_t)B;
    return sp_align(b * SP_MAX_SPLITS * 8) + b * (SP_BINS * 8 + SP_BINS * 4 + SP_CAP * 8 + SP_MAX_SPLITS * 4 + 256);
}

hipError_t launch_sample(int B, int V, int64_t ld, bool f32, const void* logits, const float* temperature,
                         const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* token,
                         float* prob, void* workspace, hipStream_t s) {
    SpArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.V = V;
    a.S = sp_splits(B, V);
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.token = token;
    a.prob = prob;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const size_t b = (size_t)B;
    a.best = reinterpret_cast<uint64_t*>(ws);
    ws += sp_align(b * SP_MAX_SPLITS * 8);
    a.mass = reinterpret_cast<uint64_t*>(ws);
    ws += b * SP_BINS * 8;
    a.list = reinterpret_cast<uint64_t*>(ws);
    ws += b * SP_CAP * 8;
    a.cnt = reinterpret_cast<uint32_t*>(ws);
    ws += b * SP_BINS * 4;
    a.n = reinterpret_cast<uint32_t*>(ws);
    ws += b * 256;
    a.low = reinterpret_cast<uint32_t*>(ws);
    return f32 ? sp_launch<float>(a, B, s) : sp_launch<uint16_t>(a, B, s);
}

}  // namespace ds4
