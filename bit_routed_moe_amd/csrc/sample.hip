// Token sampling: temperature, top-k, top-p, min-p and one given random number
// per row.
//
// The tokens of a row in (logit descending, index ascending) order have
// weights w_i = exp((l_i - max) / T).  Each filter keeps a prefix of that
// order, so the kept set is the shortest of three prefixes, its mass the least
// of three masses, and the sampled token is the one at which the running sum
// first exceeds u times that mass.  Nothing has to be sorted: each question is
// "where does a running count or sum cross a value", answered by a histogram
// over (max - l) / T (64 bins per unit) and then among the tokens of one bin.
//
// Weights are held as integers, round(w * 2^43) in 64 bits, from a 64-bit exp:
// integer sums do not depend on the order of additions, so the histogram's
// atomics and every sum below are reproducible, and a border is moved by at
// most 2^-44 of the largest weight per token.  Tokens below e^-31 of the
// largest weight round to 0 and are never chosen.
//
// One workgroup of 16 waves per row; every pass re-reads the row (from L2
// after the first), the next step's loads in flight while one is worked on.
#include "common.hpp"
#include "launch.hpp"

namespace ds4 {

namespace {

constexpr int SP_THREADS = 1024;
constexpr int SP_BINS = 2048;           // bin b: b <= 64 (max - l) / T < b + 1
constexpr double SP_PER_UNIT = 64.0;
constexpr int SP_CAP = 1024;            // tokens compared with each other at once
constexpr int SP_UNROLL = 4;             // loads of 16 bytes per lane and step (fp32 logits)
constexpr double SP_ONE = 8796093022208.0;   // 2^43
constexpr uint64_t SP_ONE_I = (uint64_t)1 << 43;

struct SpArgs {
    const void* logits;
    int64_t ld;
    int V;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t* top_k;
    int32_t* token;
    float* prob;
};

struct SpShared {
    uint32_t cnt[SP_BINS];       // histogram, then running counts (inclusive)
    uint64_t mass[SP_BINS];      // the same for weights
    uint32_t scnt[SP_BINS];      // histogram of a piece of one bin
    uint64_t smass[SP_BINS];
    uint64_t key[SP_CAP];        // collected tokens: route_key and weight
    uint64_t w[SP_CAP];
    uint64_t red[SP_THREADS / WAVE + 1];
    uint32_t redc[SP_THREADS / WAVE + 1];
    uint32_t n;                  // collected tokens
    int bin;
    uint64_t ans, anskey, answ;
};

__device__ __forceinline__ uint32_t sp_k32(float l) { return (uint32_t)(route_key(l, 0) >> 32); }

// (max - l) / T; 0 for the largest logits themselves, also infinite ones.
__device__ __forceinline__ double sp_dist(float l, float mx, double inv_t) {
    return l == mx ? 0.0 : ((double)mx - (double)l) * inv_t;
}
// Bin of a distance, SP_BINS and above for tokens of no weight.
__device__ __forceinline__ int sp_bin(double d) { return d < 32.0 ? (int)(d * SP_PER_UNIT) : SP_BINS; }
__device__ __forceinline__ uint64_t sp_weight(double d) {
    return d < 31.0 ? (uint64_t)__double2ll_rn(exp(-d) * SP_ONE) : 0;
}

// f(logit, index) for every token of the row that is above -infinity and not
// NaN, in no particular order.
template <typename T, typename F>
__device__ __forceinline__ void sp_each(const T* row, int V, const F& f) {
    constexpr int N = 16 / sizeof(T);
    const uintptr_t p = reinterpret_cast<uintptr_t>(row);
    const int skip = (int)(p & 15) / (int)sizeof(T);    // elements of the first 16 bytes before the row
    const u32x4* base = reinterpret_cast<const u32x4*>(p & ~(uintptr_t)15);
    const int nch = (skip + V + N - 1) / N;
    constexpr int UN = SP_UNROLL / (4 / (int)sizeof(T));   // 16 tokens per lane and step
    u32x4 v[UN], nx[UN];
#pragma unroll
    for (int j = 0; j < UN; ++j) nx[j] = base[min((int)threadIdx.x + j * SP_THREADS, nch - 1)];
#pragma unroll 1
    for (int c0 = threadIdx.x; c0 < nch; c0 += SP_THREADS * UN) {
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            v[j] = nx[j];
            nx[j] = base[min(c0 + (UN + j) * SP_THREADS, nch - 1)];
        }
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            const int c = c0 + j * SP_THREADS;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int idx = c * N + i - skip;
                float l;
                if constexpr (sizeof(T) == 4)
                    l = __uint_as_float(v[j][i]);
                else
                    l = __uint_as_float((i & 1) ? v[j][i >> 1] & 0xFFFF0000u : v[j][i >> 1] << 16);
                if (c < nch && idx >= 0 && idx < V && l > -INFINITY) f(l, idx);
            }
        }
    }
}

// Adds a token to a histogram.  Lanes that all meet in one bin (equal logits)
// add up first: same-address LDS atomics take one lane after the other.
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

// Histogram -> inclusive running counts and sums, two bins per thread.
__device__ __forceinline__ void sp_scan(uint32_t* cnt, uint64_t* mass, SpShared& s) {
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    __syncthreads();
    const uint32_t c0 = cnt[2 * tid], c1 = cnt[2 * tid + 1];
    const uint64_t m0 = mass[2 * tid], m1 = mass[2 * tid + 1];
    uint32_t c = c0 + c1;
    uint64_t m = m0 + m1;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t cu = __shfl_up(c, o, WAVE);
        const uint64_t mu = __shfl_up(m, o, WAVE);
        if (lane >= o) {
            c += cu;
            m += mu;
        }
    }
    if (lane == 63) {
        s.redc[wv] = c;
        s.red[wv] = m;
    }
    __syncthreads();
    for (int i = 0; i < wv; ++i) {
        c += s.redc[i];
        m += s.red[i];
    }
    __syncthreads();
    cnt[2 * tid + 1] = c;
    mass[2 * tid + 1] = m;
    cnt[2 * tid] = c - c1;
    mass[2 * tid] = m - m1;
    __syncthreads();
}

// First bin whose running count (by_rank) or sum reaches t >= 1; SP_BINS if none.
__device__ __forceinline__ int sp_find(const uint32_t* cnt, const uint64_t* mass, bool by_rank, uint64_t t,
                                       SpShared& s) {
    const int tid = threadIdx.x;
    if (tid == 0) s.bin = SP_BINS;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int b = 2 * tid + i;
        const uint64_t here = by_rank ? cnt[b] : mass[b];
        const uint64_t before = b == 0 ? 0 : (by_rank ? cnt[b - 1] : mass[b - 1]);
        if (before < t && t <= here) s.bin = b;
    }
    __syncthreads();
    const int b = s.bin;
    __syncthreads();
    return b;
}

// A crossing: the running sum up to and with the token (mass), the token's
// weight and index.
struct SpHit {
    uint64_t mass, w;
    int index;
};

// Among the s.n collected tokens, which continue a running count c0 and sum
// m0, the one at which the count (by_rank) or the sum reaches t.
__device__ __forceinline__ SpHit sp_among(SpShared& s, uint64_t c0, uint64_t m0, bool by_rank, uint64_t t) {
    const int tid = threadIdx.x, n = (int)s.n;
    if (tid < n) {
        const uint64_t k = s.key[tid], w = s.w[tid];
        uint64_t c = c0 + 1, m = m0 + w;
        for (int j = 0; j < n; ++j) {
            if (s.key[j] > k) {
                ++c;
                m += s.w[j];
            }
        }
        if (by_rank ? c == t : (m >= t && m - w < t)) {
            s.ans = m;
            s.answ = w;
            s.anskey = k;
        }
    }
    __syncthreads();
    SpHit h;
    h.mass = s.ans;
    h.w = s.answ;
    h.index = (int)(0xFFFFFFFFu - (uint32_t)s.anskey);
    __syncthreads();
    return h;
}

template <typename T>
struct SpRow {
    const T* row;
    int V;
    float mx;
    double inv_t;
    int c_lo, c_hi;   // bins whose tokens are collected (all of them), c_hi < c_lo: none

    // Collects the tokens for which in(bin, k32) holds (at most SP_CAP exist).
    template <typename F>
    __device__ __forceinline__ void collect(SpShared& s, const F& in) {
        if (threadIdx.x == 0) s.n = 0;
        __syncthreads();
        sp_each(row, V, [&](float l, int idx) {
            const double d = sp_dist(l, mx, inv_t);
            const int b = sp_bin(d);
            if (b < SP_BINS && in(b, sp_k32(l))) {
                const uint32_t at = atomicAdd(&s.n, 1u);
                if (at < SP_CAP) {
                    s.key[at] = route_key(l, idx);
                    s.w[at] = sp_weight(d);
                }
            }
        });
        __syncthreads();
    }

    // The mass of all weights >= q: whole bins, and the tokens of the bins
    // around the border one by one (at least the first token's).
    __device__ __forceinline__ uint64_t mass_from(SpShared& s, float q) const {
        if (q > 1.0f) return SP_ONE_I;
        const uint64_t wq = (uint64_t)ceil((double)q * SP_ONE);
        const int bq = (int)(fmin(-log((double)q), 31.0) * SP_PER_UNIT);
        const int lo = max(bq - 1, 0), hi = min(bq + 1, SP_BINS - 1);
        uint64_t part = 0;
        sp_each(row, V, [&](float l, int) {
            const double d = sp_dist(l, mx, inv_t);
            const int b = sp_bin(d);
            if (b >= lo && b <= hi) {
                const uint64_t w = sp_weight(d);
                if (w >= wq) part += w;
            }
        });
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) part += __shfl_xor(part, o, WAVE);
        if ((threadIdx.x & 63) == 0) s.red[threadIdx.x >> 6] = part;
        __syncthreads();
        uint64_t m = lo ? s.mass[lo - 1] : 0;
        for (int i = 0; i < SP_THREADS / WAVE; ++i) m += s.red[i];
        __syncthreads();
        return m;
    }

    // The crossing at running count or sum t, which lies in bin b.
    __device__ SpHit resolve(SpShared& s, int b, bool by_rank, uint64_t t) {
        uint64_t c0 = b ? s.cnt[b - 1] : 0, m0 = b ? s.mass[b - 1] : 0;
        if (b >= c_lo && b <= c_hi) {
            // collected bins start at c_lo: count from there on
            c0 = c_lo ? s.cnt[c_lo - 1] : 0;
            m0 = c_lo ? s.mass[c_lo - 1] : 0;
            return sp_among(s, c0, m0, by_rank, t);
        }
        c_lo = 0;
        c_hi = -1;
        uint32_t n = s.cnt[b] - (uint32_t)c0;
        if (n <= SP_CAP) {
            // the first k tokens hold every later answer: keep all of them if they fit
            c_lo = by_rank && s.cnt[b] <= SP_CAP ? 0 : b;
            c_hi = b;
            const int from = c_lo;
            collect(s, [&](int bb, uint32_t) { return bb >= from && bb <= b; });
            if (from == 0) c0 = m0 = 0;
            return sp_among(s, c0, m0, by_rank, t);
        }
        // more tokens than fit: narrow the range [lo, hi] of order-preserving
        // logit bits by histograms of 2048 pieces
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
        sp_each(row, V, [&](float l, int) {
            if (sp_bin(sp_dist(l, mx, inv_t)) == b) {
                const uint32_t k = sp_k32(l);
                lo = min(lo, k);
                hi = max(hi, k);
            }
        });
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            lo = min(lo, (uint32_t)__shfl_xor((int)lo, o, WAVE));
            hi = max(hi, (uint32_t)__shfl_xor((int)hi, o, WAVE));
        }
        if ((threadIdx.x & 63) == 0) s.red[threadIdx.x >> 6] = ((uint64_t)hi << 32) | lo;
        __syncthreads();
        for (int i = 0; i < SP_THREADS / WAVE; ++i) {
            lo = min(lo, (uint32_t)s.red[i]);
            hi = max(hi, (uint32_t)(s.red[i] >> 32));
        }
        __syncthreads();
        while (n > SP_CAP && lo < hi) {   // (each round divides the range by up to 2048)
            int shift = 0;
            while (((hi - lo) >> shift) >= SP_BINS) ++shift;
            for (int i = threadIdx.x; i < SP_BINS; i += SP_THREADS) {
                s.scnt[i] = 0;
                s.smass[i] = 0;
            }
            __syncthreads();
            sp_each(row, V, [&](float l, int) {
                const double d = sp_dist(l, mx, inv_t);
                const uint32_t k = sp_k32(l);
                if (sp_bin(d) == b && k >= lo && k <= hi)
                    sp_count(s.scnt, s.smass, (int)((hi - k) >> shift), sp_weight(d));
            });
            sp_scan(s.scnt, s.smass, s);
            const int p = sp_find(s.scnt, s.smass, by_rank, t - (by_rank ? c0 : m0), s);
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
            collect(s, [&](int bb, uint32_t k) { return bb == b && k >= lo && k <= hi; });
            return sp_among(s, c0, m0, by_rank, t);
        }
        // equal logits: the j-th of them in index order
        const float val = key_value((uint64_t)hi << 32);
        const uint64_t w = sp_weight(sp_dist(val, mx, inv_t));
        const uint64_t j = by_rank ? t - c0 : (t - m0 + w - 1) / w;
        uint64_t seen = 0;
        SpHit h;
        h.mass = m0 + j * w;
        h.w = w;
        h.index = -1;
        for (int i0 = 0; i0 < V; i0 += SP_THREADS) {
            const int i = i0 + threadIdx.x;
            bool eq = false;
            if (i < V) {
                float l;
                if constexpr (sizeof(T) == 4)
                    l = row[i];
                else
                    l = bf16_to_f32(row[i]);
                eq = l > -INFINITY && sp_k32(l) == hi;
            }
            const uint64_t vote = __ballot(eq);
            if ((threadIdx.x & 63) == 0) s.redc[threadIdx.x >> 6] = (uint32_t)__popcll(vote);
            if (threadIdx.x == 0) s.bin = -1;
            __syncthreads();
            uint64_t at = seen;
            for (int k = 0; k < (int)(threadIdx.x >> 6); ++k) at += s.redc[k];
            at += __popcll(vote & (((uint64_t)1 << (threadIdx.x & 63)) - 1));
            if (eq && at + 1 == j) s.bin = i;
            __syncthreads();
            for (int k = 0; k < SP_THREADS / WAVE; ++k) seen += s.redc[k];
            h.index = s.bin;
            __syncthreads();
            if (h.index >= 0) break;
        }
        return h;
    }
};

template <typename T>
__global__ __launch_bounds__(SP_THREADS) void sample_kernel(SpArgs a) {
    __shared__ SpShared s;
    const int tid = threadIdx.x, r = blockIdx.x;
    SpRow<T> row;
    row.row = static_cast<const T*>(a.logits) + (size_t)r * a.ld;
    row.V = a.V;
    row.c_lo = 0;
    row.c_hi = -1;

    // the largest logit, at its lowest index
    uint64_t best = 0;
    sp_each(row.row, a.V, [&](float l, int idx) {
        const uint64_t k = route_key(l, idx);
        best = best > k ? best : k;
    });
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const uint64_t k = __shfl_xor(best, o, WAVE);
        best = best > k ? best : k;
    }
    if ((tid & 63) == 0) s.red[tid >> 6] = best;
    for (int i = tid; i < SP_BINS; i += SP_THREADS) {
        s.cnt[i] = 0;
        s.mass[i] = 0;
    }
    __syncthreads();
    for (int i = 0; i < SP_THREADS / WAVE; ++i) best = best > s.red[i] ? best : s.red[i];
    __syncthreads();

    const float temp = a.temperature ? a.temperature[r] : 1.0f;
    if (best == 0 || !(temp > 0.0f)) {   // nothing left to choose, or the greedy choice
        if (tid == 0) {
            a.token[r] = best == 0 ? -1 : (int)(0xFFFFFFFFu - (uint32_t)best);
            if (a.prob) a.prob[r] = best == 0 ? 0.0f : 1.0f;
        }
        return;
    }
    row.mx = key_value(best);
    row.inv_t = 1.0 / (double)temp;
    const float mx = row.mx;
    const double inv_t = row.inv_t;

    sp_each(row.row, a.V, [&](float l, int) {
        const double d = sp_dist(l, mx, inv_t);
        const int b = sp_bin(d);
        if (b < SP_BINS) sp_count(s.cnt, s.mass, b, sp_weight(d));
    });
    sp_scan(s.cnt, s.mass, s);

    // mass kept so far: of all tokens, of the first k, of top-p's prefix and
    // (a nested prefix too) of min-p's; then the token
    uint64_t kept = s.mass[SP_BINS - 1];
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
        bool by_rank = false;
        uint64_t t;
        if (step == 0) {
            const int k = a.top_k ? a.top_k[r] : 0;
            if (k <= 0 || (uint32_t)k >= s.cnt[SP_BINS - 1]) continue;   // (tokens past the bins weigh nothing)
            by_rank = true;
            t = (uint64_t)k;
        } else if (step == 1) {
            const float p = a.top_p ? a.top_p[r] : 1.0f;
            if (!(p < 1.0f)) continue;
            const double want = ceil((double)p * (double)kept);
            t = want < 1.0 ? 1 : (uint64_t)want;
            t = t < kept ? t : kept;
        } else {
            const float q = a.min_p ? a.min_p[r] : 0.0f;
            if (q > 0.0f) {
                const uint64_t m = row.mass_from(s, q);
                kept = kept < m ? kept : m;
            }
            const float u = a.u[r];
            const double at = u > 0.0f ? floor((double)u * (double)kept) : 0.0;
            t = at < (double)kept ? (uint64_t)at + 1 : kept;
            t = t < kept ? t : kept;
        }
        const int b = sp_find(s.cnt, s.mass, by_rank, t, s);
        if (by_rank && s.cnt[b] == (uint32_t)t) {
            kept = s.mass[b];
            continue;
        }
        const SpHit h = row.resolve(s, b, by_rank, t);
        if (step < 2) {
            kept = h.mass;
        } else if (tid == 0) {
            a.token[r] = h.index;
            if (a.prob) a.prob[r] = (float)((double)h.w / (double)kept);
        }
    }
}

}  // namespace

hipError_t launch_sample(int B, int V, int64_t ld, bool f32, const void* logits, const float* temperature,
                         const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* token,
                         float* prob, hipStream_t s) {
    SpArgs a{logits, ld, V, temperature, top_p, min_p, u, top_k, token, prob};
    if (f32)
        sample_kernel<float><<<B, SP_THREADS, 0, s>>>(a);
    else
        sample_kernel<uint16_t><<<B, SP_THREADS, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace ds4
