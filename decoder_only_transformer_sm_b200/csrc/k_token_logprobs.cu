// Log-probabilities of given tokens with entropy and top alternatives, and their
// gradient ("GPT-2 from Scratch", "A generation loop": the distribution a token is
// drawn from is softmax(logits / temperature)).
//
// With c = log2(e) / tau, m = max x, d = x - m, s = sum 2^(c d), w = sum 2^(c d) d:
//   lse = m / tau + log s,   log p_v = d_v / tau - log s,   H = -sum p log p = log s - w / (tau s).
// Differences to the maximum are taken before they are scaled, so the terms that
// count carry the smallest errors. Masked logits are -inf: they add nothing to s and
// w. A row of which nothing is left has lse = log p = -inf and H = 0; a row with NaN or
// +inf has NaN in all of them.
//
// Forward: one pass over the row by NT threads (a warp for short rows, a block, or with
// few long rows the blocks of a cluster). A thread keeps a running (m, s, w) and rescales it
// when a load of several vectors raises m; the threads join theirs at the end, the blocks
// through distributed shared memory. Top alternatives come from the same pass: a thread
// knows its largest value at the end (of a warp, those of two halves of its vectors), and the
// top_k-th largest of those is a bound that at least top_k values of the row reach. Only vectors
// of threads (halves) that reach it can hold one of the top_k: they are read again (from L2), and
// the few values that reach the bound are ranked by 64-bit keys (value, then lowest index). Where
// many values equal the bound, only the larger ones are gathered, and the first equal ones in the
// row's order after them; the same way -inf fills up where fewer than top_k threads saw a number.
// (Where even the larger ones are too many, a few threads holding most of a row's largest values,
// each warp keeps a sorted list.)
// 8192 x 50257 bf16: 129 us without alternatives (6.4 TB/s), 150 with five, 231 with 32 (normal logits, from a CUDA graph,
// two sets of them in turn; with a favoured token in each row, as a model's, 170 with five).
#include <cooperative_groups.h>

#include <type_traits>

#include "kernels.cuh"

namespace gpt2 {

namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float LOWEST = -3.402823466e38f;
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float nan_value() { return __uint_as_float(0x7fc00000u); }

// Unsigned numbers whose order is that of the values: -0 as +0, NaN above +inf. No value has 0 or all ones.
__device__ __forceinline__ unsigned order_of(float x) {
    const unsigned b = __float_as_uint(x + 0.f);
    if (x != x) return 0xffc00000u;
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned o) {
    if (o == 0xffc00000u) return nan_value();
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
// Larger value first, then lower index.
__device__ __forceinline__ u64 key_of(unsigned order, int v) { return ((u64)order << 32) | (unsigned)~v; }

// A row of V elements as vectors of 16 bytes: 0 .. full - 1 are whole and aligned, full holds
// the elements before them (0 .. N - 1), full + 1 those after them.
template <typename T>
struct RowVecs {
    static constexpr int N = 16 / sizeof(T);
    int head, full, V;
    __device__ __forceinline__ RowVecs(const T* row, int V_) : V(V_) {
        head = min(V, (int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(T));
        full = (V - head) / N;
    }
    __device__ __forceinline__ int count() const { return full + 2; }
    __device__ __forceinline__ int first(int i) const { return i == full ? 0 : head + min(i, full) * N; }
    __device__ __forceinline__ int last(int i) const { return i < full ? head + (i + 1) * N : i == full ? head : V; }
};

__device__ __forceinline__ void unpack(const uint4& q, float (&f)[8], bf16) {
    const unsigned u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& q, float (&f)[4], float) {
    f[0] = __uint_as_float(q.x);
    f[1] = __uint_as_float(q.y);
    f[2] = __uint_as_float(q.z);
    f[3] = __uint_as_float(q.w);
}

__device__ __forceinline__ uint4 pack(const float (&f)[8], bf16) {
    uint4 q;
    unsigned* u = reinterpret_cast<unsigned*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const unsigned*>(&t);
    }
    return q;
}
__device__ __forceinline__ uint4 pack(const float (&f)[4], float) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// Vector i element by element: for the ends of a row, and for rows whose vectors are laid out
// after another row's boundaries. What lies outside is -inf.
template <typename T>
__device__ __noinline__ uint4 gather_vec(const T* row, const RowVecs<T> rv, int i, int end) {
    constexpr unsigned NONE = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    union {
        uint4 q;
        T t[RowVecs<T>::N];
    } u;
    u.q = make_uint4(NONE, NONE, NONE, NONE);
    if (i < end) {
        const int a = rv.first(i), b = rv.last(i);
#pragma unroll
        for (int j = 0; j < RowVecs<T>::N; ++j)
            if (a + j < b) u.t[j] = row[a + j];
    }
    return u.q;
}
template <typename T>
__device__ __noinline__ void scatter_vec(T* row, const RowVecs<T> rv, int i, uint4 q) {
    union {
        uint4 q;
        T t[RowVecs<T>::N];
    } u;
    u.q = q;
    const int a = rv.first(i), b = rv.last(i);
#pragma unroll
    for (int j = 0; j < RowVecs<T>::N; ++j)
        if (a + j < b) row[a + j] = u.t[j];
}

// Vector i's bits (none at or past `end`).
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, const RowVecs<T>& rv, int i, int end) {
    if (i < min(end, rv.full)) return __ldg(reinterpret_cast<const uint4*>(row + rv.head) + i);
    return gather_vec(row, rv, i, end);
}

// Largest and smallest of U vectors, NaN passed over.
template <int U>
__device__ __forceinline__ void extremes(const uint4 (&q)[U], float& top, float& low, bf16) {
    __nv_bfloat162 hi, lo;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q[u]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hi = u + j ? __hmax2(hi, h[j]) : h[j];
            lo = u + j ? __hmin2(lo, h[j]) : h[j];
        }
    }
    const float2 a = __bfloat1622float2(hi), b = __bfloat1622float2(lo);
    top = fmaxf(a.x, a.y);
    low = fminf(b.x, b.y);
}
template <int U>
__device__ __forceinline__ void extremes(const uint4 (&q)[U], float& top, float& low, float) {
    top = NEG_INF;
    low = -NEG_INF;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[4];
        unpack(q[u], f, 0.f);
        top = fmaxf(fmaxf(top, fmaxf(f[0], f[1])), fmaxf(f[2], f[3]));
        low = fminf(fminf(low, fminf(f[0], f[1])), fminf(f[2], f[3]));
    }
}

struct Sums {
    float m, s, w;   // m = -FLT_MAX and s = 0 where nothing was seen
    __device__ __forceinline__ void raise(float to, float c) {
        const float r = ex2_approx((m - to) * c);
        w = (w - fminf(to - m, 1e30f) * s) * r;   // cut off only where r is 0 (LOGPROB_MAX_TEMPERATURE) or s is
        s *= r;
        m = to;
    }
    __device__ __forceinline__ void join(Sums o, float c) {
        const float to = fmaxf(m, o.m);
        raise(to, c);
        o.raise(to, c);
        s += o.s;
        w += o.w;
    }
    // The terms of U vectors, none above m. MASKED: there may be -inf, whose e = 0 meets d = -inf.
    template <bool MASKED, typename T, int U>
    __device__ __forceinline__ void add(const uint4 (&q)[U], float c) {
        constexpr int N = RowVecs<T>::N;
        const f32x2 m2 = pk2(-m, -m), c2 = pk2(c, c);
        f32x2 s2 = pk2(s, 0.f), w2 = pk2(w, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[N];
            unpack(q[u], f, T());
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                f32x2 d2 = add2(pk2(f[j], f[j + 1]), m2);
                float y0, y1;
                upk2(mul2(d2, c2), y0, y1);
                const f32x2 e2 = pk2(ex2_approx(y0), ex2_approx(y1));
                if (MASKED) {
                    float d0, d1;
                    upk2(d2, d0, d1);
                    d2 = pk2(fmaxf(d0, LOWEST), fmaxf(d1, LOWEST));
                }
                s2 = add2(s2, e2);
                w2 = fma2(e2, d2, w2);
            }
        }
        float s0, s1, w0, w1;
        upk2(s2, s0, s1);
        upk2(w2, w0, w1);
        s = s0 + s1;
        w = w0 + w1;
    }
};

// Inserts the keys that `pass` lanes hold into the warp's descending list (lane i: the
// i-th largest, 0 for none).
__device__ __forceinline__ void insert(u64& list, u64 key, bool pass) {
    const int lane = threadIdx.x & 31;
    for (unsigned todo = __ballot_sync(0xffffffffu, pass); todo; todo &= todo - 1) {
        const u64 k = __shfl_sync(0xffffffffu, key, __ffs(todo) - 1);
        const int at = __popc(__ballot_sync(0xffffffffu, list > k));
        const u64 up = __shfl_up_sync(0xffffffffu, list, 1);
        if (lane == at) list = k;
        else if (lane > at) list = up;
    }
}

// All threads of a row meet (NT = 32: a warp, several rows a block).
template <int NT>
__device__ __forceinline__ void meet() {
    if (NT == 32) __syncwarp();
    else __syncthreads();
}

// A row's vectors are taken by turns into groups, whose largest values bound the k-th largest from
// below: a thread's vectors, or for a warp (32 values bound too loosely) every other of a thread's.
template <int NT>
constexpr int GROUPS_OF = NT < 64 ? 64 : NT;

template <int NT>
struct ForwardSmem {
    static constexpr int GROUPS = GROUPS_OF<NT>;
    alignas(16) unsigned largest[GROUPS];   // order of each group's largest value
    // 256: what a warp finds in 32 vectors of 8, or the lists of eight. 192 hold the lists of four.
    static constexpr int ROOM = NT == 128 ? 192 : 256;
    static_assert(ROOM >= NT / 32 * LOGPROB_MAX_TOP, "each warp's list fits");
    u64 cand[ROOM];                       // keys that reach the bound
    Sums sums[NT / 32];
    float2 own[NT > 32 ? NT : 1];         // the threads' maxima and sums, see sum_without_largest
    float without[NT / 32];
    int holder;
    int again[GROUPS];                    // the groups whose values are read again
    int scan[NT / 32];
    unsigned bound;
    int n_cand, n_again;
};

// Of a cluster's first block: every block's results.
struct ClusterSmem {
    Sums sums[8];
    float without[8];
    u64 top[8 * LOGPROB_MAX_TOP];
};

// Ranks n keys in shared memory; rank(i, key) is called for those among the k largest.
template <typename F>
__device__ __forceinline__ void for_top(const u64* keys, int n, int k, int nt, F rank) {
    for (int i = threadIdx.x % nt; i < n; i += nt) {
        const u64 mine = keys[i];
        if (mine == 0) continue;
        int above = 0;
        for (int j = 0; j < n; ++j) above += keys[j] > mine;
        if (above < k) rank(above, mine);
    }
}

// Alternatives up to which a warp finds the bound by walking down from the largest value.
constexpr int WALK = 8;

constexpr unsigned ORDER_NEG_INF = 0x007fffffu;   // order_of(-inf)

// Adds to sm.cand the first `need` (at most 32) values of this order among the vectors begin .. end - 1,
// in the order of the row. (Like `lists` a function of its own: rarely needed, and registers.)
template <typename T, int NT>
__device__ __noinline__ void fill(ForwardSmem<NT>& sm, const T* x, const RowVecs<T> rv, int begin, int end, unsigned order,
                                  int need) {
    constexpr int N = RowVecs<T>::N, PER = NT / 32;
    const int tid = threadIdx.x % NT, lane = tid & 31, n0 = sm.n_cand;
    const int head = end > rv.full ? rv.head : 0, from = rv.head + min(begin, rv.full) * N - head;
    const int total = head + max(0, min(end, rv.full) - begin) * N +
                      (end > rv.full + 1 ? rv.V - (rv.head + rv.full * N) : 0);
    int found = 0;
    for (int e0 = 0; e0 < total && found < need; e0 += NT * 8) {
        unsigned hit = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = e0 + tid * 8 + j;
            if (e < total && order_of(to_f(x[e < head ? e : from + e])) == order) hit |= 1u << j;
        }
        int before = __popc(hit);   // of this and the lanes before, then of all threads before
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += v;
        }
        if (lane == 31) sm.scan[tid >> 5] = before;
        before -= __popc(hit);
        meet<NT>();
        int all = 0;
        for (int w = 0; w < PER; ++w) {
            if (w < (tid >> 5)) before += sm.scan[w];
            all += sm.scan[w];
        }
        for (int rank = found + before; hit && rank < need; hit &= hit - 1, ++rank) {
            const int e = e0 + tid * 8 + __ffs(hit) - 1;
            sm.cand[n0 + rank] = key_of(order, e < head ? e : from + e);
        }
        found += all;
        meet<NT>();
    }
    if (tid == 0) sm.n_cand = n0 + min(found, need);
    meet<NT>();
}

// Leaves in sm.cand the top_k of the chosen groups' values that reach `bound`, of those that each warp reads.
template <typename T, int NT>
__device__ __noinline__ void lists(ForwardSmem<NT>& sm, const T* x, const RowVecs<T> rv, int begin, int end, unsigned bound,
                                   int top_k) {
    constexpr int N = RowVecs<T>::N, PER = NT / 32, GROUPS = GROUPS_OF<NT>;
    const int tid = threadIdx.x % NT, lane = tid & 31, n_again = sm.n_again;
    u64 list = 0;
    // 32 lanes read STEPS vectors of a group
    constexpr int STEPS = 32 / N;
    for (int g = tid >> 5; g < n_again; g += PER) {
        const int mine = sm.again[g], j = lane % N;
        for (int i0 = begin; i0 < end; i0 += STEPS * GROUPS) {
            const int i = i0 + lane / N * GROUPS + mine;
            const int e = i < end ? rv.first(i) + j : 0;
            const bool is = i < end && e < rv.last(i);
            const unsigned o = is ? order_of(to_f(x[e])) : 0u;
            const u64 k = key_of(o, e);
            // at most top_k of the list can be among the row's
            const u64 least = __shfl_sync(0xffffffffu, list, top_k - 1);
            insert(list, k, is && o >= bound && k > least);
        }
    }
    const unsigned kept = __ballot_sync(0xffffffffu, list != 0 && lane < top_k);
    int base = 0;
    if (lane == 0 && kept) base = atomicAdd(&sm.n_cand, __popc(kept));
    base = __shfl_sync(0xffffffffu, base, 0);
    if ((kept >> lane) & 1) sm.cand[base + __popc(kept & ((1u << lane) - 1))] = list;
    meet<NT>();
}

// The vectors begin .. end - 1 of a row, for one row's threads.
template <typename T, int NT>
struct Part {
    ForwardSmem<NT>& sm;
    const T* x;
    const RowVecs<T>& rv;
    int begin, end;
    static constexpr int N = RowVecs<T>::N, GROUPS = GROUPS_OF<NT>, PER = GROUPS / 32;

    // sm.again, sm.n_again: the groups whose largest value reaches `bound` (n_again is 0, all have met).
    __device__ __forceinline__ void choose(unsigned bound) {
        const int tid = threadIdx.x % NT;
        for (int g = tid; g < GROUPS; g += NT)
            if (sm.largest[g] >= bound) sm.again[atomicAdd(&sm.n_again, 1)] = g;
        meet<NT>();
    }
    __device__ __forceinline__ void forget() {   // the candidates and the groups chosen
        meet<NT>();
        if (threadIdx.x % NT == 0) sm.n_cand = sm.n_again = 0;
        meet<NT>();
    }

    // Adds the keys of the chosen groups' values that reach `bound` to sm.cand, as far as there is room;
    // sm.n_cand counts them all.
    __device__ __forceinline__ void gather(unsigned bound, bool any_nan) {
        const int tid = threadIdx.x % NT, steps = ceil_div(end - begin, GROUPS), n_again = sm.n_again;
        const float bound_value = value_of(bound);
        constexpr int R = 2;
        for (int k0 = tid; k0 < n_again * steps; k0 += R * NT) {
            uint4 q[R];
            int at[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int k = k0 + r * NT, g = k / steps;   // vector k % steps of group again[g]
                at[r] = g < n_again ? begin + (k - g * steps) * GROUPS + sm.again[g] : end;
                q[r] = at[r] < end ? load_vec(x, rv, at[r], end) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint4 one[1] = {q[r]};
                float top, low;
                extremes(one, top, low, T());
                if (at[r] >= end || (top < bound_value && !any_nan)) continue;
                float f[N];
                unpack(q[r], f, T());
                const int first = rv.first(at[r]), last = rv.last(at[r]);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (f[j] < bound_value || first + j >= last) continue;
                    const unsigned o = order_of(f[j]);
                    if (o < bound) continue;
                    const int n = atomicAdd(&sm.n_cand, 1);
                    if (n < sm.ROOM) sm.cand[n] = key_of(o, first + j);
                }
            }
        }
        meet<NT>();
    }

    // Leaves in sm.cand (sm.n_cand of them, visible to the threads of the row) keys among which are the
    // part's top_k (all of them, if it has fewer values). any_nan: there is NaN or +inf.
    __device__ __forceinline__ void find_top(int top_k, bool any_nan) {
        const int tid = threadIdx.x % NT, lane = tid & 31;
        if (NT == 32 && top_k > WALK) {   // every lane counts those above its own
            const unsigned mine[2] = {sm.largest[lane], sm.largest[lane + 32]};
            int above[2] = {0, 0};
#pragma unroll 4
            for (int j = 0; j < GROUPS; j += 4) {
                const uint4 g = *reinterpret_cast<const uint4*>(sm.largest + j);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    above[i] += (g.x > mine[i]) + (g.y > mine[i]) + (g.z > mine[i]) + (g.w > mine[i]);
            }
            unsigned least = 0xffffffffu;
            int n = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool is = above[i] < top_k && mine[i] > ORDER_NEG_INF;
                const unsigned in = __ballot_sync(0xffffffffu, is);
                if (is) sm.again[n + __popc(in & ((1u << lane) - 1))] = lane + 32 * i;
                if (is) least = min(least, mine[i]);
                n += __popc(in);
            }
            least = __reduce_min_sync(0xffffffffu, least);
            if (lane == 0) {
                sm.bound = least;
                sm.n_again = n;
            }
        } else if (top_k <= WALK) {
            if (tid < 32) {
                unsigned key[PER], bound = 0xffffffffu;
#pragma unroll
                for (int i = 0; i < PER; ++i) key[i] = sm.largest[lane + 32 * i];
                // distinct values from the largest on, until top_k groups have reached them
                for (int n = 0; n < top_k && bound > ORDER_NEG_INF;) {
                    unsigned below = 0;
#pragma unroll
                    for (int i = 0; i < PER; ++i) below = max(below, key[i] < bound ? key[i] : 0u);
                    bound = __reduce_max_sync(0xffffffffu, below);
#pragma unroll
                    for (int i = 0; i < PER; ++i) n += __popc(__ballot_sync(0xffffffffu, key[i] == bound));
                }
                bound = max(bound, ORDER_NEG_INF + 1);
                int n = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const unsigned in = __ballot_sync(0xffffffffu, key[i] >= bound);
                    if ((in >> lane) & 1) sm.again[n + __popc(in & ((1u << lane) - 1))] = lane + 32 * i;
                    n += __popc(in);
                }
                if (lane == 0) {
                    sm.bound = bound;
                    sm.n_again = n;
                }
            }
        } else {   // every thread counts those above its own
            const unsigned mine = sm.largest[tid];
            int above = 0;
#pragma unroll 8
            for (int j = 0; j < NT; j += 4) {
                const uint4 g = *reinterpret_cast<const uint4*>(sm.largest + j);
                above += (g.x > mine) + (g.y > mine) + (g.z > mine) + (g.w > mine);
            }
            if (above < top_k && mine > ORDER_NEG_INF) {
                atomicMin(&sm.bound, mine);
                sm.again[atomicAdd(&sm.n_again, 1)] = tid;
            }
        }
        meet<NT>();
        const int n_again = sm.n_again;
        const bool few = n_again < top_k;   // groups with a number: all their numbers count
        const unsigned bound = few ? ORDER_NEG_INF + 1 : sm.bound;
        bool fits = n_again <= 2 * top_k || n_again * ceil_div(end - begin, GROUPS) * N <= sm.ROOM;
        if (fits) {
            gather(bound, any_nan);
            fits = sm.n_cand <= sm.ROOM;
        }
        if (!fits && !few) {   // many equal to the bound
            forget();
            choose(bound + 1);
            gather(bound + 1, any_nan);
            if (sm.n_cand <= sm.ROOM) {
                if (sm.n_cand < top_k) fill<T, NT>(sm, x, rv, begin, end, bound, top_k - sm.n_cand);
                return;
            }
        }
        if (!fits) {
            forget();
            choose(bound);
            lists<T, NT>(sm, x, rv, begin, end, bound, top_k);
        } else if (few && sm.n_cand < top_k) {
            fill<T, NT>(sm, x, rv, begin, end, ORDER_NEG_INF, top_k - sm.n_cand);
        }
    }
};

// Where the largest token has nearly all of the probability, log s = log(1 + r) with the sum r of all others is small, and
// s, rounded next to 1, holds little of r: with r = 4e-3 that token's log-probability was off by 1.6e-5 of its value. Up to
// this s, r is summed by itself; past it log s is above 0.06, and a few 2^-24 of s are some 1e-6 of it. (8192 x 50257 bf16
// with every row sure: 134 us instead of 128; 20000 x 512: 14.3 instead of 13.)
constexpr float SURE = 1.0625f;
__device__ __forceinline__ bool is_sure(float s) { return s >= 1.f && s < SURE; }   // (0: nothing was seen; NaN)
// log(1 + r) for r up to 1/16 by its series, cut off at r^7 / 8 < 5e-10 of it (log1pf costs short rows 1%).
__device__ __forceinline__ float log_1p_small(float r) {
    float v = 1.f / 7.f;
    v = fmaf(-r, v, 1.f / 6.f);
    v = fmaf(-r, v, 1.f / 5.f);
    v = fmaf(-r, v, 1.f / 4.f);
    v = fmaf(-r, v, 1.f / 3.f);
    v = fmaf(-r, v, 0.5f);
    return fmaf(-r * r, v, r);
}

template <int NT>
__device__ __forceinline__ float sum_of(const float (&v)[NT / 32]) {   // of the warps' values
    float sum = v[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) sum += v[w];
    return sum;
}

// The sum of the vectors begin .. end - 1 without the (only) value m that is the largest. The threads' sums are at hand (own,
// each from the thread's maximum on); that of the thread that holds m is made anew from its vectors, by all threads, element
// by element (a few each, from L2). A warp's lanes have the result, of a block's warps each leaves its part in sm.without.
template <typename T, int NT>
__device__ __forceinline__ float sum_without_largest(ForwardSmem<NT>& sm, const T* x, const RowVecs<T>& rv, int begin, int end,
                                                     float m, float c, float2 own) {
    constexpr int N = RowVecs<T>::N;
    const int tid = threadIdx.x % NT;
    if (NT > 32) own = sm.own[tid];
    const bool holds = own.x == m && own.y > 0.f;
    int holder = 0;
    if (NT > 32) {
        if (holds) sm.holder = tid;
        meet<NT>();
        holder = sm.holder;
    } else {
        holder = __ffs(__ballot_sync(0xffffffffu, holds)) - 1;
    }
    float sum = holds ? 0.f : own.y * ex2_approx((own.x - m) * c);
#pragma unroll 1
    for (int i = begin + holder + tid / N * NT; i < end; i += NT / N * NT) {
        const int e = rv.first(i) + tid % N;
        const float d = (e < rv.last(i) ? to_f(x[e]) : NEG_INF) - m;
        if (d < 0.f) sum += ex2_approx(d * c);
    }
    sum = warp_sum(sum);
    if (NT > 32) {
        if ((tid & 31) == 0) sm.without[tid >> 5] = sum;
        meet<NT>();
    }
    return sum;
}

// Threads of a block: rows of a warp share one.
template <int NT>
constexpr int BLOCK_OF = NT < 128 ? 128 : NT;

template <typename T, int NT, bool CLUSTER>
__global__ void __launch_bounds__(BLOCK_OF<NT>) token_logprobs_kernel(const T* __restrict__ logits, long long ld,
                                                                      int rows, int V, float inv_tau,
                                                                      const int* __restrict__ targets, LogprobOut out,
                                                                      int parts, unsigned* status) {
    constexpr int U = 4, ROWS = BLOCK_OF<NT> / NT, H = GROUPS_OF<NT> / NT;   // H groups a thread
    __shared__ ForwardSmem<NT> sms[ROWS];
    ForwardSmem<NT>& sm = sms[threadIdx.x / NT];
    const int tid = threadIdx.x % NT, lane = tid & 31;
    const int row = CLUSTER ? blockIdx.x / parts : blockIdx.x * ROWS + threadIdx.x / NT;
    const int part = CLUSTER ? blockIdx.x % parts : 0;
    griddep_wait();     // nothing is read or written before the kernel before this one has ended
    if (ROWS > 1 && row >= rows) return;
    const T* x = logits + (long long)row * ld;
    const RowVecs<T> rv(x, V);
    const int per = CLUSTER ? ceil_div(rv.count(), parts) : rv.count();
    const int begin = part * per, end = min(rv.count(), begin + per);
    const float c = LOG2E * inv_tau;
    if (CLUSTER) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if (tid == 0) {
        sm.n_cand = sm.n_again = 0;
        sm.bound = 0xffffffffu;
    }

    Sums a = {LOWEST, 0.f, 0.f};
    float largest[H];
#pragma unroll
    for (int h = 0; h < H; ++h) largest[h] = NEG_INF;
    // q's extremes; vector u is of the group u % H
    auto look = [&](const uint4 (&q)[U], float& top, float& low) {
        top = NEG_INF;
        low = -NEG_INF;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            uint4 some[U / H];
#pragma unroll
            for (int u = 0; u < U / H; ++u) some[u] = q[u * H + h];
            float t, l;
            extremes(some, t, l, T());
            largest[h] = fmaxf(largest[h], t);
            top = fmaxf(top, t);
            low = fminf(low, l);
        }
    };
    {
        // batches of U whole vectors
        int i = begin + tid;
        const uint4* at = reinterpret_cast<const uint4*>(x + rv.head);
        const int stop = min(end, rv.full) - (U - 1) * NT;
        uint4 q[U];
        for (; i < stop; i += U * NT) {
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = __ldg(at + i + u * NT);
            float top, low;
            look(q, top, low);
            if (top > a.m) a.raise(top, c);
            if (low > -1e30f) a.add<false, T>(q, c);
            else a.add<true, T>(q, c);
        }
        // what is left: fewer than U vectors, and the row's ends
        if (i < end) {
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = load_vec(x, rv, i + u * NT, end);
            float top, low;
            look(q, top, low);
            if (top > a.m) a.raise(top, c);
            a.add<true, T>(q, c);
        }
    }

    if (out.top_k) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int g = tid + h * NT;
            unsigned order = begin + g < end ? order_of(largest[h]) : 0u;
            if (a.s != a.s) {   // a NaN, or +inf: find out which
                for (int i = begin + g; i < end; i += GROUPS_OF<NT>)
                    for (int v = rv.first(i); v < rv.last(i); ++v) order = max(order, order_of(to_f(x[v])));
            }
            sm.largest[g] = order;
        }
    }
    // the maximum of all first, so that every thread rescales once
    const float2 own = make_float2(a.m, a.s);
    float without = 0.f;
    {
        if (NT > 32) sm.own[tid] = own;
        float m = warp_max(a.m);
        if (NT > 32) {
            if (lane == 0) sm.sums[tid >> 5].m = m;
            __syncthreads();
            m = sm.sums[0].m;
#pragma unroll
            for (int w = 1; w < NT / 32; ++w) m = fmaxf(m, sm.sums[w].m);
        }
        a.raise(m, c);
        a.s = warp_sum(a.s);
        a.w = warp_sum(a.w);
        if (NT > 32) {
            if (lane == 0) {
                sm.sums[tid >> 5].s = a.s;
                sm.sums[tid >> 5].w = a.w;
            }
            __syncthreads();
            a.s = sm.sums[0].s;
            a.w = sm.sums[0].w;
#pragma unroll
            for (int w = 1; w < NT / 32; ++w) {
                a.s += sm.sums[w].s;
                a.w += sm.sums[w].w;
            }
        } else {
            __syncwarp();
        }
    }
    // (Its place matters to the registers of all rows: after the search, 4096 x 50257 fp32 take 126 us instead of 123 on 256
    // threads; before it, 8192 x 50257 bf16 130 us instead of 128.5 on 128.)
    constexpr bool EARLY = sizeof(T) == 4 || NT == 256;
    if (EARLY && is_sure(a.s)) without = sum_without_largest<T, NT>(sm, x, rv, begin, end, a.m, c, own);
    if (out.top_k && (CLUSTER || a.s != 0.f)) Part<T, NT>{sm, x, rv, begin, end}.find_top(out.top_k, a.s != a.s);
    if (!EARLY && is_sure(a.s)) without = sum_without_largest<T, NT>(sm, x, rv, begin, end, a.m, c, own);
    const u64* keys = sm.cand;
    int n_keys = out.top_k ? sm.n_cand : 0;
    if constexpr (CLUSTER) {
        __shared__ ClusterSmem cs;
        auto cluster = cg::this_cluster();
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // every block has started
        ClusterSmem* first = cluster.map_shared_rank(&cs, 0);
        if (tid == 0) {
            first->sums[part] = a;
            if (is_sure(a.s)) first->without[part] = sum_of<NT>(sm.without);
        }
        if (out.top_k) {
            if (tid < out.top_k && tid >= n_keys) first->top[part * out.top_k + tid] = 0;
            for_top(sm.cand, n_keys, out.top_k, NT, [&](int r, u64 k) { first->top[part * out.top_k + r] = k; });
        }
        cluster.sync();
        if (part != 0) return;
        a = cs.sums[0];
        for (int i = 1; i < parts; ++i) a.join(cs.sums[i], c);
        keys = cs.top;
        n_keys = parts * out.top_k;
        if (is_sure(a.s)) {   // then the part with the largest value was
            without = 0.f;
            for (int i = 0; i < parts; ++i) {
                const Sums b = cs.sums[i];
                without += b.m == a.m && b.s > 0.f ? cs.without[i] : b.s * ex2_approx((b.m - a.m) * c);
            }
        }
    } else if (NT > 32 && is_sure(a.s)) {
        without = sum_of<NT>(sm.without);
    }
    griddep_launch();   // the next kernel's blocks may come: not earlier, they would crowd on the SMs with room
    const float z_max = a.m * inv_tau;
    const bool bad = a.s != a.s || z_max == -NEG_INF, empty = !bad && (a.s == 0.f || z_max == NEG_INF);
    const float log_s = is_sure(a.s) ? log_1p_small(without) : logf(a.s);
    auto settle = [&](float v, float nothing) { return bad ? nan_value() : empty ? nothing : v; };
    auto logp_of = [&](float v) {   // (the difference of two logits may pass fp32's range where that of their z does not)
        const float d = v - a.m;
        return settle((d >= LOWEST ? d * inv_tau : v * inv_tau - z_max) - log_s, NEG_INF);
    };
    if (tid == 0) {
        if (out.lse) out.lse[row] = settle(z_max + log_s, NEG_INF);
        if (out.entropy) out.entropy[row] = settle(log_s - a.w / a.s * inv_tau, 0.f);
        if (out.logp) {
            int t = targets[row];
            if (t < -1 || t >= V) {
                atomicOr(status, STATUS_BAD_TOKEN);
                t = min(max(t, 0), V - 1);
            }
            out.logp[row] = t < 0 ? 0.f : logp_of(to_f(x[t]));
        }
    }
    if (a.s == 0.f && tid < out.top_k) {   // every logit is -inf (logits whose z all overflow keep their order)
        out.top_ids[(long long)row * out.top_k + tid] = tid;
        out.top_logp[(long long)row * out.top_k + tid] = NEG_INF;
    }
    if (a.s != 0.f) for_top(keys, n_keys, out.top_k, NT, [&](int r, u64 k) {
        out.top_ids[(long long)row * out.top_k + r] = (int)~(unsigned)k;
        out.top_logp[(long long)row * out.top_k + r] = logp_of(value_of((unsigned)(k >> 32)));
    });
}

// dx_v = (1/tau) [ g (1[v = t] - p_v) - h p_v (log p_v + H) ], g = dlogp (0 at an ignored
// target), h = dentropy; with d = z_v - lse: p = e^d, and where p is 0 only the target's g is
// left. One pass, bound by reading x and writing dx; NT threads take a run of vectors of a row,
// a block of at least 128 threads the runs of 128 / NT rows.
// dx may be x: a thread writes only what it has read (and x[t] is read by the thread that writes it). 4096 x 50257 bf16, a
// quarter of the rows not read: 120 us (6.0 TB/s; from a CUDA graph on the same buffers).
template <typename T, int NT>
__global__ void __launch_bounds__(NT < 128 ? 128 : NT)
    token_logprobs_bwd_kernel(const T* x0, long long ld, int rows, int V, float tau, float inv_tau,
                              const int* __restrict__ targets, const float* __restrict__ lse,
                              const float* __restrict__ dlogp, const float* __restrict__ entropy,
                              const float* __restrict__ dentropy, T* dx0, long long ldd, int parts, unsigned* status) {
    constexpr int N = RowVecs<T>::N, U = 4;
    constexpr int ROWS = NT < 128 ? 128 / NT : 1;
    const int row = blockIdx.x / parts * ROWS + threadIdx.x / NT, part = blockIdx.x % parts, lane = threadIdx.x % NT;
    griddep_wait();     // nothing is read or written before the kernel before this one has ended
    if (row >= rows) return;
    const T* x = x0 + (long long)row * ld;
    T* dx = dx0 + (long long)row * ldd;
    int t = targets ? targets[row] : -1;
    if (t < -1 || t >= V) {
        if (lane == 0) atomicOr(status, STATUS_BAD_TOKEN);
        t = min(max(t, 0), V - 1);
    }
    const float L = lse[row];
    const float g = dlogp && t >= 0 ? dlogp[row] : 0.f, h = dentropy ? dentropy[row] : 0.f;
    const float H = h != 0.f ? entropy[row] : 0.f;
    const bool none = (g == 0.f && h == 0.f) || L == NEG_INF;
    const float A = -(g + h * H) * inv_tau, B = -h * inv_tau;
    const RowVecs<T> rv(dx, V);   // the vectors of what is written
    const int per = ceil_div(rv.count(), parts), end = min(rv.count(), (part + 1) * per);
    // whole vectors where x has the boundaries of dx, else element by element
    const int whole = (((uintptr_t)x ^ (uintptr_t)dx) & 15) == 0 ? min(end, rv.full) : 0;
    const uint4* from = reinterpret_cast<const uint4*>(x + rv.head);
    uint4* to = reinterpret_cast<uint4*>(dx + rv.head);
    const int i0 = part * per + lane;
    if (none) {
        griddep_launch();
        for (int i = i0; i < end; i += NT) {
            if (i < rv.full) to[i] = make_uint4(0, 0, 0, 0);
            else scatter_vec(dx, rv, i, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    auto load = [&](uint4 (&q)[U], int i) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = i + u * NT;
            if (k < whole) q[u] = from[k];
            else if (k < end) q[u] = gather_vec(x, rv, k, end);
        }
    };
    const f32x2 it2 = pk2(inv_tau, inv_tau), l2 = pk2(-L, -L), e2 = pk2(LOG2E, LOG2E), A2 = pk2(A, A), B2 = pk2(B, B);
    uint4 q[U];
    load(q, i0);
    // The target has g (1 - p) in place of -g p. Where it is nearly sure, the difference keeps little: it is -expm1(d) there,
    // with a d that is right relative to itself. By the thread whose vector it is in. (64 x 1000 bf16 3.0 us, 2.8 without.)
    float of_target = g * inv_tau;
    bool sure = false;
    if (t >= 0) {
        const int after = t - rv.head, k = after < 0 ? rv.full : after < rv.full * N ? (int)((unsigned)after / N) : rv.full + 1;
        if (k >= part * per && k < end && (unsigned)(k - part * per) % NT == lane) {
            const float d = fmaf(-tau, L, to_f(x[t])) * inv_tau;
            sure = d > -0.5f;   // p above 0.6
            if (sure) of_target = ex2_approx(d * LOG2E) * fmaf(B, d, -h * H * inv_tau) - of_target * expm1f(d);
        }
    }
    for (int i = i0; i < end; i += U * NT) {
        uint4 next[U];
        load(next, i + U * NT);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = i + u * NT;
            if (k >= end) break;
            float r[N];
            unpack(q[u], r, T());
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const f32x2 d2 = fma2(pk2(r[j], r[j + 1]), it2, l2);
                float d0, d1, y0, y1;
                upk2(d2, d0, d1);
                upk2(mul2(d2, e2), y0, y1);
                // where p is 0 (d below -104, -inf where masked) its factor need only be finite
                const f32x2 f2 = fma2(B2, pk2(fmaxf(d0, -128.f), fmaxf(d1, -128.f)), A2);
                upk2(mul2(pk2(ex2_approx(y0), ex2_approx(y1)), f2), r[j], r[j + 1]);
            }
            const int at = t - rv.first(k);
            if ((unsigned)at < (unsigned)N && t < rv.last(k)) {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j == at) r[j] = sure ? of_target : r[j] + of_target;
            }
            if (k < rv.full) to[k] = pack(r, T());
            else scatter_vec(dx, rv, k, pack(r, T()));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = next[u];
    }
    griddep_launch();   // the next kernel's blocks may come: not earlier, they would crowd on the SMs with room
}

// NT threads a row.
template <typename T, int NT>
void launch_rows(const Ctx& ctx, const T* logits, long long ld, int rows, int V, float inv_tau, const int* targets,
                 const LogprobOut& out) {
    launch_pdl(ctx, token_logprobs_kernel<T, NT, false>, dim3(ceil_div(rows, BLOCK_OF<NT> / NT)), dim3(BLOCK_OF<NT>), 0,
               logits, ld, rows, V, inv_tau, targets, out, 1, ctx.status);
}

// A cluster of `parts` blocks of 128 threads a row.
template <typename T>
void launch_split(const Ctx& ctx, const T* logits, long long ld, int rows, int V, float inv_tau, const int* targets,
                  const LogprobOut& out, int parts) {
    launch_pdl_clusters(ctx, parts, token_logprobs_kernel<T, 128, true>, dim3(rows * parts), dim3(128), 0, logits, ld, rows,
                        V, inv_tau, targets, out, parts, ctx.status);
}

}  // namespace

template <typename T>
void launch_token_logprobs(const Ctx& ctx, const T* logits, long long ld, int rows, int V, float temperature,
                           const int* targets, const LogprobOut& out) {
    const float inv_tau = 1.f / temperature;
    // A warp a row where the row is short, and with many rows up to 8192: no block to wait for (8192 rows of 1024 bf16
    // logits 9.1 us against 18.4, of 8192 with five alternatives 38.5 against 41.7). For many alternatives, which a warp
    // takes longer to rank, only with many rows, of up to 16 KB (with 20: 20000 x 512 bf16 39 us against 90, 8192 x
    // 8192 54 against 63; but 8192 x 6000 fp32 61.6 against 56.8, 200 x 1500 7.0 against 5.6).
    const bool many = rows >= 8 * ctx.num_sms;
    const bool warp = out.top_k <= WALK ? V <= 2048 || (V <= 8192 && many) : many && V <= 16384 / (int)sizeof(T);
    // Few rows: as many blocks a row as give every SM two, while a thread still has a vector.
    int parts = 8;
    while (parts > 1 && ((long long)rows * parts > 2 * ctx.num_sms || V < parts * 128 * RowVecs<T>::N)) parts /= 2;
    // 256 threads for rows of 120 KB and more: with 128, the rows under way together are more than L2 holds, and what
    // is read again comes from memory (4096 x 131072 bf16, five alternatives: 179 us against 202; 4096 x 50257 fp32
    // 136 against 152; but 8192 x 16384 bf16 80 against 58).
    if (warp) launch_rows<T, 32>(ctx, logits, ld, rows, V, inv_tau, targets, out);
    else if (parts > 1) launch_split<T>(ctx, logits, ld, rows, V, inv_tau, targets, out, parts);
    else if (V >= 120000 / (int)sizeof(T)) launch_rows<T, 256>(ctx, logits, ld, rows, V, inv_tau, targets, out);
    else launch_rows<T, 128>(ctx, logits, ld, rows, V, inv_tau, targets, out);
    ++*ctx.launches;
}

template <typename T>
void launch_token_logprobs_bwd(const Ctx& ctx, const T* logits, long long ld, int rows, int V, float temperature,
                               const int* targets, const float* lse, const float* dlogp, const float* entropy,
                               const float* dentropy, T* dlogits, long long ldd) {
    // As few threads a row, 32 at least and 256 at most, as leave a thread four vectors or one round of loads. With 256
    // for every row 12149 x 2123 bf16 take 57 us instead of 29, 20000 x 1000 60 instead of 17, 64 x 1000 2.5 instead of 2.9;
    // with one row a block 100000 x 65 fp32 take 104 us instead of 44.5.
    const int vecs = V / RowVecs<T>::N + 2;
    auto launch = [&](auto threads) {
        constexpr int NT = decltype(threads)::value, ROWS = NT < 128 ? 128 / NT : 1;
        // sixteen vectors a thread; fewer, down to two, where that leaves an SM less than eight blocks
        int per = 16;
        while (per > 2 && (long long)rows * ceil_div(vecs, NT * per) < 8 * ctx.num_sms) per /= 2;
        const int parts = ceil_div(vecs, NT * per);
        launch_pdl(ctx, token_logprobs_bwd_kernel<T, NT>, dim3(ceil_div(rows, ROWS) * parts), dim3(NT * ROWS), 0, logits, ld,
                   rows, V, temperature, 1.f / temperature, targets, lse, dlogp, entropy, dentropy, dlogits, ldd, parts, ctx.status);
    };
    if (vecs <= 32 * 4) launch(std::integral_constant<int, 32>());
    else if (vecs <= 64 * 4) launch(std::integral_constant<int, 64>());
    else if (vecs <= 128 * 4) launch(std::integral_constant<int, 128>());
    else launch(std::integral_constant<int, 256>());
    ++*ctx.launches;
}

#define INSTANTIATE(T)                                                                                               \
    template void launch_token_logprobs<T>(const Ctx&, const T*, long long, int, int, float, const int*,             \
                                           const LogprobOut&);                                                       \
    template void launch_token_logprobs_bwd<T>(const Ctx&, const T*, long long, int, int, float, const int*,         \
                                               const float*, const float*, const float*, const float*, T*, long long);
INSTANTIATE(float)
INSTANTIATE(bf16)
#undef INSTANTIATE

}  // namespace gpt2
