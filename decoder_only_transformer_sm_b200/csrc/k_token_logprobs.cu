// Log-probabilities of given tokens with entropy and top alternatives, and their
// gradient ("GPT-2 from Scratch", "A generation loop": the distribution a token is
// drawn from is softmax(logits / temperature)).
//
// With z = x / tau, m = max z, d = z - m, s = sum e^d, w = sum e^d d:
//   lse = m + log s,   log p_v = d_v - log s,   H = -sum p log p = log s - w / s.
// Masked logits are -inf: they add nothing to s and w. A row of which nothing is
// left (m = -inf) has lse = log p = -inf and H = 0; a row with NaN or +inf has NaN
// in all of them.
#include "kernels.cuh"

namespace gpt2 {

namespace {

constexpr float NEG_INF = -__builtin_huge_valf();

// 64-bit keys whose order is that of (value, then lowest index): the value's bits
// turned into an unsigned order (-0 as +0, NaN above everything), then ~index. No
// entry has the key 0 or all ones.
__device__ __forceinline__ unsigned long long order_key(float x, int v) {
    unsigned b = __float_as_uint(x + 0.f);
    b = (b & 0x80000000u) ? ~b : b | 0x80000000u;
    if (x != x) b = 0xffc00000u;   // above +inf, and no key is all ones
    return ((unsigned long long)b << 32) | (unsigned)~v;
}

template <typename T>
__global__ void __launch_bounds__(256) token_logprobs_kernel(const T* __restrict__ logits, long long ld, int V,
                                                             float inv_tau, const int* __restrict__ targets,
                                                             LogprobOut out, unsigned* status) {
    __shared__ float red[3][8];
    __shared__ unsigned long long best[8];
    const int row = blockIdx.x, tid = threadIdx.x;
    const T* x = logits + (long long)row * ld;
    float m = NEG_INF;
    bool nan = false;
    for (int v = tid; v < V; v += 256) {
        const float z = to_f(x[v]) * inv_tau;
        nan |= z != z;
        m = fmaxf(m, z);
    }
    m = warp_max(m);
    nan = __syncthreads_or(nan);
    if ((tid & 31) == 0) red[0][tid >> 5] = m;
    __syncthreads();
    for (int i = 0; i < 8; ++i) m = fmaxf(m, red[0][i]);
    const bool empty = m == NEG_INF && !nan, bad = nan || m == -NEG_INF;
    const float m0 = empty || bad ? 0.f : m;
    float s = 0.f, w = 0.f;
    for (int v = tid; v < V; v += 256) {
        const float d = to_f(x[v]) * inv_tau - m0;
        const float e = expf(d);
        s += e;
        if (e > 0.f) w += e * d;
    }
    s = warp_sum(s);
    w = warp_sum(w);
    if ((tid & 31) == 0) {
        red[1][tid >> 5] = s;
        red[2][tid >> 5] = w;
    }
    __syncthreads();
    s = w = 0.f;
    for (int i = 0; i < 8; ++i) {
        s += red[1][i];
        w += red[2][i];
    }
    const float log_s = logf(s);
    const float nanv = __uint_as_float(0x7fc00000u);
    auto settle = [&](float v, float nothing) { return bad ? nanv : empty ? nothing : v; };
    if (tid == 0) {
        if (out.lse) out.lse[row] = settle(m + log_s, NEG_INF);
        if (out.entropy) out.entropy[row] = settle(log_s - w / s, 0.f);
        if (out.logp) {
            int t = targets[row];
            if (t < -1 || t >= V) {
                atomicOr(status, STATUS_BAD_TOKEN);
                t = min(max(t, 0), V - 1);
            }
            out.logp[row] = t < 0 ? 0.f : settle(to_f(x[t]) * inv_tau - m0 - log_s, NEG_INF);
        }
    }
    unsigned long long below = ~0ull;
    for (int j = 0; j < out.top_k; ++j) {
        unsigned long long k = 0;
        for (int v = tid; v < V; v += 256) {
            const unsigned long long c = order_key(to_f(x[v]), v);
            if (c < below && c > k) k = c;
        }
        for (int o = 16; o; o >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
        __syncthreads();
        if ((tid & 31) == 0) best[tid >> 5] = k;
        __syncthreads();
        for (int i = 0; i < 8; ++i) k = max(k, best[i]);
        below = k;
        if (tid == 0) {
            const int v = (int)~(unsigned)k;
            out.top_ids[(long long)row * out.top_k + j] = v;
            out.top_logp[(long long)row * out.top_k + j] = settle(to_f(x[v]) * inv_tau - m0 - log_s, NEG_INF);
        }
    }
}

// dx_v = (1/tau) [ g (1[v = t] - p_v) - h p_v (log p_v + H) ], g = dlogp (0 at an ignored
// target), h = dentropy; p_v = e^(z_v - lse). Where p_v is 0 only the target's g is left.
template <typename T>
__global__ void __launch_bounds__(256) token_logprobs_bwd_kernel(const T* logits, long long ld, int V, float inv_tau,
                                                                 const int* __restrict__ targets,
                                                                 const float* __restrict__ lse,
                                                                 const float* __restrict__ dlogp,
                                                                 const float* __restrict__ entropy,
                                                                 const float* __restrict__ dentropy, T* dlogits,
                                                                 long long ldd, unsigned* status) {
    const int row = blockIdx.x;
    const T* x = logits + (long long)row * ld;
    T* dx = dlogits + (long long)row * ldd;
    int t = targets ? targets[row] : -1;
    if (t < -1 || t >= V) {
        if (threadIdx.x == 0) atomicOr(status, STATUS_BAD_TOKEN);
        t = min(max(t, 0), V - 1);
    }
    const float L = lse[row];
    const float g = dlogp && t >= 0 ? dlogp[row] : 0.f, h = dentropy ? dentropy[row] : 0.f;
    const float H = dentropy ? entropy[row] : 0.f;
    const bool none = (g == 0.f && h == 0.f) || L == NEG_INF;
    for (int v = threadIdx.x; v < V; v += 256) {
        float r = 0.f;
        if (!none) {
            const float d = fmaf(to_f(x[v]), inv_tau, -L);
            const float p = expf(d);
            if (!(p == 0.f)) r = -p * (g + h * (d + H));
            if (v == t) r += g;
        }
        dx[v] = from_f<T>(r * inv_tau);
    }
}

}  // namespace

template <typename T>
void launch_token_logprobs(const Ctx& ctx, const T* logits, long long ld, int rows, int V, float temperature,
                           const int* targets, const LogprobOut& out) {
    token_logprobs_kernel<T><<<rows, 256, 0, ctx.stream>>>(logits, ld, V, 1.f / temperature, targets, out, ctx.status);
    ++*ctx.launches;
}

template <typename T>
void launch_token_logprobs_bwd(const Ctx& ctx, const T* logits, long long ld, int rows, int V, float temperature,
                               const int* targets, const float* lse, const float* dlogp, const float* entropy,
                               const float* dentropy, T* dlogits, long long ldd) {
    token_logprobs_bwd_kernel<T><<<rows, 256, 0, ctx.stream>>>(logits, ld, V, 1.f / temperature, targets, lse, dlogp,
                                                               entropy, dentropy, dlogits, ldd, ctx.status);
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
