// int8 x int8 products with a scale for each row of either operand:
//
//   out(m, n) = epilogue( (sum_k A(m, k) B(n, k)) sa[m] sb[n] )
//
// The sum is a 32-bit integer, exact for K <= 131071 (128^2 K < 2^31); it is
// rounded once to fp32 and multiplied by sa[m], then sb[n], in fp32.
#include "kernels.cuh"

namespace gpt2 {

namespace {

// One scaled sum through the epilogue. GELU in the tanh form for fp32 results
// and in the logistic form for bf16 ones (gelu_for).
template <int KIND, typename O>
__device__ __forceinline__ O finish(int acc, float sa, float sb, float bias, float resid) {
    float u = ((float)acc * sa) * sb;
    if (KIND != EPI_STORE) u += bias;
    if (KIND == EPI_BIAS_GELU) u = gelu_for<O>(u);
    if (KIND == EPI_BIAS_RESID) u += resid;
    return from_f<O>(u);
}

// ---------------------------------------------------------------- any strides
// 64 x 64 outputs per block of 256 threads (4 x 4 each), 64 bytes of K staged at a
// time as 32-bit words for dp4a. Rows may start at any byte: words are put together
// from single bytes.
constexpr int ST = 64, SKW = 16;

template <int KIND, typename O>
__global__ void __launch_bounds__(256) matmul_i8_simt_kernel(I8Product p) {
    __shared__ int as[SKW][ST + 1], bs[SKW][ST + 1];
    const int tiles_n = ceil_div(p.N, ST);
    const int m0 = (int)(blockIdx.x / tiles_n) * ST, n0 = (int)(blockIdx.x % tiles_n) * ST;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += 4 * SKW) {
        for (int i = threadIdx.x; i < SKW * ST; i += 256) {
            const int r = i / SKW, w = i % SKW;
            int a = 0, b = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = k0 + 4 * w + j;
                if (k < p.K) {
                    if (m0 + r < p.M) a |= (p.A[(long long)(m0 + r) * p.lda + k] & 0xff) << (8 * j);
                    if (n0 + r < p.N) b |= (p.B[(long long)(n0 + r) * p.ldb + k] & 0xff) << (8 * j);
                }
            }
            as[w][r] = a;
            bs[w][r] = b;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < SKW; ++w) {
            int a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = as[w][ty + 16 * i];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = bs[w][tx + 16 * j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty + 16 * i;
        if (m >= p.M) continue;
        const float sa = p.sa[m];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx + 16 * j;
            if (n >= p.N) continue;
            const float bias = KIND != EPI_STORE ? p.bias[n] : 0.f;
            const float resid = KIND == EPI_BIAS_RESID ? p.resid[(long long)m * p.ldr + n] : 0.f;
            reinterpret_cast<O*>(p.out)[(long long)m * p.ldo + n] =
                finish<KIND, O>(acc[i][j], sa, p.sb[n], bias, resid);
        }
    }
}

template <int KIND, typename O>
bool launch_kind(const Ctx& ctx, const I8Product& p) {
    const long long tiles = (long long)ceil_div(p.N, ST) * ceil_div(p.M, ST);
    matmul_i8_simt_kernel<KIND, O><<<(unsigned)tiles, 256, 0, ctx.stream>>>(p);
    ++*ctx.launches;
    return true;
}

}  // namespace

bool launch_matmul_i8(const Ctx& ctx, const I8Product& p) {
    switch (p.kind) {
    case EPI_STORE: return p.out_f32 ? launch_kind<EPI_STORE, float>(ctx, p) : launch_kind<EPI_STORE, bf16>(ctx, p);
    case EPI_BIAS: return p.out_f32 ? launch_kind<EPI_BIAS, float>(ctx, p) : launch_kind<EPI_BIAS, bf16>(ctx, p);
    case EPI_BIAS_GELU:
        return p.out_f32 ? launch_kind<EPI_BIAS_GELU, float>(ctx, p) : launch_kind<EPI_BIAS_GELU, bf16>(ctx, p);
    case EPI_BIAS_RESID: return launch_kind<EPI_BIAS_RESID, float>(ctx, p);
    default: return false;
    }
}

}  // namespace gpt2
