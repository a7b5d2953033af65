// Symmetric 8-bit quantisation of rows: the operands of the int8 products
// (k_matmul_i8.cu), activations by token and weights by output channel.
//
//   a = max_k |x_k|,  scale = fl32(a / 127),  q_k = rne(127 x_k / a)
//
// q is the nearest whole number (ties to even) of the exact quotient, so the
// codes do not depend on how the quotient is rounded: t = x * fl32(127 / a)
// is within 2^-23 * 127 < 1.6e-5 of it, and only a t closer than 3e-5 to the
// border between two codes is decided by a 64-bit division (there 127 x is
// exact, and a quotient that is not a border differs from one by more than
// 2^-41 relative, so rounding the division cannot make a tie).
#include "kernels.cuh"

namespace gpt2 {

namespace {

struct RowScale {
    float a;      // max |x|
    float pre;    // power of two that keeps 127 / (a pre) finite
    float inv;    // 127 / (a pre)
};

__device__ __forceinline__ RowScale row_scale(unsigned amax_bits) {
    RowScale r;
    r.a = __uint_as_float(amax_bits);
    r.pre = r.a < 1e-30f ? 1.2676506e30f : 1.f;   // 2^100
    r.inv = 127.f / (r.a * r.pre);
    return r;
}

__device__ __noinline__ int code_at_border(float x, float a) { return (int)rint(127.0 * (double)x / (double)a); }

__device__ __forceinline__ int code(float x, const RowScale& r) {
    const float t = (x * r.pre) * r.inv;
    const float n = rintf(t);
    if (fabsf(fabsf(t - n) - 0.5f) < 3e-5f) return code_at_border(x, r.a);
    return (int)n;
}

template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T* __restrict__ x, long long ldx, int K,
                                                            int8_t* __restrict__ q, long long ldq,
                                                            float* __restrict__ scale) {
    __shared__ unsigned part[8];
    const T* xr = x + (long long)blockIdx.x * ldx;
    int8_t* qr = q + (long long)blockIdx.x * ldq;
    // the bits of |x| order like its value, with inf and NaN above every finite one
    unsigned m = 0;
    for (int k = threadIdx.x; k < K; k += 256) m = max(m, __float_as_uint(to_f(xr[k])) & 0x7fffffffu);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = part[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = max(m, part[w]);
    const bool fine = m < 0x7f800000u;
    if (threadIdx.x == 0) scale[blockIdx.x] = fine ? __uint_as_float(m) / 127.f : __uint_as_float(0x7fc00000u);
    const RowScale r = row_scale(m);
    for (int k = threadIdx.x; k < K; k += 256) qr[k] = fine && m ? (int8_t)code(to_f(xr[k]), r) : (int8_t)0;
}

}  // namespace

template <typename T>
void launch_quantize_rows(const Ctx& ctx, const T* x, long long ldx, int rows, int K, int8_t* q, long long ldq,
                          float* scale) {
    quantize_rows_kernel<T><<<rows, 256, 0, ctx.stream>>>(x, ldx, K, q, ldq, scale);
    ++*ctx.launches;
}

template void launch_quantize_rows<float>(const Ctx&, const float*, long long, int, int, int8_t*, long long, float*);
template void launch_quantize_rows<bf16>(const Ctx&, const bf16*, long long, int, int, int8_t*, long long, float*);

}  // namespace gpt2
