// Symmetric 8-bit quantisation of rows: the operands of the int8 products
// (k_matmul_i8.cu), activations by token and weights by output channel.
//
//   a = max_k |x_k|,  scale = fl32(a / 127),  q_k = rne(127 x_k / a)
//
// q is the nearest whole number (ties to even) of the exact quotient, so the
// codes do not depend on how the quotient is rounded: t = x * fl32(127 / a)
// is within 3 * 2^-24 * 127 < 2.3e-5 of it, and only a t closer than 3e-5 to the
// border between two codes is decided by a 64-bit division (there 127 x is
// exact, and a quotient that is not a border differs from one by more than
// 2^-41 relative, so rounding the division cannot make a tie).
//
// Bound by memory: a row is read once, as 16-byte vectors that stay in registers
// (up to 8 a thread) between the maximum and the codes. Rows may start at
// any element and codes at any byte: the elements before a row's first 16-byte boundary
// and after its last one are held one a thread, and the codes go through shared memory,
// laid out there like the memory they go to, so that they leave in 16-byte stores too.
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

// The bits of |x| order like its value, with inf and NaN above every finite one.
__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Rows of any length: a block a row, read twice.
template <typename T>
__global__ void __launch_bounds__(256) quantize_long_rows_kernel(const T* __restrict__ x, long long ldx, int K,
                                                                 int8_t* __restrict__ q, long long ldq,
                                                                 float* __restrict__ scale) {
    __shared__ unsigned part[8];
    const T* xr = x + (long long)blockIdx.x * ldx;
    int8_t* qr = q + (long long)blockIdx.x * ldq;
    unsigned m = 0;
    for (int k = threadIdx.x; k < K; k += 256) m = max(m, magnitude(to_f(xr[k])));
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

__device__ __forceinline__ float element(const uint4& q, int j, float) {
    return __uint_as_float(j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w);
}
__device__ __forceinline__ float element(const uint4& q, int j, bf16) {
    const unsigned w = j < 2 ? q.x : j < 4 ? q.y : j < 6 ? q.z : q.w;
    return __uint_as_float((j & 1) ? w & 0xffff0000u : w << 16);
}

constexpr int QT = 256, QV = 8;   // threads a block, vectors a thread

// G threads a row, QT / G rows a block.
template <typename T, int G>
__global__ void __launch_bounds__(QT) quantize_rows_kernel(const T* __restrict__ x, long long ldx, int rows, int K,
                                                           int8_t* __restrict__ q, long long ldq,
                                                           float* __restrict__ scale) {
    constexpr int N = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t staged[];   // QT / G rows of room_of(K) bytes
    __shared__ unsigned part[QT / 32];
    const int t = threadIdx.x % G, in_block = threadIdx.x / G;
    const long long row = (long long)blockIdx.x * (QT / G) + in_block;
    const bool live = row < rows;
    const T* xr = x + (live ? row : 0) * ldx;
    int8_t* qr = q + (live ? row : 0) * ldq;
    const int head = min(K, (int)((16 - ((uintptr_t)xr & 15)) & 15) / (int)sizeof(T));
    const int full = (K - head) / N, tail = K - head - full * N;
    // this thread's vectors, and its element of the head and of the tail
    uint4 v[QV];
    float h = 0.f, e = 0.f;
    unsigned m = 0;
    if (live) {
#pragma unroll
        for (int i = 0; i < QV; ++i)
            v[i] = t + i * G < full ? __ldg(reinterpret_cast<const uint4*>(xr + head) + t + i * G) : make_uint4(0, 0, 0, 0);
        if (t < head) h = to_f(xr[t]);
        if (t < tail) e = to_f(xr[K - tail + t]);
        m = max(magnitude(h), magnitude(e));
#pragma unroll
        for (int i = 0; i < QV; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) m = max(m, magnitude(element(v[i], j, T())));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (G > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
        m = part[in_block * (G / 32)];
#pragma unroll
        for (int w = 1; w < G / 32; ++w) m = max(m, part[in_block * (G / 32) + w]);
    }
    const bool fine = m < 0x7f800000u;
    if (live && t == 0) scale[row] = fine ? __uint_as_float(m) / 127.f : __uint_as_float(0x7fc00000u);
    const RowScale r = row_scale(fine && m ? m : 0x3f800000u);
    const bool zero = !fine;   // (a row of zeros has codes 0 by any scale)
    const int lead = (int)((uintptr_t)qr & 15);
    int8_t* room = reinterpret_cast<int8_t*>(staged) + in_block * ((K + 15 + 16 + 15) / 16 * 16) + lead;
    if (live) {
        if (t < head) room[t] = zero ? 0 : code(h, r);
        if (t < tail) room[K - tail + t] = zero ? 0 : code(e, r);
        const bool words = ((lead + head) & 3) == 0;
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            if (t + i * G < full) {
                int c[N];
#pragma unroll
                for (int j = 0; j < N; ++j) c[j] = zero ? 0 : code(element(v[i], j, T()), r);
                int8_t* at = room + head + (t + i * G) * N;
                if (words) {
#pragma unroll
                    for (int j = 0; j < N; j += 4)
                        *reinterpret_cast<unsigned*>(at + j) = (c[j] & 0xff) | (c[j + 1] & 0xff) << 8 |
                                                               (c[j + 2] & 0xff) << 16 | (unsigned)c[j + 3] << 24;
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) at[j] = (int8_t)c[j];
                }
            }
        }
    }
    if (G > 32) __syncthreads();
    else __syncwarp();
    if (live) {
        // whole 16-byte segments of the memory the codes go to, single bytes at its ends
        const int first = (16 - lead) & 15, last = max(first, K - ((lead + K) & 15));
        for (int k = first + 16 * t; k + 16 <= last; k += 16 * G)
            *reinterpret_cast<uint4*>(qr + k) = *reinterpret_cast<const uint4*>(room + k);
        if (t < min(first, K)) qr[t] = room[t];
        if (t < K - last) qr[last + t] = room[last + t];
    }
}

template <typename T, int G>
void launch_short(const Ctx& ctx, const T* x, long long ldx, int rows, int K, int8_t* q, long long ldq, float* scale) {
    const size_t room = (size_t)(QT / G) * ((K + 15 + 16 + 15) / 16 * 16);
    quantize_rows_kernel<T, G><<<ceil_div(rows, QT / G), QT, room, ctx.stream>>>(x, ldx, rows, K, q, ldq, scale);
}

}  // namespace

template <typename T>
void launch_quantize_rows(const Ctx& ctx, const T* x, long long ldx, int rows, int K, int8_t* q, long long ldq,
                          float* scale) {
    // the fewest threads a row that hold it in registers
    const int vecs = K / (16 / (int)sizeof(T));
    if (vecs <= 32 * QV)
        launch_short<T, 32>(ctx, x, ldx, rows, K, q, ldq, scale);
    else if (vecs <= 128 * QV)
        launch_short<T, 128>(ctx, x, ldx, rows, K, q, ldq, scale);
    else if (vecs <= 256 * QV)
        launch_short<T, 256>(ctx, x, ldx, rows, K, q, ldq, scale);
    else
        quantize_long_rows_kernel<T><<<rows, 256, 0, ctx.stream>>>(x, ldx, K, q, ldq, scale);
    ++*ctx.launches;
}

template void launch_quantize_rows<float>(const Ctx&, const float*, long long, int, int, int8_t*, long long, float*);
template void launch_quantize_rows<bf16>(const Ctx&, const bf16*, long long, int, int, int8_t*, long long, float*);

}  // namespace gpt2
