// Symmetric 8-bit quantisation of rows: the operands of the int8 products
// (k_matmul_i8.cu), activations by token and weights by output channel.
//
//   a = max_k |x_k|,  scale = fl32(a / 127),  q_k = rne(127 x_k / a)
//
// q is the nearest whole number (ties to even) of the exact quotient, so the
// codes do not depend on how the quotient is rounded: t = x * fl32(127 / a)
// is within 2 * 2^-24 * 127 < 1.6e-5 of it, so its nearest whole number n is q or,
// close to a border between two codes, q's neighbour, and e = 127 x - n a, compared
// with a / 2, decides which. For bf16 x (8 bits) e is exact in fp32, and every vector is
// checked by it: ties are common there (127 x / a with two 8-bit significands). For fp32 x
// only a t closer than 1.7e-5 to a border is, with e as a sum of two fp32 numbers:
// 127 x and n a each as a product and its rounding error (fma), whose differences are exact
// that close to each other. 127 and a carry a power of two that keeps 127 x finite; rows
// whose largest value is below 1e-30, where 127 / a could overflow, take the 64-bit quotient
// (127 x is exact, and a quotient that is not a border differs from one by more than 2^-41
// relative, so rounding the division cannot make a tie).
//
// Bound by memory: a row is read once, as 16-byte vectors that stay in registers
// (up to 8 a thread, 8 to 256 threads a row) between the maximum and the codes. Rows may start at
// any element and codes at any byte: the elements before a row's first 16-byte boundary
// and after its last one are held one a thread, and the codes go through shared memory,
// laid out there like the memory they go to, so that they leave in 16-byte stores too. Where
// rows and codes are whole vectors (ALIGNED) none of that is needed: the codes go straight out.
// 50257 x 1024 fp32 38 us (6.8 TB/s), 4096 x 6400 bf16 13.4 us (5.9 TB/s), 16384 x 1599 bf16 21.3 us, 16384 x 1600 14.2 (from
// a CUDA graph on the same buffers). Rows that do not fit in registers (past 8192 fp32 or 16384 bf16 values) are read twice,
// value by value: 4096 x 8200 fp32 45.7 us, 4096 x 8192 25.7; 2048 x 16400 bf16 50.3, 2048 x 16384 17.4.
#include "kernels.cuh"

namespace gpt2 {

namespace {

// t + MAGIC has the nearest whole number of t (ties to even, |t| < 2^22) in its low bits.
constexpr float MAGIC = 12582912.f;   // 3 * 2^22
constexpr float BORDER = 0.5f - 1.7e-5f;

// What a row's codes are made with.
struct Step {
    float a, inv;     // largest magnitude; 127 / a, or 0 where a is too small (or no number)
    float c, as;      // 127 and a times the power of two
    __device__ __forceinline__ explicit Step(float a_) : a(a_) {
        inv = a > 1e-30f ? 127.f / a : 0.f;
        const float s = a > 1e30f ? 0.00390625f : 1.f;
        c = 127.f * s;
        as = a * s;
    }
};

// n (in the low bits of `code`) moved to its neighbour if e = 127 x - n a says so: d = |e| - a / 2.
__device__ __forceinline__ void decide(unsigned& code, float e, float d) {
    if (d > 0.f || (d == 0.f && (code & 1u))) code += e > 0.f ? 1u : ~0u;
}

// Codes of N values as N bytes (inv is not 0).
__device__ __forceinline__ void codes(const float (&x)[8], const Step& st, unsigned (&out)[2], bf16) {
    unsigned c[8];
    float e[8], far = 0.f;
    const f32x2 i2 = pk2(st.inv, st.inv), up = pk2(MAGIC, MAGIC), down = pk2(MAGIC, MAGIC), a2 = pk2(st.as, st.as),
                c2 = pk2(st.c, st.c), minus = pk2(-1.f, -1.f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const f32x2 v = pk2(x[j], x[j + 1]);
        const f32x2 n = add2(mul2(v, i2), up);
        float n0, n1;
        upk2(n, n0, n1);
        upk2(fma2(fma2(n, minus, down), a2, mul2(v, c2)), e[j], e[j + 1]);   // -n a + 127 x
        far = fmaxf(far, fmaxf(fabsf(e[j]), fabsf(e[j + 1])));
        c[j] = __float_as_uint(n0);
        c[j + 1] = __float_as_uint(n1);
    }
    const float half = 0.5f * st.as;
    if (far >= half) {
#pragma unroll
        for (int j = 0; j < 8; ++j) decide(c[j], e[j], fabsf(e[j]) - half);
    }
#pragma unroll
    for (int j = 0; j < 8; j += 4)
        out[j / 4] = __byte_perm(__byte_perm(c[j], c[j + 1], 0x0040), __byte_perm(c[j + 2], c[j + 3], 0x0040), 0x5410);
}
__device__ __forceinline__ void codes(const float (&x)[4], const Step& st, unsigned (&out)[1], float) {
    unsigned c[4];
    float n[4], far = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float t = x[j] * st.inv, m = t + MAGIC;
        n[j] = m - MAGIC;
        far = fmaxf(far, fabsf(t - n[j]));
        c[j] = __float_as_uint(m);
    }
    if (far > BORDER) {
        const float half = 0.5f * st.as;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = x[j] * st.c, q = n[j] * st.as, e = p - q;
            const float low = fmaf(x[j], st.c, -p) - fmaf(n[j], st.as, -q);
            // e is within a rounding error of 127 x - n a, `low` is what it lacks
            decide(c[j], e, (fabsf(e) - half) + (e > 0.f ? low : -low));
        }
    }
    out[0] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}
// The code of one value, decided where it has to be by the 64-bit quotient (inv = 0: always).
__device__ __noinline__ unsigned code(float x, float a, float inv) {
    const float t = x * inv, n = t + MAGIC;
    if (fabsf(t - (n - MAGIC)) > BORDER || inv == 0.f)
        return a > 0.f ? (unsigned)(int)rint(127.0 * (double)x / (double)a) & 0xffu : 0u;
    return __float_as_uint(n) & 0xffu;
}
// A row whose inv is 0, value by value (read again, so that the pass over the others need not keep it).
template <int N, int G, typename T>
__device__ __forceinline__ void slow_codes(const T* x, int8_t* out, int t, int full, const Step& st) {
    for (int i = t; i < full; i += G) {
#pragma unroll 1
        for (int j = 0; j < N; ++j) out[i * N + j] = (int8_t)code(to_f(x[i * N + j]), st.a, st.inv);
    }
}

// The bits of |x| order like its value, with inf and NaN above every finite one.
__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Rows of any length: a block a row, read twice.
template <typename T>
__global__ void __launch_bounds__(256) quantize_long_rows_kernel(const T* __restrict__ x, long long ldx, int K,
                                                                 int8_t* __restrict__ q, long long ldq,
                                                                 float* __restrict__ scale) {
    __shared__ unsigned part[8];
    griddep_wait();     // nothing is read or written before the kernel before this one has ended
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
    griddep_launch();   // the next kernel's blocks may come: not earlier, they would crowd on the SMs with room
    const bool fine = m < 0x7f800000u;
    if (threadIdx.x == 0) scale[blockIdx.x] = fine ? __uint_as_float(m) / 127.f : __uint_as_float(0x7fc00000u);
    const Step st(fine ? __uint_as_float(m) : 0.f);
    for (int k = threadIdx.x; k < K; k += 256) qr[k] = (int8_t)code(to_f(xr[k]), st.a, st.inv);
}

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
// Largest magnitude of a vector, NaN above all: two at a time for bf16 (`m` in both halves).
__device__ __forceinline__ unsigned larger(unsigned m, const uint4& q, bf16) {
    const unsigned u[4] = {q.x, q.y, q.z, q.w};
    __nv_bfloat162 r = *reinterpret_cast<const __nv_bfloat162*>(&m);
#pragma unroll
    for (int i = 0; i < 4; ++i) r = __hmax2_nan(r, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[i])));
    return *reinterpret_cast<const unsigned*>(&r);
}
__device__ __forceinline__ unsigned larger(unsigned m, const uint4& q, float) {
    constexpr unsigned K1 = 0x7fffffffu;
    return max(max(m, max(q.x & K1, q.y & K1)), max(q.z & K1, q.w & K1));
}
__device__ __forceinline__ unsigned whole(unsigned m, bf16) { return max(m << 16, m & 0xffff0000u); }
__device__ __forceinline__ unsigned whole(unsigned m, float) { return m; }

constexpr int QV = 8;   // vectors a thread

// G threads a row, QT a block.
template <typename T, int G, int QT, bool ALIGNED>
__global__ void __launch_bounds__(QT, 1024 / QT) quantize_rows_kernel(const T* __restrict__ x, long long ldx, int rows, int K,
                                                           int8_t* __restrict__ q, long long ldq,
                                                           float* __restrict__ scale) {
    constexpr int N = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t staged[];   // QT / G rows of room_of(K) bytes
    __shared__ unsigned part[QT / 32];
    griddep_wait();     // nothing is read or written before the kernel before this one has ended
    const int t = threadIdx.x % G, in_block = threadIdx.x / G;
    const long long row = (long long)blockIdx.x * (QT / G) + in_block;
    const bool live = row < rows;
    const T* xr = x + (live ? row : 0) * ldx;
    int8_t* qr = q + (live ? row : 0) * ldq;
    const int head = ALIGNED ? 0 : min(K, (int)((16 - ((uintptr_t)xr & 15)) & 15) / (int)sizeof(T));
    const int full = (K - head) / N, tail = ALIGNED ? 0 : K - head - full * N;
    // this thread's vectors, and its element of the head and of the tail
    uint4 v[QV];
    float h = 0.f, e = 0.f;
    unsigned m = 0;
    if (live) {
#pragma unroll
        for (int i = 0; i < QV; ++i)
            v[i] = t + i * G < full ? __ldg(reinterpret_cast<const uint4*>(xr + head) + t + i * G) : make_uint4(0, 0, 0, 0);
        if (!ALIGNED && t < head) h = to_f(xr[t]);
        if (!ALIGNED && t < tail) e = to_f(xr[K - tail + t]);
#pragma unroll
        for (int i = 0; i < QV; ++i) m = larger(m, v[i], T());
        m = max(whole(m, T()), max(magnitude(h), magnitude(e)));
    }
    if (G < 32) {
#pragma unroll
        for (int o = G / 2; o; o /= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    } else {
        m = __reduce_max_sync(0xffffffffu, m);
    }
    if (G > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
        m = part[in_block * (G / 32)];
#pragma unroll
        for (int w = 1; w < G / 32; ++w) m = max(m, part[in_block * (G / 32) + w]);
    }
    griddep_launch();   // the next kernel's blocks may come: not earlier, they would crowd on the SMs with room
    const bool fine = m < 0x7f800000u;
    if (live && t == 0) scale[row] = fine ? __uint_as_float(m) / 127.f : __uint_as_float(0x7fc00000u);
    const Step st(fine ? __uint_as_float(m) : 0.f);
    if (ALIGNED) {
        if (!live) return;
        if (st.inv == 0.f) {
            slow_codes<N, G>(xr, qr, t, full, st);
            return;
        }
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            if (t + i * G < full) {
                float f[N];
                unsigned c[N / 4];
                unpack(v[i], f, T());
                codes(f, st, c, T());
                if (N == 8) *reinterpret_cast<uint2*>(qr + (t + i * G) * N) = make_uint2(c[0], c[N / 4 - 1]);
                else *reinterpret_cast<unsigned*>(qr + (t + i * G) * N) = c[0];
            }
        }
        return;
    }
    const int lead = (int)((uintptr_t)qr & 15);
    int8_t* room = reinterpret_cast<int8_t*>(staged) + in_block * ((K + 15 + 16 + 15) / 16 * 16) + lead;
    if (live) {
        if (t < head) room[t] = (int8_t)code(h, st.a, st.inv);
        if (t < tail) room[K - tail + t] = (int8_t)code(e, st.a, st.inv);
        const bool words = ((lead + head) & 3) == 0;
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            if (t + i * G < full) {
                float f[N];
                unsigned c[N / 4];
                unpack(v[i], f, T());
                codes(f, st, c, T());
                int8_t* at = room + head + (t + i * G) * N;
#pragma unroll
                for (int j = 0; j < N / 4; ++j) {
                    if (words) {
                        reinterpret_cast<unsigned*>(at)[j] = c[j];
                    } else {
#pragma unroll
                        for (int b = 0; b < 4; ++b) at[4 * j + b] = (int8_t)(c[j] >> (8 * b));
                    }
                }
            }
        }
        if (st.inv == 0.f) slow_codes<N, G>(xr + head, room + head, t, full, st);
    }
    if (G > 32) __syncthreads();
    else __syncwarp();
    if (live) {
        // whole 16-byte segments of the memory the codes go to, single bytes at its ends
        const int first = (16 - lead) & 15, last = max(first, K - ((lead + K) & 15));
        for (int k = first + 16 * t; k + 16 <= last; k += 16 * G)
            *reinterpret_cast<uint4*>(qr + k) = *reinterpret_cast<const uint4*>(room + k);
        for (int k = t; k < min(first, K); k += G) qr[k] = room[k];
        for (int k = last + t; k < K; k += G) qr[k] = room[k];
    }
}

template <typename T, int G, int QT = (G > 128 ? G : 128)>
void launch_short(const Ctx& ctx, const T* x, long long ldx, int rows, int K, int8_t* q, long long ldq, float* scale) {
    constexpr int N = 16 / sizeof(T);
    const long long strides = rows > 1 ? ldx | ldq : 0;   // one row has none (1 x 6400 bf16: 2.7 us as unaligned, 2.0)
    const bool aligned = ((uintptr_t)x & 15) == 0 && ((uintptr_t)q & (N - 1)) == 0 && (strides | K) % N == 0;
    const int grid = ceil_div(rows, QT / G);
    if (aligned)
        launch_pdl(ctx, quantize_rows_kernel<T, G, QT, true>, dim3(grid), dim3(QT), 0, x, ldx, rows, K, q, ldq, scale);
    else
        launch_pdl(ctx, quantize_rows_kernel<T, G, QT, false>, dim3(grid), dim3(QT),
                   (size_t)(QT / G) * ((K + 15 + 16 + 15) / 16 * 16), x, ldx, rows, K, q, ldq, scale);
}

}  // namespace

template <typename T>
void launch_quantize_rows(const Ctx& ctx, const T* x, long long ldx, int rows, int K, int8_t* q, long long ldq,
                          float* scale) {
    // the fewest threads a row that hold it in registers
    const int vecs = K / (16 / (int)sizeof(T));
    if (vecs <= 32)   // eight: four rows a warp
        launch_short<T, 8>(ctx, x, ldx, rows, K, q, ldq, scale);
    else if (vecs <= 32 * QV)
        launch_short<T, 32>(ctx, x, ldx, rows, K, q, ldq, scale);
    else if (vecs <= 128 * QV)
        launch_short<T, 128>(ctx, x, ldx, rows, K, q, ldq, scale);
    else if (vecs <= 256 * QV)
        launch_short<T, 256>(ctx, x, ldx, rows, K, q, ldq, scale);
    else
        launch_pdl(ctx, quantize_long_rows_kernel<T>, dim3(rows), dim3(256), 0, x, ldx, K, q, ldq, scale);
    ++*ctx.launches;
}

template void launch_quantize_rows<float>(const Ctx&, const float*, long long, int, int, int8_t*, long long, float*);
template void launch_quantize_rows<bf16>(const Ctx&, const bf16*, long long, int, int, int8_t*, long long, float*);

}  // namespace gpt2
