// int8 products of a few rows (M <= 8; k_matmul_i8.cu has the others and what they compute):
// weight streaming. Each warp takes RG rows of B at a time, a lane 16
// bytes of each per step (two steps in flight); the matching bytes of the M rows of A come from
// L1. Lane r * MM + m finishes element (m, n0 + r); its scales are requested first, so that a
// warp's life is about one trip to memory.
//
// lm_head of one token (50304 x 768, from a CUDA graph): 6.6 us with the weights in L2, 7.3 us from memory (5.3 TB/s),
// of which about 2 us are the launch and the first load; 2 rows 6.9 and 11 us, 8 rows 13.2 and 17.6 us, where the loads
// of the rows of A from L1 are as many as those of B.
#include "kernels.cuh"

namespace gpt2 {

namespace {

constexpr int GV_THREADS = 128;

// One scaled sum through the epilogue. GELU in the tanh form for fp32 results and in the
// logistic form for bf16 ones (gelu_for).
template <int KIND, typename O>
__device__ __forceinline__ O finish(int acc, float sa, float sb, float bias, float resid) {
    float u = ((float)acc * sa) * sb;
    if (KIND != EPI_STORE) u += bias;
    if (KIND == EPI_BIAS_GELU) u = gelu_for<O>(u);
    if (KIND == EPI_BIAS_RESID) u += resid;
    return from_f<O>(u);
}

// The last bytes of a row, K % 16 of them, and zeros: what follows a row belongs to nobody.
__device__ __forceinline__ int4 load_tail(const int8_t* row, int K) {
    int w[4] = {0, 0, 0, 0};
    for (int i = 0; i < (K & 15); ++i) w[i >> 2] |= (row[(K & ~15) + i] & 0xff) << (8 * (i & 3));
    return make_int4(w[0], w[1], w[2], w[3]);
}
// 16 bytes at any address, from aligned 32-bit words; the first and the last bytes of the operand
// (lo .. hi), where a word would touch others, from single ones.
__device__ __forceinline__ int4 load_any(const int8_t* at, const int8_t* lo, const int8_t* hi) {
    const int off = (int)((uintptr_t)at & 3);
    const unsigned* word = reinterpret_cast<const unsigned*>(at - off);
    unsigned w[4] = {0, 0, 0, 0};
    if (at - off >= lo && at - off + 20 <= hi) {
        unsigned u[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = __ldg(word + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(u[i], u[i + 1], 8 * off);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i >> 2] |= (unsigned)(uint8_t)at[i] << (8 * (i & 3));
    }
    return make_int4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ int dot16(int4 a, int4 b, int acc) {
    return __dp4a(a.w, b.w, __dp4a(a.z, b.z, __dp4a(a.y, b.y, __dp4a(a.x, b.x, acc))));
}

template <int KIND, typename O, int MM, int RG, bool BYTES>
__global__ void __launch_bounds__(GV_THREADS) matmul_i8_rows_kernel(I8Product p) {
    const int lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * (GV_THREADS / 32) + (threadIdx.x >> 5)) * RG;
    griddep_wait();     // nothing is read or written before the kernel before this one has ended
    if (n0 >= p.N) return;
    const int chunks = p.K / 16;
    const int8_t* b[RG];
#pragma unroll
    for (int r = 0; r < RG; ++r) b[r] = p.B + (long long)min(n0 + r, p.N - 1) * p.ldb;
    const int8_t* a[MM];
#pragma unroll
    for (int m = 0; m < MM; ++m) a[m] = p.A + (long long)min(m, p.M - 1) * p.lda;
    const int8_t* b_end = p.B + (long long)(p.N - 1) * p.ldb + p.K;
    const int8_t* a_end = p.A + (long long)(p.M - 1) * p.lda + p.K;
    auto load = [&](const int8_t* row, int j, const int8_t* lo, const int8_t* hi) {   // its j-th 16 bytes
        if (j >= chunks) return make_int4(0, 0, 0, 0);
        return BYTES ? load_any(row + 16 * j, lo, hi) : __ldg(reinterpret_cast<const int4*>(row) + j);
    };
    const int my_m = lane % MM, my_n = n0 + lane / MM;
    const bool mine = lane < RG * MM && my_m < p.M && my_n < p.N;
    float sa = 0.f, sb = 0.f, bias = 0.f, resid = 0.f;
    int acc[RG][MM] = {};
    for (int j0 = lane; j0 < chunks; j0 += 64) {
        int4 w[2][RG];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < RG; ++r)
                w[u][r] = load(b[r], j0 + 32 * u, p.B, b_end);
        if (j0 == lane && mine) {
            sa = __ldg(p.sa + my_m);
            sb = __ldg(p.sb + my_n);
            if (KIND != EPI_STORE) bias = __ldg(p.bias + my_n);
            if (KIND == EPI_BIAS_RESID) resid = p.resid[(long long)my_m * p.ldr + my_n];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            int4 x[MM];
#pragma unroll
            for (int m = 0; m < MM; ++m) x[m] = load(a[m], j0 + 32 * u, p.A, a_end);
#pragma unroll
            for (int m = 0; m < MM; ++m)
#pragma unroll
                for (int r = 0; r < RG; ++r) acc[r][m] = dot16(x[m], w[u][r], acc[r][m]);
        }
    }
    griddep_launch();   // the next kernel's blocks may come: not earlier, they would crowd on the SMs with room
    if (lane >= chunks && mine) {   // a lane that the loop above passed by
        sa = __ldg(p.sa + my_m);
        sb = __ldg(p.sb + my_n);
        if (KIND != EPI_STORE) bias = __ldg(p.bias + my_n);
        if (KIND == EPI_BIAS_RESID) resid = p.resid[(long long)my_m * p.ldr + my_n];
    }
    if ((p.K & 15) && lane == 0) {
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            const int4 w = load_tail(b[r], p.K);
#pragma unroll
            for (int m = 0; m < MM; ++m)
                acc[r][m] = dot16(load_tail(a[m], p.K), w, acc[r][m]);
        }
    }
    int sum = 0;
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int m = 0; m < MM; ++m) {
            const int t = __reduce_add_sync(0xffffffffu, acc[r][m]);
            if (lane == r * MM + m) sum = t;
        }
    if (mine) reinterpret_cast<O*>(p.out)[(long long)my_m * p.ldo + my_n] = finish<KIND, O>(sum, sa, sb, bias, resid);
}

template <int KIND, typename O, int MM>
void launch_rows(const Ctx& ctx, const I8Product& p, bool whole) {
    // four rows a warp once that leaves every SM eight warps, else one; one where they are put together from words
    constexpr int W = GV_THREADS / 32;
    const dim3 four(ceil_div(p.N, 4 * W)), one(ceil_div(p.N, W)), block(GV_THREADS);
    if (!whole) launch_pdl(ctx, matmul_i8_rows_kernel<KIND, O, MM, 1, true>, one, block, 0, p);
    else if (p.N >= 4 * 8 * ctx.num_sms) launch_pdl(ctx, matmul_i8_rows_kernel<KIND, O, MM, 4, false>, four, block, 0, p);
    else launch_pdl(ctx, matmul_i8_rows_kernel<KIND, O, MM, 1, false>, one, block, 0, p);
}

template <int KIND, typename O>
void launch_kind(const Ctx& ctx, const I8Product& p, bool whole) {
    if (p.M == 1) launch_rows<KIND, O, 1>(ctx, p, whole);
    else if (p.M == 2) launch_rows<KIND, O, 2>(ctx, p, whole);
    else if (p.M <= 4) launch_rows<KIND, O, 4>(ctx, p, whole);
    else launch_rows<KIND, O, I8_FEW_ROWS>(ctx, p, whole);
}

}  // namespace

void launch_matmul_i8_rows(const Ctx& ctx, const I8Product& p, bool whole) {
    switch (p.kind) {
    case EPI_STORE:
        return p.out_f32 ? launch_kind<EPI_STORE, float>(ctx, p, whole) : launch_kind<EPI_STORE, bf16>(ctx, p, whole);
    case EPI_BIAS:
        return p.out_f32 ? launch_kind<EPI_BIAS, float>(ctx, p, whole) : launch_kind<EPI_BIAS, bf16>(ctx, p, whole);
    case EPI_BIAS_GELU:
        return p.out_f32 ? launch_kind<EPI_BIAS_GELU, float>(ctx, p, whole)
                         : launch_kind<EPI_BIAS_GELU, bf16>(ctx, p, whole);
    default: return launch_kind<EPI_BIAS_RESID, float>(ctx, p, whole);
    }
}

}  // namespace gpt2
