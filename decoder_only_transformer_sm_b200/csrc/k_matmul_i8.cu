// int8 x int8 products with a scale for each row of either operand:
//
//   out(m, n) = epilogue( (sum_k A(m, k) B(n, k)) sa[m] sb[n] )
//
// The sum is a 32-bit integer, exact for K <= 131071 (128^2 K < 2^31); it is
// rounded once to fp32 and multiplied by sa[m], then sb[n], in fp32.
//
// Three kernels, chosen by the shape and the alignment of the operands:
//   M <= 8, 16-byte rows   weight streaming (below): bound by reading B once
//   M > 8, 16-byte rows    tcgen05 (kind::i8) with TMA operands
//   other strides          dp4a on words put together from bytes
#include <cudaTypedefs.h>

#include <atomic>

#include "kernels.cuh"
#include "tc_ptx.cuh"

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

// ---------------------------------------------------------------- few rows
// Weight streaming for M <= MM rows: each warp takes RG rows of B at a time, a lane 16
// bytes of each per step (two steps in flight); the matching bytes of the M rows of A come from L1.
// Lane r * MM + m finishes element (m, n0 + r).
constexpr int GV_M = 8, GV_THREADS = 128;

// 16 bytes of a row of K, its bytes past K read as 0 (they belong to nobody).
__device__ __forceinline__ int4 load16(const int8_t* row, int j, int K) {
    const int left = K - 16 * j;
    if (left >= 16) return __ldg(reinterpret_cast<const int4*>(row) + j);
    int w[4] = {0, 0, 0, 0};
    for (int i = 0; i < left; ++i) w[i >> 2] |= (row[16 * j + i] & 0xff) << (8 * (i & 3));
    return make_int4(w[0], w[1], w[2], w[3]);
}

template <int KIND, typename O, int MM, int RG>
__global__ void __launch_bounds__(GV_THREADS) matmul_i8_rows_kernel(I8Product p) {
    const int lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * (GV_THREADS / 32) + (threadIdx.x >> 5)) * RG;
    if (n0 >= p.N) return;
    const int chunks = ceil_div(p.K, 16);
    const int8_t* b[RG];
#pragma unroll
    for (int r = 0; r < RG; ++r) b[r] = p.B + (long long)min(n0 + r, p.N - 1) * p.ldb;
    int acc[RG][MM] = {};
    for (int j0 = lane; j0 < chunks; j0 += 64) {
        int4 w[2][RG];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < RG; ++r)
                w[u][r] = j0 + 32 * u < chunks ? load16(b[r], j0 + 32 * u, p.K) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int j = j0 + 32 * u;
            if (j >= chunks) break;
#pragma unroll
            for (int m = 0; m < MM; ++m) {
                const int4 a = load16(p.A + (long long)min(m, p.M - 1) * p.lda, j, p.K);
#pragma unroll
                for (int r = 0; r < RG; ++r) {
                    acc[r][m] = __dp4a(a.x, w[u][r].x, acc[r][m]);
                    acc[r][m] = __dp4a(a.y, w[u][r].y, acc[r][m]);
                    acc[r][m] = __dp4a(a.z, w[u][r].z, acc[r][m]);
                    acc[r][m] = __dp4a(a.w, w[u][r].w, acc[r][m]);
                }
            }
        }
    }
    int mine = 0;
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int m = 0; m < MM; ++m) {
            const int t = __reduce_add_sync(0xffffffffu, acc[r][m]);
            if (lane == r * MM + m) mine = t;
        }
    const int m = lane % MM, n = n0 + lane / MM;
    if (lane < RG * MM && m < p.M && n < p.N) {
        const float bias = KIND != EPI_STORE ? p.bias[n] : 0.f;
        const float resid = KIND == EPI_BIAS_RESID ? p.resid[(long long)m * p.ldr + n] : 0.f;
        reinterpret_cast<O*>(p.out)[(long long)m * p.ldo + n] = finish<KIND, O>(mine, p.sa[m], p.sb[n], bias, resid);
    }
}

template <int KIND, typename O, int MM>
void launch_rows(const Ctx& ctx, const I8Product& p) {
    // four rows a warp once that leaves every SM eight warps, else one
    constexpr int W = GV_THREADS / 32;
    if (p.N >= 4 * 8 * ctx.num_sms)
        matmul_i8_rows_kernel<KIND, O, MM, 4><<<ceil_div(p.N, 4 * W), GV_THREADS, 0, ctx.stream>>>(p);
    else
        matmul_i8_rows_kernel<KIND, O, MM, 1><<<ceil_div(p.N, W), GV_THREADS, 0, ctx.stream>>>(p);
}

// ---------------------------------------------------------------- tensor cores
// Persistent kernel, a CTA walks output tiles of 128 x BN. Warp 0 streams 128-byte-wide
// K blocks of both operands with TMA into a ring of STAGES; warp 1 issues tcgen05.mma
// (kind::i8, 128 x BN x 32) into one of two int32 accumulators in tensor memory; the epilogue
// warps read the other one (a lane is a row), scale it and turn it around in a swizzled
// shared-memory buffer of their own, so that memory sees whole 128-byte row segments. Rows and
// columns past the operands come as zeros from TMA and are not stored.
template <int BN>
struct Tile {
    static constexpr int BM = 128, BK = 128;
    static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 6 : 8;
    static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI_WARPS = BN >= 128 ? 8 : 4;
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr int WCOLS = BN / (EPI_WARPS / 4);   // columns of a warp
    static constexpr int TMEM_COLS = 2 * BN;
};

struct TileCtl {
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base, abort;
};

constexpr int EPI_ROWS = 32 * 128;   // a warp's staging: 32 rows of 128 bytes
constexpr int EPI_COLS = 256;        // and 32 columns' scales and biases

template <int BN>
constexpr size_t tile_smem() {
    return (size_t)Tile<BN>::STAGES * Tile<BN>::STAGE_BYTES + Tile<BN>::EPI_WARPS * (EPI_ROWS + EPI_COLS) +
           sizeof(TileCtl) + 16;
}

struct TileGrid {
    int tiles_m, tiles_n, m_fastest, k_blocks;
    int vec_out, vec_resid;   // rows of out (resid) are whole 16-byte segments
    __device__ __forceinline__ void at(int u, int& mb, int& nb) const {
        mb = m_fastest ? u % tiles_m : u / tiles_n;
        nb = m_fastest ? u / tiles_m : u % tiles_n;
    }
};

// Byte offset of 16-byte segment c of row r in a buffer of 128-byte rows: the XOR spreads
// eight rows over all banks.
__device__ __forceinline__ uint32_t seg(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// A warp's buffer (32 rows x COLS elements of type E) to or from memory rows
// row0 .. row0 + 31, columns col0 .. col0 + COLS - 1 (those inside M x N).
template <typename E, int COLS, bool STORE>
__device__ __forceinline__ void move_rows(uint8_t* buf, E* mem, long long ld, int row0, int col0, int M, int N, int vec) {
    constexpr int PER = 16 / sizeof(E), SEGS = COLS / PER, STEP = 32 / SEGS;
    const int lane = threadIdx.x & 31;
    if (vec) {
        const int c = lane % SEGS, col = col0 + c * PER;
#pragma unroll
        for (int r = lane / SEGS; r < 32; r += STEP) {
            if (row0 + r >= M || col >= N) continue;
            E* g = mem + (long long)(row0 + r) * ld + col;
            E* s = reinterpret_cast<E*>(buf + seg(r, c));
            if (col + PER <= N) {
                if (STORE) *reinterpret_cast<uint4*>(g) = *reinterpret_cast<const uint4*>(s);
                else *reinterpret_cast<uint4*>(s) = *reinterpret_cast<const uint4*>(g);
            } else {
                for (int i = 0; i < N - col; ++i) {
                    if (STORE) g[i] = s[i];
                    else s[i] = g[i];
                }
            }
        }
        return;
    }
    for (int r = 0; r < 32 && row0 + r < M; ++r) {
#pragma unroll
        for (int c = lane; c < COLS; c += 32) {
            if (col0 + c >= N) continue;
            E* g = mem + (long long)(row0 + r) * ld + col0 + c;
            E* s = reinterpret_cast<E*>(buf + seg(r, c / PER)) + c % PER;
            if (STORE) *g = *s;
            else *s = *g;
        }
    }
}

template <int KIND, typename O, int BN>
__global__ void __launch_bounds__(Tile<BN>::THREADS, 1)
    matmul_i8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, I8Product p,
                        TileGrid grid, unsigned* status) {
    using L = Tile<BN>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* epi = smem + L::STAGES * L::STAGE_BYTES;
    TileCtl* ctl = reinterpret_cast<TileCtl*>(epi + L::EPI_WARPS * (EPI_ROWS + EPI_COLS));
    volatile uint32_t* abort = &ctl->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = grid.tiles_m * grid.tiles_n;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            tc::mbar_init(&ctl->full[s], 1);
            tc::mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&ctl->acc_full[b], 1);
            tc::mbar_init(&ctl->acc_empty[b], L::EPI_WARPS);
        }
        tc::mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        tc::fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&ctl->tmem_base, L::TMEM_COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            tc::tma_prefetch_desc(&tmA);
            tc::tma_prefetch_desc(&tmB);
            uint32_t it = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < tiles && ok; u += gridDim.x) {
                int mb, nb;
                grid.at(u, mb, nb);
                for (int kb = 0; kb < grid.k_blocks; ++kb, ++it) {
                    const int s = it % L::STAGES;
                    if (!tc::mbar_wait(&ctl->empty[s], ((it / L::STAGES) & 1) ^ 1, abort, status)) {
                        ok = false;
                        break;
                    }
                    tc::mbar_expect_tx(&ctl->full[s], L::STAGE_BYTES);
                    uint8_t* sa = smem + s * L::STAGE_BYTES;
                    tc::tma_load_2d(sa, &tmA, kb * L::BK, mb * L::BM, &ctl->full[s]);
                    tc::tma_load_2d(sa + L::A_BYTES, &tmB, kb * L::BK, nb * BN, &ctl->full[s]);
                }
            }
            if (!ok) {   // given up: nobody may wait for the loads in flight, and they must land before the CTA ends
                volatile uint32_t no_abort = 0;
                for (uint32_t j = it > L::STAGES ? it - L::STAGES : 0; j < it; ++j)
                    tc::mbar_wait(&ctl->full[j % L::STAGES], (j / L::STAGES) & 1, &no_abort, status);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = tc::idesc_i8_s32(L::BM, BN);
            uint32_t it = 0, acc_it = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < tiles && ok; u += gridDim.x, ++acc_it) {
                const uint32_t ab = acc_it & 1;
                if (!tc::mbar_wait(&ctl->acc_empty[ab], ((acc_it >> 1) & 1) ^ 1, abort, status)) break;
                tc::fence_after_sync();
                const uint32_t d_tmem = tmem + ab * BN;
                for (int kb = 0; kb < grid.k_blocks; ++kb, ++it) {
                    const int s = it % L::STAGES;
                    if (!tc::mbar_wait(&ctl->full[s], (it / L::STAGES) & 1, abort, status)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t a_base = tc::smem_u32(smem + s * L::STAGE_BYTES);
#pragma unroll
                    for (int kk = 0; kk < L::BK / 32; ++kk) {
                        const uint64_t da = tc::smem_desc_sw128(a_base + kk * 32, 16, 1024);
                        const uint64_t db = tc::smem_desc_sw128(a_base + L::A_BYTES + kk * 32, 16, 1024);
                        tc::mma_i8(d_tmem, da, db, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
                    }
                    tc::mma_commit(&ctl->empty[s]);
                }
                tc::mma_commit(&ctl->acc_full[ab]);
            }
            // every MMA issued has completed once `drain` fires; this wait ignores an abort (TMEM must not
            // be freed under running MMAs) but is bounded in time
            volatile uint32_t no_abort = 0;
            tc::mma_commit(&ctl->drain);
            tc::mbar_wait(&ctl->drain, 0, &no_abort, status);
        }
    } else {
        constexpr int FULL = 128 / (int)sizeof(O), CW = L::WCOLS < FULL ? L::WCOLS : FULL;   // columns of a staged chunk
        constexpr int PER = 16 / sizeof(O);
        const int ew = warp - 2, quarter = warp & 3, cbase = (ew >> 2) * L::WCOLS;
        uint8_t* buf = epi + ew * EPI_ROWS;
        float* cols = reinterpret_cast<float*>(epi + L::EPI_WARPS * EPI_ROWS + ew * EPI_COLS);
        uint32_t acc_it = 0;
        for (int u = blockIdx.x; u < tiles; u += gridDim.x, ++acc_it) {
            int mb, nb;
            grid.at(u, mb, nb);
            const uint32_t ab = acc_it & 1;
            const int row0 = mb * L::BM + quarter * 32, n0 = nb * BN + cbase;
            const float sa = row0 + lane < p.M ? p.sa[row0 + lane] : 0.f;
            // lane l holds the scale and the bias of column l of the next 32
            auto column = [&](const float* v, int c) { return c + lane < p.N ? __ldg(v + c + lane) : 0.f; };
            float sb = column(p.sb, n0), bias = KIND != EPI_STORE ? column(p.bias, n0) : 0.f;
            uint32_t ok = 0;
            if (lane == 0) ok = tc::mbar_wait(&ctl->acc_full[ab], (acc_it >> 1) & 1, abort, status) ? 1u : 0u;
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            tc::fence_after_sync();
            const uint32_t taddr = tmem + ab * BN + cbase + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
            for (int c0 = 0; c0 < L::WCOLS; c0 += CW) {
                if (n0 + c0 >= p.N || row0 >= p.M) break;
                if (KIND == EPI_BIAS_RESID) {
                    move_rows<float, CW, false>(buf, const_cast<float*>(p.resid), p.ldr, row0, n0 + c0, p.M, p.N,
                                                grid.vec_resid);
                    __syncwarp();
                }
#pragma unroll
                for (int h = 0; h < CW; h += 32) {
                    cols[lane] = sb;
                    if (KIND != EPI_STORE) cols[32 + lane] = bias;
                    __syncwarp();
                    const int next = n0 + c0 + h + 32;
                    sb = column(p.sb, next);
                    if (KIND != EPI_STORE) bias = column(p.bias, next);
                    float acc[32];
                    tc::tmem_ld_32x32b_x32(taddr + c0 + h, acc);
#pragma unroll
                    for (int c = 0; c < 32; c += PER) {
                        alignas(16) O v[PER];
                        uint8_t* at = buf + seg(lane, (h + c) / PER);
                        const float4 in = KIND == EPI_BIAS_RESID ? *reinterpret_cast<const float4*>(at)
                                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
                        const float r[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
                        for (int i = 0; i < PER; i += 4) {
                            const float4 s4 = *reinterpret_cast<const float4*>(cols + c + i);
                            const float4 b4 = KIND != EPI_STORE ? *reinterpret_cast<const float4*>(cols + 32 + c + i)
                                                                : make_float4(0.f, 0.f, 0.f, 0.f);
                            v[i] = finish<KIND, O>(__float_as_int(acc[c + i]), sa, s4.x, b4.x, r[0]);
                            v[i + 1] = finish<KIND, O>(__float_as_int(acc[c + i + 1]), sa, s4.y, b4.y, r[1]);
                            v[i + 2] = finish<KIND, O>(__float_as_int(acc[c + i + 2]), sa, s4.z, b4.z, r[2]);
                            v[i + 3] = finish<KIND, O>(__float_as_int(acc[c + i + 3]), sa, s4.w, b4.w, r[3]);
                        }
                        *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(v);
                    }
                    __syncwarp();
                }
                move_rows<O, CW, true>(buf, reinterpret_cast<O*>(p.out), p.ldo, row0, n0 + c0, p.M, p.N, grid.vec_out);
                __syncwarp();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl->acc_empty[ab]);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, L::TMEM_COLS);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 f = fn.load();
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        void* sym = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &sym, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(sym);
            fn.store(f);
        }
    }
    return f;
}

// int8 [rows][K], row stride ld; boxes of 128 bytes x box_rows, 128-byte swizzle.
bool make_map(CUtensorMap* m, const int8_t* ptr, long long rows, int K, long long ld, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Raises a kernel's shared-memory limit once on each device.
template <typename F>
void allow_smem(F* kernel, size_t bytes, std::atomic<unsigned long long>& done) {
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load() & bit)) return;
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    done.fetch_or(bit);
}

bool whole_segments(const void* p, long long ld, int es) { return ((uintptr_t)p & 15) == 0 && (ld * es) % 16 == 0; }

template <int KIND, typename O, int BN>
bool launch_tc(const Ctx& ctx, const I8Product& p) {
    using L = Tile<BN>;
    CUtensorMap ta, tb;
    if (!make_map(&ta, p.A, p.M, p.K, p.lda, L::BM) || !make_map(&tb, p.B, p.N, p.K, p.ldb, BN)) return false;
    TileGrid g;
    g.tiles_m = ceil_div(p.M, L::BM);
    g.tiles_n = ceil_div(p.N, BN);
    g.k_blocks = ceil_div(p.K, L::BK);
    // the operand of the fast index is read again for every slow block: the smaller one, which stays in L2
    g.m_fastest = p.M < p.N;
    g.vec_out = whole_segments(p.out, p.ldo, sizeof(O));
    g.vec_resid = KIND == EPI_BIAS_RESID && whole_segments(p.resid, p.ldr, 4);
    static std::atomic<unsigned long long> done{0};
    allow_smem(matmul_i8_tc_kernel<KIND, O, BN>, tile_smem<BN>(), done);
    matmul_i8_tc_kernel<KIND, O, BN><<<min(g.tiles_m * g.tiles_n, ctx.num_sms), L::THREADS, tile_smem<BN>(), ctx.stream>>>(
        ta, tb, p, g, ctx.status);
    return true;
}

template <int KIND, typename O>
bool launch_kind(const Ctx& ctx, const I8Product& p) {
    ++*ctx.launches;
    if (whole_segments(p.A, p.lda, 1) && whole_segments(p.B, p.ldb, 1)) {
        if (p.M <= GV_M) {
            if (p.M == 1) launch_rows<KIND, O, 1>(ctx, p);
            else if (p.M == 2) launch_rows<KIND, O, 2>(ctx, p);
            else if (p.M <= 4) launch_rows<KIND, O, 4>(ctx, p);
            else launch_rows<KIND, O, 8>(ctx, p);
            return true;
        }
        // the widest tile that still gives every SM one
        const int tiles_m = ceil_div(p.M, 128);
        auto fills = [&](int bn) { return (long long)tiles_m * ceil_div(p.N, bn) >= ctx.num_sms; };
        if (fills(256)) return launch_tc<KIND, O, 256>(ctx, p);
        if (fills(128)) return launch_tc<KIND, O, 128>(ctx, p);
        if (fills(64)) return launch_tc<KIND, O, 64>(ctx, p);
        return launch_tc<KIND, O, 32>(ctx, p);
    }
    const long long tiles = (long long)ceil_div(p.N, ST) * ceil_div(p.M, ST);
    matmul_i8_simt_kernel<KIND, O><<<(unsigned)tiles, 256, 0, ctx.stream>>>(p);
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
