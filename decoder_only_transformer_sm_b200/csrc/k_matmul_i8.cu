// int8 x int8 products with a scale for each row of either operand:
//
//   out(m, n) = epilogue( (sum_k A(m, k) B(n, k)) sa[m] sb[n] )
//
// The sum is a 32-bit integer, exact for K <= 131071 (128^2 K < 2^31); it is
// rounded once to fp32 and multiplied by sa[m], then sb[n], in fp32.
//
// Chosen by the shape and the alignment of the operands:
//   M <= 8                 weight streaming (k_matmul_i8_rows.cu): bound by reading B once. The tensor cores have a tile's
//                          start and chain of K blocks whatever M: 8 x 2304 x 768 2.8 us streamed, 5.5 with them, 8 x 6400
//                          x 1600 7.7 (weights from memory) and 10.6; only a vocabulary's width evens that out (x 50304 x
//                          768, weights from memory: M = 4 13.3 and 16.7, 5 16.6 and 14.1, 8 17.6 and 15.6)
//   M > 8, 16-byte rows    tcgen05 (kind::i8) with TMA operands
//   M > 8, other rows      tcgen05 with operands that warps put together from aligned words
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>

#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace gpt2 {

namespace {

// Two scaled sums through the epilogue, in packed arithmetic. GELU in the tanh form for fp32 results and
// in the logistic form for bf16 ones, as gelu_for.
template <int KIND, typename O>
__device__ __forceinline__ f32x2 finish2(int a0, int a1, f32x2 sa, f32x2 sb, f32x2 bias, f32x2 resid) {
    f32x2 u = mul2(pk2((float)a0, (float)a1), sa);
    u = KIND == EPI_STORE ? mul2(u, sb) : fma2(u, sb, bias);
    if (KIND == EPI_BIAS_RESID) u = add2(u, resid);
    if (KIND == EPI_BIAS_GELU) {
        float x, y;
        upk2(u, x, y);
        if (sizeof(O) == 4) {
            u = pk2(gelu_tanh(x), gelu_tanh(y));
        } else {   // u / (1 + 2^(u (K1 + K2 u^2))), the logistic form of the tanh one
            constexpr float K1 = -2.0f * 0.7978845608028654f * 1.4426950408889634f, K2 = K1 * 0.044715f;
            float e0, e1;
            upk2(mul2(u, fma2(mul2(u, u), pk2(K2, K2), pk2(K1, K1))), e0, e1);
            upk2(add2(pk2(ex2_approx(e0), ex2_approx(e1)), pk2(1.f, 1.f)), e0, e1);
            u = mul2(u, pk2(rcp_approx(e0), rcp_approx(e1)));
        }
    }
    return u;
}

// ---------------------------------------------------------------- tensor cores
// From a CUDA graph, three sets of operands in turn: 16384 x 2304 x 768 with bias 30 us (1.9 POP/s), 16384 x 768 x 768 with
// residual 29 us, 2048 x 6400 x 1600 with GELU 25 us; in long runs, under the power cap, the first takes 36.5 us (1.6 POP/s),
// the last 28. 8192^3 400 us (2.7 POP/s; 330 us with operands of zeros: power). With bf16 results the epilogue is the longer
// part of a tile up to some ten K blocks: 16384 x 2304 takes 18 us with one, 30 with six, 92 with 25 (3.1 a block and 14).
//
// Persistent kernel: a CTA, or a pair of CTAs (a cluster of two, cta_group::2), walks output
// tiles of 128 CTAS x BN. Warp 0 streams 128-byte-wide K blocks of both operands with TMA into a
// ring of STAGES; warp 1 (of the pair's first CTA) issues tcgen05.mma (kind::i8, 128 CTAS x BN x 32)
// into one of two int32 accumulators in tensor memory; the epilogue warps read the other one (a lane
// is a row), scale it and turn it around in shared memory, 32 rows of 128 bytes at a time, which leave
// by a TMA store or as 16-byte stores of the warp (single elements where rows are not whole 16-byte
// segments). Rows and columns past the operands come as zeros from TMA and are not stored.
// Rows that start anywhere (BYTES): eight more warps take the place of the TMA loads.
// Of tiles up to 128 columns two threads issue the MMAs, every other K block each: one gets one MMA
// per 120 cycles or so through, however narrow it is. Their two sums are added in the epilogue (128 x 768
// x 6400: 14.8 us, with one thread 18.3; then a CTA's 55 bytes a cycle of loads bound it).
// A pair shares its B rows, so a K block costs each CTA 32 KB of shared memory and of L2
// traffic for 256 x 256 outputs a pair, where one CTA alone needs 48 KB for 128 x 256.
template <int BN, int CTAS, bool BYTES = false>
struct Tile {
    static constexpr int BM = 128, BK = 128;   // rows of a CTA
    static constexpr int B_ROWS = BN / CTAS;   // B rows in a CTA's shared memory
    static constexpr int A_BYTES = BM * BK, B_BYTES = B_ROWS * BK, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN >= 256 ? 5 : BN >= 128 ? 4 : 8;   // even where two threads issue MMAs
    static constexpr int EPI_WARPS = BN >= 256 ? 16 : BN >= 128 ? 8 : 4;
    static constexpr int BYTE_WARPS = BYTES ? 8 : 0;
    static constexpr int ISSUERS = BN <= 128 ? 2 : 1;    // threads that issue MMAs, each into a sum of its own
    static constexpr int THREADS = 32 * (1 + ISSUERS + EPI_WARPS + BYTE_WARPS);
    static constexpr int WCOLS = BN / (EPI_WARPS / 4);   // columns of a warp
    static constexpr int TMEM_COLS = 2 * ISSUERS * BN;
    static constexpr int EPI_BUFS = BN >= 256 ? 1 : 2;   // a warp's staging buffers
    static constexpr int EPI_COLS = 8 * BN;              // bytes of the tile's column scales and biases
};

struct TileCtl {
    uint64_t full[8], empty[8], acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base, abort;
};

constexpr int EPI_ROWS = 32 * 128;   // a staging buffer: 32 rows of 128 bytes

template <typename L>
constexpr size_t tile_smem() {
    return (size_t)L::STAGES * L::STAGE_BYTES + L::EPI_WARPS * L::EPI_BUFS * EPI_ROWS + L::EPI_COLS + sizeof(TileCtl) + 16;
}

struct TileGrid {
    int tiles_m, tiles_n, m_fastest, k_blocks;
    int vec_out, vec_resid;   // rows of out (resid) are whole 16-byte segments
    int tma_out;              // results leave by TMA stores
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
    const int c = lane % SEGS, col = col0 + c * PER;
    if (vec && row0 + 32 <= M && col0 + COLS <= N) {   // nothing cut off: all loads, then all stores
        uint4 t[32 / STEP];
        char* g = reinterpret_cast<char*>(mem + (long long)(row0 + lane / SEGS) * ld + col);
        const long long pitch = STEP * ld * (long long)sizeof(E);
#pragma unroll
        for (int i = 0; i < 32 / STEP; ++i)
            t[i] = STORE ? *reinterpret_cast<const uint4*>(buf + seg(lane / SEGS + i * STEP, c))
                         : *reinterpret_cast<const uint4*>(g + i * pitch);
#pragma unroll
        for (int i = 0; i < 32 / STEP; ++i)
            *reinterpret_cast<uint4*>(STORE ? reinterpret_cast<uint8_t*>(g + i * pitch)
                                            : buf + seg(lane / SEGS + i * STEP, c)) = t[i];
        return;
    }
    if (vec) {
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
    // rows that start anywhere: an element a lane, eight rows loaded before the first is stored
#pragma unroll 1
    for (int e = lane; e < COLS; e += 32) {
        if (col0 + e >= N) continue;
        E* g = mem + (long long)row0 * ld + col0 + e;
        uint8_t* at = buf + (e % PER) * sizeof(E);
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += 8) {
            E t[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (row0 + r0 + r < M)
                    t[r] = STORE ? *reinterpret_cast<const E*>(at + seg(r0 + r, e / PER)) : g[(r0 + r) * ld];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (row0 + r0 + r < M)
                    *(STORE ? g + (r0 + r) * ld : reinterpret_cast<E*>(at + seg(r0 + r, e / PER))) = t[r];
        }
    }
}

// 16 bytes of results.
__device__ __forceinline__ void put(uint8_t* at, const f32x2 (&v)[2], float) {
    *reinterpret_cast<ulonglong2*>(at) = ulonglong2{v[0], v[1]};
}
__device__ __forceinline__ void put(uint8_t* at, const f32x2 (&v)[4], bf16) {
    unsigned u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x, y;
        upk2(v[i], x, y);
        const __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
        u[i] = *reinterpret_cast<const unsigned*>(&t);
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(u[0], u[1], u[2], u[3]);
}

// One warp's part of a K block of 128 rows from row0 on of an operand whose rows start at any
// byte, in the 128-byte-swizzle layout that TMA writes: pieces of 16 bytes, four a lane, each put
// together from five aligned 32-bit words, all loads before the first store. Rows past the
// operand are read as its last one (and not stored). EDGE: the first K block, and those near the
// rows' end: what lies past K counts as zero, and the pieces whose words would touch a byte outside
// the operand (at its first and its last byte only) are put together from single bytes.
struct Gather {
    const int8_t* base;
    long long ld;
    int row0, rows;
    static constexpr int PIECES = 128 * 8 / (8 * 32);   // 8 warps
    struct Words {
        unsigned u[PIECES][5];
    };
    __device__ __forceinline__ const int8_t* piece(int i, int k0) const {
        return base + (long long)min(row0 + (i >> 3), rows - 1) * ld + k0 + 16 * (i & 7);
    }
    __device__ __forceinline__ bool inside(const int8_t* word, int K) const {
        return word >= base && word + 20 <= base + (long long)(rows - 1) * ld + K;
    }
    template <bool EDGE>
    __device__ __forceinline__ void load(Words& w, int k0, int K, int i0) const {
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int i = i0 + 256 * j;
            const int8_t* at = piece(i, k0);
            const int8_t* word = at - ((uintptr_t)at & 3);
            const bool ok = !EDGE || inside(word, K);
#pragma unroll
            for (int x = 0; x < 5; ++x) w.u[j][x] = ok ? __ldg(reinterpret_cast<const unsigned*>(word) + x) : 0u;
        }
    }
    template <bool EDGE>
    __device__ __forceinline__ void store(uint8_t* dst, const Words& w, int k0, int K, int i0) const {
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int i = i0 + 256 * j;
            const int8_t* at = piece(i, k0);
            const int off = (int)((uintptr_t)at & 3);
            unsigned q[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) q[x] = __funnelshift_r(w.u[j][x], w.u[j][x + 1], 8 * off);
            if (EDGE) {
                const int left = K - (k0 + 16 * (i & 7));   // bytes of the row from here on
                if (left > 0 && !inside(at - off, K)) {
                    q[0] = q[1] = q[2] = q[3] = 0;
#pragma unroll 1
                    for (int b = 0; b < min(left, 16); ++b) {
                        const unsigned v = (unsigned)(uint8_t)at[b] << (8 * (b & 3));
#pragma unroll
                        for (int x = 0; x < 4; ++x) q[x] |= (b >> 2) == x ? v : 0u;
                    }
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int n = left - 4 * x;
                    q[x] = n >= 4 ? q[x] : n <= 0 ? 0u : q[x] & ((1u << (8 * n)) - 1);
                }
            }
            *reinterpret_cast<uint4*>(dst + seg(i >> 3, i & 7)) = make_uint4(q[0], q[1], q[2], q[3]);
        }
    }
};

template <int KIND, typename O, int BN, int CTAS, bool BYTES = false>
__global__ void __launch_bounds__(Tile<BN, CTAS, BYTES>::THREADS, 1)
    matmul_i8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmO, I8Product p, TileGrid grid, unsigned* status) {
    using L = Tile<BN, CTAS, BYTES>;
    constexpr bool PAIR = CTAS == 2;
    static_assert(!BYTES || (BN == 128 && CTAS == 1), "rows that start anywhere: 128 x 128 tiles");
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* epi = smem + L::STAGES * L::STAGE_BYTES;
    TileCtl* ctl = reinterpret_cast<TileCtl*>(epi + L::EPI_WARPS * L::EPI_BUFS * EPI_ROWS + L::EPI_COLS);
    volatile uint32_t* abort = &ctl->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = grid.tiles_m * grid.tiles_n;
    const int rank = PAIR ? (int)tc::cluster_rank() : 0;
    const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::STAGES; ++s) {
            tc::mbar_init(&ctl->full[s], BYTES ? L::BYTE_WARPS : 1);
            tc::mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&ctl->acc_full[b], L::ISSUERS);
            tc::mbar_init(&ctl->acc_empty[b], CTAS * L::EPI_WARPS);
        }
        tc::mbar_init(&ctl->drain, L::ISSUERS);
        ctl->abort = 0;
        tc::fence_barrier_init();
    }
    griddep_wait();   // also before the allocation: tensor memory is not held while the kernel before may want it
    if (warp == 1) {
        if (PAIR) {
            tc::tmem_alloc_pair(&ctl->tmem_base, L::TMEM_COLS);
            tc::tmem_relinquish_pair();
        } else {
            tc::tmem_alloc(&ctl->tmem_base, L::TMEM_COLS);
            tc::tmem_relinquish();
        }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (PAIR) tc::cluster_sync();
    else __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = ctl->tmem_base;
    griddep_launch();

    constexpr int LAST = 2 + L::EPI_WARPS + L::BYTE_WARPS;   // the second issuing warp
    if (BYTES && warp >= 2 + L::EPI_WARPS && warp < LAST) {
        const int bw = warp - 2 - L::EPI_WARPS;
        uint32_t it = 0, ok = 1;
        for (int u = first; u < tiles && ok; u += step) {
            int mb, nb;
            grid.at(u, mb, nb);
            for (int kb = 0; kb < grid.k_blocks; ++kb, ++it) {
                const int s = it % L::STAGES;
                if (lane == 0) ok = tc::mbar_wait(&ctl->empty[s], ((it / L::STAGES) & 1) ^ 1, abort, status) ? 1u : 0u;
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                uint8_t* sa = smem + s * L::STAGE_BYTES;
                const Gather ga = {p.A, p.lda, mb * L::BM, p.M}, gb = {p.B, p.ldb, nb * BN, p.N};
                const int k0 = kb * L::BK, i0 = bw * 32 + lane;
                Gather::Words wa, wb;
                if (kb > 0 && k0 + 132 <= p.K) {   // (a piece's last word may reach three bytes past it)
                    ga.load<false>(wa, k0, p.K, i0);
                    gb.load<false>(wb, k0, p.K, i0);
                    ga.store<false>(sa, wa, k0, p.K, i0);
                    gb.store<false>(sa + L::A_BYTES, wb, k0, p.K, i0);
                } else {
                    ga.load<true>(wa, k0, p.K, i0);
                    gb.load<true>(wb, k0, p.K, i0);
                    ga.store<true>(sa, wa, k0, p.K, i0);
                    gb.store<true>(sa + L::A_BYTES, wb, k0, p.K, i0);
                }
                tc::fence_proxy_async_smem();   // the MMA reads through the async proxy
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl->full[s]);
            }
        }
    } else if (warp == 0) {
        if (lane == 0 && !BYTES) {
            tc::tma_prefetch_desc(&tmA);
            tc::tma_prefetch_desc(&tmB);
            uint32_t it = 0;
            bool ok = true;
            for (int u = first; u < tiles && ok; u += step) {
                int mb, nb;
                grid.at(u, mb, nb);
                const int m0 = (mb * CTAS + rank) * L::BM, n0 = nb * BN + rank * L::B_ROWS;
                for (int kb = 0; kb < grid.k_blocks; ++kb, ++it) {
                    const int s = it % L::STAGES;
                    if (!tc::mbar_wait(&ctl->empty[s], ((it / L::STAGES) & 1) ^ 1, abort, status)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = smem + s * L::STAGE_BYTES;
                    if (PAIR) {
                        // both CTAs' bytes are counted on the first one's barrier
                        const uint32_t bar = tc::map_rank(&ctl->full[s], 0);
                        if (rank == 0) tc::mbar_expect_tx(&ctl->full[s], 2 * L::STAGE_BYTES);
                        tc::tma_load_2d_pair(sa, &tmA, kb * L::BK, m0, bar);
                        tc::tma_load_2d_pair(sa + L::A_BYTES, &tmB, kb * L::BK, n0, bar);
                    } else {
                        tc::mbar_expect_tx(&ctl->full[s], L::STAGE_BYTES);
                        tc::tma_load_2d(sa, &tmA, kb * L::BK, m0, &ctl->full[s]);
                        tc::tma_load_2d(sa + L::A_BYTES, &tmB, kb * L::BK, n0, &ctl->full[s]);
                    }
                }
            }
            if (!ok) {   // given up: nobody may wait for the loads in flight, and they must land before the CTA ends
                volatile uint32_t no_abort = 0;
                if (rank == 0) {
                    for (uint32_t j = it > L::STAGES ? it - L::STAGES : 0; j < it; ++j)
                        tc::mbar_wait(&ctl->full[j % L::STAGES], (j / L::STAGES) & 1, &no_abort, status);
                } else {   // their barrier is the other CTA's: 1 ms
                    const unsigned long long t0 = tc::globaltimer();
                    while (tc::globaltimer() - t0 < 1000000ull) {
                    }
                }
            }
            if (PAIR && rank == 1) {
                // The first CTA's MMAs also arrive here: its shared memory must outlive the last of these arrivals, those
                // that free the last stages and `drain` (acc_full's are the epilogue's). Waited for after the last load,
                // so that the limit is on the last K blocks, not on the whole product.
                volatile uint32_t no_abort = 0;
                for (uint32_t j = it > L::STAGES ? it - L::STAGES : 0; j < it && ok; ++j)
                    ok = tc::mbar_wait(&ctl->empty[j % L::STAGES], (j / L::STAGES) & 1, abort, status);
                tc::mbar_wait(&ctl->drain, 0, &no_abort, status);
            }
        }
    } else if (warp == 1 || warp == LAST) {
        if (lane == 0 && rank == 0) {
            // Every other K block of the CTA's whole run, so that a stage is always the same thread's: one that saw
            // only every other phase of a barrier could take an old one's parity for its own.
            const uint32_t mine = warp == 1 ? 0 : 1;
            static_assert(L::ISSUERS == 1 || L::STAGES % L::ISSUERS == 0, "a stage belongs to one issuing thread");
            constexpr uint32_t idesc = tc::idesc_i8_s32(L::BM * CTAS, BN);
            uint32_t it = 0, acc_it = 0;
            bool ok = true;
            for (int u = first; u < tiles && ok; u += step, ++acc_it) {
                const uint32_t ab = acc_it & 1;
                if (!tc::mbar_wait(&ctl->acc_empty[ab], ((acc_it >> 1) & 1) ^ 1, abort, status)) break;
                tc::fence_after_sync();
                const uint32_t d_tmem = tmem + (ab * L::ISSUERS + mine) * BN;
                uint32_t add = 0;   // the tile's first MMA overwrites
                for (int kb = 0; kb < grid.k_blocks; ++kb, ++it) {
                    if (L::ISSUERS > 1 && it % L::ISSUERS != mine) continue;
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
                        if (PAIR) tc::mma_i8_pair(d_tmem, da, db, idesc, add);
                        else tc::mma_i8(d_tmem, da, db, idesc, add);
                        add = 1;
                    }
                    if (PAIR) tc::mma_commit_pair(&ctl->empty[s]);
                    else tc::mma_commit(&ctl->empty[s]);
                }
                if (PAIR) tc::mma_commit_pair(&ctl->acc_full[ab]);
                else tc::mma_commit(&ctl->acc_full[ab]);
            }
            // every MMA issued has completed once `drain` fires; this wait ignores an abort (TMEM must not
            // be freed under running MMAs) but is bounded in time
            volatile uint32_t no_abort = 0;
            if (PAIR) tc::mma_commit_pair(&ctl->drain);
            else tc::mma_commit(&ctl->drain);
            tc::mbar_wait(&ctl->drain, 0, &no_abort, status);
        }
    } else {
        constexpr int CW = 128 / (int)sizeof(O);   // columns of a chunk
        constexpr int PER = 16 / sizeof(O);
        const bool tma_out = grid.tma_out;
        const int ew = warp - 2, quarter = warp & 3, cbase = (ew >> 2) * L::WCOLS;
        uint8_t* bufs = epi + ew * L::EPI_BUFS * EPI_ROWS;
        float* cols = reinterpret_cast<float*>(epi + L::EPI_WARPS * L::EPI_BUFS * EPI_ROWS) + 2 * cbase;
        // The next tile's row scale, and of the four warps that share columns one's scale or bias each:
        // warp `quarter` of them holds values 32 quarter + lane + 128 i of scales, then biases.
        constexpr int NV = (KIND == EPI_STORE ? 1 : 2) * L::WCOLS, NC = (NV + 127) / 128;
        float sa = 0.f, col_value[NC];
        auto fetch = [&](int u) {
            if (u >= tiles) return;
            int mb, nb;
            grid.at(u, mb, nb);
            const int row = (mb * CTAS + rank) * L::BM + quarter * 32 + lane;
            sa = row < p.M ? __ldg(p.sa + row) : 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int j = 128 * i + 32 * quarter + lane, col = nb * BN + cbase + j % L::WCOLS;
                col_value[i] = j < NV && col < p.N ? __ldg((j < L::WCOLS ? p.sb : p.bias) + col) : 0.f;
            }
        };
        fetch(first);
        uint32_t acc_it = 0, chunk = 0, live = 1;
        for (int u = first; u < tiles; u += step, ++acc_it) {
            int mb, nb;
            grid.at(u, mb, nb);
            const uint32_t ab = acc_it & 1;
            const int row0 = (mb * CTAS + rank) * L::BM + quarter * 32, n0 = nb * BN + cbase;
            tc::named_barrier(1 + (ew >> 2), 128);   // the last tile's values have been read
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (128 * i + 32 * quarter + lane < NV) cols[128 * i + 32 * quarter + lane] = col_value[i];
            const f32x2 row_scale = pk2(sa, sa);
            tc::named_barrier(1 + (ew >> 2), 128);
            fetch(u + step);
            // The buffer for columns c0 .. once its last store has read it, with the residual in it.
            // The first chunk's is made ready before the accumulator is.
            auto ready = [&](int c0) {
                if (tma_out) {
                    if (lane == 0) tc::bulk_wait_read<L::EPI_BUFS - 1>();
                    __syncwarp();
                }
                if (KIND == EPI_BIAS_RESID) {
                    move_rows<float, CW, false>(bufs + (chunk % L::EPI_BUFS) * EPI_ROWS, const_cast<float*>(p.resid),
                                                p.ldr, row0, n0 + c0, p.M, p.N, grid.vec_resid);
                    __syncwarp();
                }
            };
            const bool any = n0 < p.N && row0 < p.M;
            if (any) ready(0);
            uint32_t ok = live;
            if (lane == 0 && live) ok = tc::mbar_wait(&ctl->acc_full[ab], (acc_it >> 1) & 1, abort, status) ? 1u : 0u;
            live = __shfl_sync(0xffffffffu, ok, 0);
            if (!live) continue;   // given up: on to the other warps' barriers of the tiles left
            tc::fence_after_sync();
            auto release = [&] {   // this warp has read its part of the accumulator
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) tc::mbar_arrive_remote(tc::map_rank(&ctl->acc_empty[ab], 0));
                    else tc::mbar_arrive(&ctl->acc_empty[ab]);
                }
            };
            const uint32_t taddr = tmem + ab * L::ISSUERS * BN + cbase + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
            for (int c0 = 0; c0 < L::WCOLS; c0 += CW, ++chunk) {
                if (n0 + c0 >= p.N || row0 >= p.M) break;
                if (c0 > 0) ready(c0);
                uint8_t* buf = bufs + (chunk % L::EPI_BUFS) * EPI_ROWS;
#pragma unroll
                for (int h = 0; h < CW; h += 32) {
                    float acc[32];
                    if (L::ISSUERS > 1 && grid.k_blocks > 1) {
                        float more[32];
                        tc::tmem_ld2_32x32b_x32(taddr + c0 + h, taddr + BN + c0 + h, acc, more);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            acc[i] = __int_as_float(__float_as_int(acc[i]) + __float_as_int(more[i]));
                    } else {   // one K block: the sum of the thread whose turn it was
                        const uint32_t of = L::ISSUERS > 1 ? acc_it % L::ISSUERS : 0;
                        tc::tmem_ld_32x32b_x32(taddr + of * BN + c0 + h, acc);
                    }
#pragma unroll
                    for (int c = 0; c < 32; c += PER) {
                        uint8_t* at = buf + seg(lane, (h + c) / PER);
                        f32x2 v[PER / 2], in[2] = {};
                        if (KIND == EPI_BIAS_RESID) {
                            const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(at);
                            in[0] = q.x;
                            in[1] = q.y;
                        }
#pragma unroll
                        for (int i = 0; i < PER; i += 4) {
                            const float* col = cols + c0 + h + c + i;
                            const ulonglong2 s4 = *reinterpret_cast<const ulonglong2*>(col);
                            const ulonglong2 b4 = KIND != EPI_STORE ? *reinterpret_cast<const ulonglong2*>(col + L::WCOLS)
                                                                    : ulonglong2{0, 0};
                            const int* a4 = reinterpret_cast<const int*>(acc) + c + i;
                            v[i / 2] = finish2<KIND, O>(a4[0], a4[1], row_scale, s4.x, b4.x, in[0]);
                            v[i / 2 + 1] = finish2<KIND, O>(a4[2], a4[3], row_scale, s4.y, b4.y, in[1]);
                        }
                        put(at, v, O());
                    }
                }
                __syncwarp();
                if (c0 + CW >= L::WCOLS || n0 + c0 + CW >= p.N) release();
                if (tma_out) {
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tc::tma_store_2d(&tmO, buf, n0 + c0, row0);
                        tc::bulk_commit();
                    }
                } else {
                    move_rows<O, CW, true>(buf, reinterpret_cast<O*>(p.out), p.ldo, row0, n0 + c0, p.M, p.N, grid.vec_out);
                    __syncwarp();
                }
            }
            if (!any) release();
        }
        if (lane == 0) tc::bulk_wait<0>();
    }
    tc::fence_before_sync();
    __syncwarp();
    if (PAIR) tc::cluster_sync();   // nobody's shared or tensor memory is used any more
    else __syncthreads();
    if (warp == 1) {
        if (PAIR) tc::tmem_dealloc_pair(tmem, L::TMEM_COLS);
        else tc::tmem_dealloc(tmem, L::TMEM_COLS);
    }
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

// [rows][cols] with row stride ld (elements); boxes of box_cols (128 bytes) x box_rows, 128-byte swizzle.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, int es, const void* ptr, long long rows, int cols, long long ld,
              int box_cols, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * es};
    cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, type, 2, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

template <int KIND, typename O, int BN, int CTAS, bool BYTES = false>
bool launch_tc(const Ctx& ctx, const I8Product& p) {
    using L = Tile<BN, CTAS, BYTES>;
    constexpr int CW = 128 / (int)sizeof(O);
    CUtensorMap ta = {}, tb = {}, to = {};   // zeros where not used
    const CUtensorMapDataType I8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    TileGrid g;
    g.tiles_m = ceil_div(p.M, L::BM * CTAS);
    g.tiles_n = ceil_div(p.N, BN);
    g.k_blocks = ceil_div(p.K, L::BK);
    // the operand of the fast index is read again for every slow block: the smaller one, which stays in L2
    g.m_fastest = p.M < p.N;
    g.vec_out = whole_segments(p.out, p.ldo, sizeof(O));
    g.vec_resid = KIND == EPI_BIAS_RESID && whole_segments(p.resid, p.ldr, 4);
    if (!BYTES && (!make_map(&ta, I8, 1, p.A, p.M, p.K, p.lda, L::BK, L::BM) ||
        !make_map(&tb, I8, 1, p.B, p.N, p.K, p.ldb, L::BK, L::B_ROWS)))
        return false;
    // TMA stores are asynchronous, but their bursts hold up the operands' loads: they pay for fp32 results
    // and short sums (16384 x 2304 in bf16: K = 128 19.2 us against 22.2 with plain stores, K = 768 31.7 against 30.4;
    // 16384 x 768 x 768 in fp32 with residual 28.7 against 31.1).
    // They write whole 16-byte segments, so a row that ends inside one (its padding is the caller's) is not theirs.
    g.tma_out = g.vec_out && (p.N * sizeof(O)) % 16 == 0 && (sizeof(O) == 4 || g.k_blocks <= 4);
    if (g.tma_out) {
        if (!make_map(&to, sizeof(O) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      sizeof(O), p.out, p.M, p.N, p.ldo, CW, 32))
            return false;
    }
    auto kernel = matmul_i8_tc_kernel<KIND, O, BN, CTAS, BYTES>;
    static std::atomic<unsigned long long> done{0};
    allow_smem(kernel, tile_smem<L>(), done);
    return launch_pdl_clusters(ctx, CTAS, kernel, dim3(CTAS * min(g.tiles_m * g.tiles_n, ctx.num_sms / CTAS)),
                               dim3(L::THREADS), tile_smem<L>(), ta, tb, to, p, g, ctx.status) == cudaSuccess;
}

template <int KIND, typename O>
bool launch_kind(const Ctx& ctx, const I8Product& p, bool whole) {
    if (whole) {
        // The tile width by its time: a start, then for each round of tiles over the SMs the K blocks and what
        // of the epilogue the next tile's products do not cover. A K block costs narrow tiles hardly less (their A
        // rows are as many, and an MMA of few columns takes as long to issue); they win while they fill SMs that
        // wide ones leave idle. (us, measured with both operands in L2: 64 x 2304 x 768 4.4 with 64 columns, 7.2
        // with a pair; 1024 x 2304 x 768 7.4 with 64, 5.4 with 128, 8.2 with a pair; 256 x 50304 x 768 26.8, 18.4, 14.2.)
        const int kb = ceil_div(p.K, 128);
        auto time = [&](int bm, int bn, int units, float start, float block, float tile) {
            const float tiles = (float)ceil_div(p.M, bm) * (float)ceil_div(p.N, bn);
            return start + ceilf(tiles / units) * (kb * block + tile);
        };
        const float t256 = time(256, 256, ctx.num_sms / 2, 3.9f, 0.36f, 1.1f);
        const float t128 = time(128, 128, ctx.num_sms, 2.5f, 0.26f, 0.7f);
        const float t64 = time(128, 64, ctx.num_sms, 2.4f, 0.24f, 0.6f);
        if (t256 <= t128 && t256 <= t64) return launch_tc<KIND, O, 256, 2>(ctx, p);
        return t128 <= t64 ? launch_tc<KIND, O, 128, 1>(ctx, p) : launch_tc<KIND, O, 64, 1>(ctx, p);
    }
    return launch_tc<KIND, O, 128, 1, true>(ctx, p);
}

}  // namespace

bool launch_matmul_i8(const Ctx& ctx, const I8Product& product) {
    ++*ctx.launches;
    // A single row's stride is never used, so it must not decide the path: one token of K bytes, packed, would send
    // padded weights through the rows that start anywhere (1 x 50304 x 763: 41 us, 20 as whole segments).
    I8Product p = product;
    if (p.M == 1) p.lda = (p.K + 15) / 16 * 16;
    if (p.N == 1) p.ldb = (p.K + 15) / 16 * 16;
    const bool whole = whole_segments(p.A, p.lda, 1) && whole_segments(p.B, p.ldb, 1), f32 = p.out_f32;
    if (p.M <= I8_FEW_ROWS) {
        launch_matmul_i8_rows(ctx, p, whole);
        return true;
    }
    switch (p.kind) {
    case EPI_STORE: return f32 ? launch_kind<EPI_STORE, float>(ctx, p, whole) : launch_kind<EPI_STORE, bf16>(ctx, p, whole);
    case EPI_BIAS: return f32 ? launch_kind<EPI_BIAS, float>(ctx, p, whole) : launch_kind<EPI_BIAS, bf16>(ctx, p, whole);
    case EPI_BIAS_GELU:
        return f32 ? launch_kind<EPI_BIAS_GELU, float>(ctx, p, whole) : launch_kind<EPI_BIAS_GELU, bf16>(ctx, p, whole);
    case EPI_BIAS_RESID: return launch_kind<EPI_BIAS_RESID, float>(ctx, p, whole);
    default: return false;
    }
}

}  // namespace gpt2
